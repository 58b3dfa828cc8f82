"""The paged 8-bit cache without a GPU: refusals of the C entry points before any launch,
workspace sizes, and the oracle's number formats pinned to independent statements."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_linear_sm_b200 as sla
from block_sparse_linear_sm_b200 import workloads as wl
from oracle import cache_oracle as co

IA, UN, WS = sla.SLA_ERR_INVALID_ARG, sla.SLA_ERR_UNSUPPORTED, sla.SLA_ERR_WORKSPACE


def config(**kw):
    base = dict(B=2, H=8, H_kv=2, d=128, n_pages=16, max_blocks=8)
    base.update(kw)
    return wl.CacheConfig(**base)


def ref(c):
    return ctypes.byref(sla.make_cache_config(c))


def buffers(**kw):
    """A cache of addresses that are never dereferenced."""
    m = sla.sla_cache()
    for name, a in dict(k=256, v=512, k_scale=16, v_scale=16, k_mean=16, weight=16, block_table=16,
                        status=256).items():
        setattr(m, name, kw.get(name, a))
    return ctypes.byref(m)


BAD = [
    (dict(), sla.SLA_OK),
    (dict(B=0), IA), (dict(H=0, H_kv=0), IA), (dict(H_kv=0), IA), (dict(d=0), IA), (dict(n_pages=0), IA),
    (dict(max_blocks=0), IA), (dict(H=7), IA), (dict(kind=2), IA), (dict(kind=-1), IA),
    (dict(scale=-1.0), IA), (dict(scale=float("nan")), IA), (dict(scale=float("inf")), IA),
    (dict(d=96), UN), (dict(B=1025), UN), (dict(B=1024), sla.SLA_OK), (dict(H=2048, H_kv=2), UN),
    (dict(max_blocks=4097), UN), (dict(max_blocks=4096), sla.SLA_OK),
    (dict(n_pages=(1 << 24)), UN), (dict(n_pages=(1 << 24) - 1), sla.SLA_OK),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_cache_config_checks(kw, code):
    c = config(**kw)
    assert sla.sla_cache_validate_config(c) == code
    ok = code == sla.SLA_OK
    assert (sla.sla_cache_attend_workspace_bytes(c, 1) > 0) == ok
    assert (sla.sla_cache_evict_workspace_bytes(c, 64) > 0) == ok
    if not ok:
        L = sla.lib()
        assert L.sla_cache_append(16, 16, ref(c), buffers(), 1, 16, None, None, None) == code
        assert L.sla_cache_route(16, ref(c), buffers(), 1, 16, None, 4, 16, None) == code
        assert L.sla_cache_attend(16, ref(c), buffers(), 1, 16, None, None, 0, 0, 32, 256, 1 << 30, None) == code
        assert L.sla_cache_evict(ref(c), buffers(), 16, 64, 0, 0, 16, 16, 16, 32, 256, 1 << 30, None) == code


def test_null_config_and_struct_layouts():
    assert sla.lib().sla_cache_validate_config(None) == IA
    src = open(sla.HEADER_PATH).read()
    import re
    for struct, cls in (("sla_cache_config", sla.sla_cache_config), ("sla_cache", sla.sla_cache)):
        end = src.index("} %s;" % struct)
        body = src[src.rindex("typedef struct {", 0, end):end]
        names = re.findall(r"^\s*(?:const\s+)?(?:int32_t|float|void)\s*\*?\s*(\w+);", body, re.M)
        assert names == [f for f, _ in cls._fields_]


MISSING = ["k", "v", "k_scale", "v_scale", "block_table", "status"]


@pytest.mark.parametrize("kw", [{n: None} for n in MISSING] + [dict(k=264), dict(v=520), dict(k_scale=18),
                         dict(k_mean=20), dict(weight=20), dict(block_table=18), dict(status=128), dict(v=256)])
def test_every_call_refuses_bad_buffers(kw):
    L, c, m = sla.lib(), ref(config()), buffers(**kw)
    assert L.sla_cache_append(16, 16, c, m, 1, 16, None, None, None) == IA
    assert L.sla_cache_route(16, c, m, 1, 16, None, 4, 16, None) == IA
    assert L.sla_cache_attend(16, c, m, 1, 16, None, None, 0, 0, 32, 256, 1 << 30, None) == IA
    assert L.sla_cache_evict(c, m, 16, 64, 0, 0, 16, 16, 16, 32, 256, 1 << 30, None) == IA


def test_append_refusals():
    L, c = sla.lib(), ref(config())

    def call(k=16, v=16, T=1, lens=16, n_new=None, lens_out=None):
        return L.sla_cache_append(k, v, c, buffers(), T, lens, n_new, lens_out, None)

    assert call(k=None) == call(v=None) == call(lens=None) == IA
    assert call(k=24) == call(v=24) == call(lens=18) == call(n_new=18) == call(lens_out=18) == IA
    assert call(T=0) == call(T=-1) == IA
    assert call(T=8 * 64 + 1) == IA          # more than any sequence can hold
    assert call(lens_out=16) == IA           # would overwrite what other blocks still read


def test_route_refusals():
    L, c = sla.lib(), ref(config())

    def call(q=16, T=1, lens=16, n_new=None, top_n=4, sel=16, m=None):
        return L.sla_cache_route(q, c, m or buffers(), T, lens, n_new, top_n, sel, None)

    assert call(q=None) == call(lens=None) == call(sel=None) == call(q=24) == call(sel=18) == IA
    assert call(T=0) == call(top_n=0) == call(m=buffers(k_mean=None)) == IA
    assert call(T=65) == call(top_n=65) == UN


def test_attend_refusals():
    cfg = config()
    L, c = sla.lib(), ref(cfg)

    def call(q=16, T=1, lens=16, n_new=None, sel=None, top_n=0, window=0, out=32, ws=256, nbytes=None, m=None):
        if nbytes is None:
            nbytes = sla.sla_cache_attend_workspace_bytes(cfg, max(T, 1), max(top_n, 0), max(window, 0), True)
        return L.sla_cache_attend(q, c, m or buffers(), T, lens, n_new, sel, top_n, window, out, ws, nbytes, None)

    assert call(q=None) == call(lens=None) == call(out=None) == call(q=24) == call(out=24) == IA
    assert call(out=16) == IA                                  # out is q
    assert call(T=0) == call(window=-1) == call(top_n=-1) == IA
    assert call(sel=16, top_n=0) == call(sel=None, top_n=4) == call(sel=18, top_n=4) == IA
    assert call(T=65, nbytes=1 << 30) == call(sel=16, top_n=65, nbytes=1 << 30) == UN
    assert call(ws=None) == call(ws=128) == WS
    need = sla.sla_cache_attend_workspace_bytes(cfg, 1, 0, 0, True)
    assert call(nbytes=need - 1) == WS
    wide = config(H=64, H_kv=2)                                # 32 heads a group: 33 rows each are too many
    assert sla.sla_cache_attend_workspace_bytes(wide, 32) > 0
    assert sla.sla_cache_attend_workspace_bytes(wide, 33) == 0


def test_evict_refusals():
    cfg = config()
    L, c = sla.lib(), ref(cfg)

    def call(lens=16, budget=64, sink=0, recent=0, dst=16, w=16, kept=16, lens_out=32, ws=256, nbytes=1 << 20, m=None):
        return L.sla_cache_evict(c, m or buffers(), lens, budget, sink, recent, dst, w, kept, lens_out, ws, nbytes, None)

    for kw in (dict(lens=None), dict(dst=None), dict(w=None), dict(kept=None), dict(lens_out=None), dict(lens=18),
               dict(dst=18), dict(w=20), dict(kept=18), dict(lens_out=18), dict(lens_out=16), dict(budget=0),
               dict(budget=8 * 64 + 1), dict(sink=-1), dict(recent=-1), dict(sink=40, recent=25),
               dict(sink=2**31 - 1, recent=2**31 - 1), dict(m=buffers(weight=None))):
        assert call(**kw) == IA, kw
    need = sla.sla_cache_evict_workspace_bytes(cfg, 64)
    assert call(ws=None) == call(ws=128) == call(nbytes=need - 1) == WS
    assert sla.sla_cache_evict_workspace_bytes(cfg, 0) == sla.sla_cache_evict_workspace_bytes(cfg, 513) == 0


@pytest.mark.parametrize("n_new", [None, 2048])
def test_append_refuses_to_write_lengths_that_it_reads(n_new):
    """lens_out may share no element (here two of four bytes) with lens or n_new."""
    L, c = sla.lib(), ref(config())
    for at in [1020, 1024, 1028] + ([2044, 2048, 2052] if n_new else []):
        assert L.sla_cache_append(16, 16, c, buffers(), 1, 1024, n_new, at, None) == IA, at


def test_evict_refuses_to_write_lengths_that_it_reads():
    L, c = sla.lib(), ref(config())
    for at in (1020, 1024, 1028):
        assert L.sla_cache_evict(c, buffers(), 1024, 64, 0, 0, 16, 16, 16, at, 256, 1 << 20, None) == IA, at


def test_a_buffer_longer_than_a_sequence_needs_its_lengths():
    """Without n_new all T rows would be taken, which no sequence can hold."""
    L, c = sla.lib(), ref(config())
    for T in (8 * 64 + 1, 2**31 - 1):
        assert L.sla_cache_append(16, 16, c, buffers(), T, 16, None, None, None) == IA
    # with it only what the device sees can be wrong; refused here for its lens_out
    assert L.sla_cache_append(16, 16, c, buffers(), 8 * 64 + 1, 1024, 2048, 1024, None) == IA


def test_the_caches_tensors_cannot_be_replaced():
    """Their addresses are taken once: another tensor in their place would never be read, and
    the one that the kernels read would be gone."""
    cache = object.__new__(sla.SlaCache)
    for name in sla.SlaCache.__slots__:
        with pytest.raises(AttributeError, match="replaced"):
            setattr(cache, name, 1)
        with pytest.raises(AttributeError, match="replaced"):
            delattr(cache, name)


def test_python_cache_refuses_tensors_that_the_kernels_could_not_take():
    with pytest.raises(ValueError, match="CUDA"):
        sla.SlaCache.empty(config(), device="cpu")


# ---------------------------------------------------------------------------
# the oracle's formats
# ---------------------------------------------------------------------------

def test_code_tables_are_torchs():
    u = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    np.testing.assert_array_equal(co.code_table(co.E4M3), u.view(torch.float8_e4m3fn).double().numpy())
    np.testing.assert_array_equal(co.code_table(co.INT8), u.view(torch.int8).double().numpy())


@pytest.mark.parametrize("kind", [co.E4M3, co.INT8])
def test_rounding_is_the_nearest_code_with_ties_to_even(kind):
    t = np.unique(co.code_table(kind)[np.isfinite(co.code_table(kind))])
    t = t[np.abs(t) <= (448 if kind == co.E4M3 else 127)]
    mid = (t[1:] + t[:-1]) / 2
    x = np.concatenate([t, mid, mid * (1 + 1e-9), mid * (1 - 1e-9), np.random.default_rng(1).uniform(t[0], t[-1], 4000)])
    got = co.round_codes(x, kind)
    assert np.isin(got, t).all()
    best = np.abs(x[:, None] - t[None]).min(1)
    np.testing.assert_array_equal(np.abs(x - got), best)
    if kind == co.E4M3:
        want = torch.from_numpy(x).float()
        exact = want.double().numpy() == x                     # what float32 holds exactly
        np.testing.assert_array_equal(want.to(torch.float8_e4m3fn).double().numpy()[exact], got[exact])
    else:
        np.testing.assert_array_equal(got, np.round(x))


@pytest.mark.parametrize("kind,top", [(co.E4M3, 448.0), (co.INT8, 127.0)])
def test_scales_are_the_least_power_of_two(kind, top):
    for a in [0.0, 2.0 ** -133, 2.0 ** -100, 1e-20, 0.1, 1.0, top, top * 1.0000001, top * 2, 3.0, 1e30, 2.0 ** 120]:
        s = co.scale_of(a, kind)
        assert np.log2(s) == np.round(np.log2(s)) and a <= top * s and s >= 2.0 ** -110
        assert s == 2.0 ** -110 or a > top * s / 2
