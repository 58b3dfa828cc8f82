"""The paged 8-bit cache on the GPU against its float64 oracle: append, route, attend and
evict, alone and as one serving loop.

Codes, scales, page means, moved weights and lists have to be equal (power-of-two scales
make every step but the code's rounding exact). Outputs of the attention: bf16 rounding
(2^-8 of the value), the probabilities rounded to fp16 before the product with V (2^-11 of
each term, so 2^-11 of sum p |v|) and fp32 sums, exponentials and scores (2^-16 of sum p |v|
covers scores up to 2^5 at 2^-21 and the rest).
Attention weights: fp32 throughout; a score of magnitude up to 2^5 with error 2^-21 relative
gives 2^-16 of a probability, and sums of R rows stay below that.
"""
import numpy as np
import pytest
import torch

import block_sparse_linear_sm_b200 as sla
from block_sparse_linear_sm_b200 import workloads as wl
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

E4M3, INT8 = co.E4M3, co.INT8
DT = {E4M3: torch.float8_e4m3fn, INT8: torch.int8}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def codes_of(t):
    return co.code_table(INT8 if t.dtype == torch.int8 else E4M3)[t.view(torch.uint8).cpu().numpy()]


class Pair:
    """A device cache and its oracle with the same shuffled pages and, once filled, the same
    contents. Pages of no sequence and unwritten slots start as garbage (NaN codes, NaN
    scales) on the device."""

    def __init__(self, B=2, H=4, H_kv=2, d=128, max_blocks=6, kind=E4M3, scale=0.0, spare=4, seed=0, garbage=True):
        self.rng = np.random.default_rng(seed)
        n_pages = B * max_blocks + spare
        self.cfg = wl.CacheConfig(B=B, H=H, H_kv=H_kv, d=d, n_pages=n_pages, max_blocks=max_blocks, kind=kind,
                                  scale=scale)
        order = self.rng.permutation(n_pages)
        self.table, self.spare = order[:B * max_blocks].reshape(B, max_blocks), order[B * max_blocks:]
        self.o = co.Cache(self.cfg, self.table)
        self.c = sla.SlaCache.empty(self.cfg)
        self.c.block_table.copy_(i32(self.table))
        self.lens = np.zeros(B, int)
        if garbage:
            for t in (self.c.k, self.c.v):
                t.view(torch.uint8).fill_(0x7f)
            for t in (self.c.k_scale, self.c.v_scale, self.c.k_mean, self.c.weight):
                t.fill_(float("nan"))

    def kv(self, T, mean=0.0, std=1.0):
        c = self.cfg
        k = std * self.rng.standard_normal((c.B, c.H_kv, T, c.d)) + mean
        v = std * self.rng.standard_normal((c.B, c.H_kv, T, c.d))
        return bf16(k), bf16(v)

    def queries(self, T, std=1.0):
        return bf16(std * self.rng.standard_normal((self.cfg.B, self.cfg.H, T, self.cfg.d)))

    def append(self, k, v, n_new=None, stream=None):
        n = np.full(self.cfg.B, k.shape[2]) if n_new is None else np.asarray(n_new)
        out = torch.full((self.cfg.B,), -5, dtype=torch.int32, device="cuda")
        sla.sla_cache_append(k, v, self.cfg, self.c, i32(self.lens), None if n_new is None else i32(n), out)
        self.lens = self.o.append(f64(k), f64(v), self.lens, n)
        assert out.tolist() == self.lens.tolist()

    def fill(self, lens, **kw):
        """Appends up to `lens` tokens in two calls."""
        lens = np.asarray(lens)
        first = lens // 3
        for n in (first, lens - first):
            if n.max() > 0:
                self.append(*self.kv(int(n.max()), **kw), n_new=n)
        self.status()

    def status(self, want=(0, 0)):
        assert sla.sla_check_device_status(self.c.status) == want

    def used(self):
        """[(sequence, block, full)] of the blocks in use."""
        return [(b, j, (j + 1) * 64 <= n) for b, n in enumerate(self.lens) for j in range(-(-n // 64))]

    def check(self, table=None):
        """Pages in use equal the oracle's, bit for bit."""
        table = self.table if table is None else table
        k, v = codes_of(self.c.k), codes_of(self.c.v)
        ks, vs, mean = f64(self.c.k_scale), f64(self.c.v_scale), f64(self.c.k_mean)
        for b, j, full in self.used():
            p = table[b, j]
            np.testing.assert_array_equal(ks[p], self.o.ks[p])
            np.testing.assert_array_equal(vs[p], self.o.vs[p])
            np.testing.assert_array_equal(k[p], self.o.k[p])
            np.testing.assert_array_equal(v[p], self.o.v[p])
            if full:
                np.testing.assert_array_equal(mean[p], self.o.mean[p])
        w = f64(self.c.weight)
        for b, n in enumerate(self.lens):
            np.testing.assert_array_equal(w[b, :, :n], self.o.weight[b, :, :n])

    def attend(self, q, n_new=None, sel=None, window=0, weight=True, out=None, ws=None):
        c, T = self.cfg, q.shape[2]
        cache = self.c if weight else sla.SlaCache(**{n: getattr(self.c, n) for n in
                                                      ("k", "v", "k_scale", "v_scale", "k_mean", "block_table",
                                                       "status")}, weight=None)
        out = torch.full_like(q, float("nan")) if out is None else out
        top_n = 0 if sel is None else sel.shape[2]
        if ws is None:
            ws = torch.full((sla.sla_cache_attend_workspace_bytes(c, T, top_n, window, weight),), 0xff,
                            dtype=torch.uint8, device="cuda")
        sla.sla_cache_attend(q, c, cache, i32(self.lens), None if n_new is None else i32(n_new),
                             None if sel is None else i32(sel), window, out, ws)
        return out

    def check_attend(self, q, n_new=None, sel=None, window=0):
        """out and the added weights against the oracle; returns out."""
        n = np.full(self.cfg.B, q.shape[2]) if n_new is None else np.asarray(n_new)
        before = f64(self.c.weight)
        out = self.attend(q, n_new, sel, window)
        self.status()
        want, mag, got = self.o.attend(f64(q), self.lens, n, sel, window, add_weight=True)
        err = np.abs(f64(out) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag), np.nanmax(err)
        after = f64(self.c.weight)
        for b, m in enumerate(self.lens):
            add = after[b, :, :m] - before[b, :, :m]
            tol = 2.0 ** -16 * got[b, :, :m] + 2.0 ** -23 * np.abs(after[b, :, :m])
            assert np.all(np.abs(add - got[b, :, :m]) <= tol)
            # slots behind the last token are left as they were
            np.testing.assert_array_equal(after[b, :, m:], before[b, :, m:])
            self.o.weight[b, :, :m] = after[b, :, :m]
        plain = self.attend(q, n_new, sel, window, weight=False)
        assert torch.equal(plain.view(torch.int16), out.view(torch.int16))
        return out


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("d,H_kv", [(64, 1), (64, 3), (128, 2)])
def test_append_holds_what_the_definition_says(kind, d, H_kv):
    p = Pair(B=6, H=H_kv, H_kv=H_kv, d=d, max_blocks=5, kind=kind, seed=d + H_kv)
    for n_new in ([0, 1, 63, 64, 65, 200], [1, 1, 1, 1, 1, 1], [64, 62, 1, 0, 130, 2], [3, 0, 5, 7, 64, 11]):
        # magnitudes that grow make open pages take a larger scale
        k, v = p.kv(max(n_new), std=float(2.0 ** p.rng.integers(-3, 4)))
        p.append(k, v, n_new)
        p.check()
    p.status()


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_one_at_a_time(kind):
    p = Pair(B=2, H=1, H_kv=1, d=64, max_blocks=3, kind=kind, seed=3)
    p.lens = np.array([0, 0])
    for i in range(130):
        k, v = p.kv(1, std=0.02 * (1 + i % 17))
        p.append(k, v, [1, int(i % 2 == 0)])
    p.check()
    p.status()


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_extreme_magnitudes(kind):
    p = Pair(B=4, H=1, H_kv=1, d=64, max_blocks=2, kind=kind, seed=4)
    k, v = p.kv(70)
    k[0] *= 0                          # zeros: the least scale
    k[1] = (k[1].float() * 2.0 ** -120).bfloat16()   # below what the least scale resolves
    k[2] = (k[2].float() * 2.0 ** 110).bfloat16()
    v[3, :, 5:] = 0
    p.append(k, v)
    p.check()
    k, v = p.kv(3)
    k[0] *= 0                          # zero rows behind rows leave the page's scale alone
    p.append(k, v)
    p.check()
    p.status()


def test_append_leaves_other_pages_and_rows_alone():
    p = Pair(B=2, H=2, H_kv=2, max_blocks=4)
    p.fill([100, 30])
    before = [t.clone() for t in (p.c.k.view(torch.uint8), p.c.v.view(torch.uint8), p.c.k_scale, p.c.weight)]
    k, v = p.kv(4)
    k[:, :, 1:] = float("nan")         # rows that n_new leaves out are not read
    p.append(k, v, [1, 0])
    p.status()
    page = p.table[0, 1]
    touched = np.zeros(p.cfg.n_pages, bool)
    touched[page] = True
    keep = torch.from_numpy(~touched).cuda()
    assert torch.equal(p.c.k.view(torch.uint8)[keep], before[0][keep])
    assert torch.equal(p.c.v.view(torch.uint8)[keep], before[1][keep])
    assert torch.equal(p.c.k_scale.view(torch.int32)[keep], before[2].view(torch.int32)[keep])
    assert torch.equal(p.c.weight.view(torch.int32)[1], before[3].view(torch.int32)[1])
    p.check()


def test_append_reports_values_it_cannot_hold():
    p = Pair(B=2, H=1, H_kv=1, d=64, max_blocks=2, kind=INT8)
    k, v = p.kv(10)
    k[0, 0, 2, 5], k[0, 0, 3, 1], v[1, 0, 4, 7] = float("nan"), float("-inf"), float("inf")
    p.append(k, v)
    p.check()
    p.status((sla.SLA_ERR_DEVICE_CHECK, 113))
    p.status()


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_of_few_rows_from_a_buffer_longer_than_a_sequence(kind):
    """T is the buffers' row pitch: n_new says what is taken."""
    p = Pair(B=3, H=2, H_kv=2, d=64, max_blocks=2, kind=kind, seed=5)
    for n_new in ([10, 0, 128], [100, 64, 0], [18, 1, 0]):
        k, v = p.kv(300)
        for b, n in enumerate(n_new):
            k[b, :, n:] = v[b, :, n:] = float("nan")
        p.append(k, v, n_new)
        p.check()
        p.status()
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    sla.sla_cache_append(k, v, p.cfg, p.c, i32(p.lens), i32([1, 300, 129]), out)
    assert out.tolist() == p.lens.tolist()
    p.status((sla.SLA_ERR_DEVICE_CHECK, 111))
    p.check()


def test_append_refuses_on_the_device_what_does_not_fit():
    p = Pair(B=5, H=1, H_kv=1, d=64, max_blocks=2)
    p.fill([10, 10, 10, 10, 10])
    before = p.c.k.view(torch.uint8).clone()
    k, v = p.kv(4)
    out = torch.zeros(5, dtype=torch.int32, device="cuda")
    for lens, n_new in (([126, -1, 129, 10, 10], [3, 1, 1, -1, 5]),):
        sla.sla_cache_append(k, v, p.cfg, p.c, i32(lens), i32(n_new), out)
        assert out.tolist() == lens
        p.status((sla.SLA_ERR_DEVICE_CHECK, 111))
    assert torch.equal(p.c.k.view(torch.uint8), before)
    # a page number out of range: that block alone is left out
    p.c.block_table[0, 0], p.c.block_table[1, 0] = p.cfg.n_pages, -1
    sla.sla_cache_append(k, v, p.cfg, p.c, i32([10] * 5), i32([1, 1, 0, 0, 0]), out)
    p.status((sla.SLA_ERR_DEVICE_CHECK, 110))
    assert torch.equal(p.c.k.view(torch.uint8), before)


# ---------------------------------------------------------------------------
# attend
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv,T", [(1, 1, 1), (4, 2, 1), (5, 1, 3), (16, 1, 1), (6, 2, 7), (16, 1, 2), (32, 2, 3),
                                      (16, 1, 8), (20, 1, 9)])
def test_attend_all_tokens(kind, d, H, H_kv, T):
    p = Pair(B=4, H=H, H_kv=H_kv, d=d, max_blocks=6, kind=kind, seed=H + T)
    p.fill([max(T, 1), 64, 129, 384])
    p.check_attend(p.queries(T))
    p.check_attend(p.queries(T, std=3.0), n_new=[T, 0, (T + 1) // 2, 1])


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("lens", [[0, 1], [2, 63], [65, 0], [127, 128], [4096, 4095], [1000, 37]])
def test_attend_lengths(kind, lens):
    p = Pair(B=2, H=8, H_kv=2, d=128, max_blocks=64, kind=kind, seed=sum(lens))
    p.fill(lens)
    out = p.check_attend(p.queries(1))
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any()


def test_attend_more_rows_than_tokens():
    """Rows whose slot would be negative see nothing."""
    p = Pair(B=2, H=2, H_kv=1, d=64)
    p.fill([2, 5])
    out = p.check_attend(p.queries(6))
    assert not out[0, :, :4].any() and not out[1, :, :1].any()


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 100000])
@pytest.mark.parametrize("T,H", [(1, 4), (5, 4), (7, 20)])
def test_attend_window(window, T, H):
    p = Pair(B=3, H=H, H_kv=2, d=64, max_blocks=8, kind=INT8, seed=window)
    p.fill([500, 70, 6])
    p.check_attend(p.queries(T), window=window)


def lists(p, rows, top_n):
    sel = np.full((p.cfg.B, p.cfg.H_kv, top_n), -1)
    for (b, h), r in rows.items():
        sel[b, h, :len(r)] = r
    return sel


@pytest.mark.parametrize("window", [0, 1, 70, 300])
@pytest.mark.parametrize("T,H", [(1, 8), (4, 8), (5, 32)])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_attend_selected_blocks(window, T, H, kind):
    p = Pair(B=3, H=H, H_kv=2, d=128, max_blocks=12, kind=kind, seed=window + T)
    p.fill([700, 130, 20])
    # ragged lists, an empty one, blocks that the window holds too, the open block itself
    sel = lists(p, {(0, 0): [0, 3, 9], (0, 1): [1, 2, 4, 6, 10], (1, 0): [0], (1, 1): [0, 1, 2]}, 5)
    sel[1, 1] = [-1, 0, -1, 1, 2]
    out = p.check_attend(p.queries(T), sel=sel, window=window)
    if window == 0:
        assert not out[2].any()   # no block, no window


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("T,H", [(1, 4), (3, 32), (5, 32)])
def test_attend_lists_longer_than_the_sequence(window, T, H):
    """64 entries, anywhere between the -1, of which the valid ones are few."""
    p = Pair(B=4, H=H, H_kv=2, d=64, max_blocks=40, seed=window + H)
    p.fill([40 * 64, 200, 64, 5])
    rng = np.random.default_rng(T)
    sel = np.full((4, 2, 64), -1, np.int32)
    for b, n in enumerate((40, 4, 1, 1)):
        for hk in range(2):
            keep = np.sort(rng.permutation(n)[:max(1, n - 3 * hk)])
            sel[b, hk, np.sort(rng.permutation(64)[:len(keep)])] = keep
    sel[1, 0] = -1
    sel[1, 0, [0, 31, 32, 63]] = [0, 1, 2, 3]
    q = p.queries(T)
    out = p.check_attend(q, sel=sel, window=window)
    for bad in ([0, 31, 33, 63], [0, 1, 2, 3]):   # an entry too large behind the last valid one
        sel[1, 0] = -1
        sel[1, 0, bad] = [0, 1, 2, 3]
        sel[1, 0, 40 if bad[2] == 2 else 62] = 3
        sel[1, 0, 63] = 4
        got = p.attend(q, sel=sel, window=window, weight=False)
        p.status((sla.SLA_ERR_DEVICE_CHECK, 112))
        assert torch.equal(got, out)


@pytest.mark.parametrize("T,H", [(1, 4), (6, 16)])
def test_attend_longest_list(T, H):
    p = Pair(B=1, H=H, H_kv=1, d=64, max_blocks=70, seed=9)
    p.fill([70 * 64])
    p.check_attend(p.queries(T), sel=lists(p, {(0, 0): list(range(3, 67))}, 64), window=65)


@pytest.mark.parametrize("H", [4, 160])
def test_attend_reports_bad_lists_pages_and_lengths(H):
    p = Pair(B=2, H=H, H_kv=2, d=64, max_blocks=6, seed=10)
    p.fill([300, 200])
    q = p.queries(1)
    good = lists(p, {(0, 0): [1, 3], (0, 1): [2], (1, 0): [0, 2]}, 3)
    want = p.attend(q, sel=good, weight=False)
    p.status()
    for bad in ([1, 3, 3], [1, 3, 2], [1, 3, 5], [1, 3, 2**31 - 1]):   # twice, descending, beyond the last block
        sel = good.copy()
        sel[0, 0] = bad
        out = p.attend(q, sel=sel, weight=False)
        p.status((sla.SLA_ERR_DEVICE_CHECK, 112))
        assert torch.equal(out, want), bad
    # a page out of range is as if its tokens were not there
    for page in (-1, p.cfg.n_pages, 2**31 - 1):
        p.c.block_table[0, 3] = page
        out = p.attend(q, sel=good, weight=False)
        p.status((sla.SLA_ERR_DEVICE_CHECK, 110))
        sel = good.copy()
        sel[0, 0] = [1, -1, -1]
        assert torch.equal(out, p.attend(q, sel=sel, weight=False))
        p.status()
    p.c.block_table.copy_(i32(p.table))
    # a length out of range: that sequence sees nothing
    for n in (-1, 6 * 64 + 1):
        p.lens = np.array([300, n])
        out = p.attend(q, weight=False)
        p.status((sla.SLA_ERR_DEVICE_CHECK, 111))
        assert not out[1].any() and out[0].any()
    p.lens = np.array([300, 200])
    out = p.attend(q, n_new=[1, 2], weight=False)
    p.status((sla.SLA_ERR_DEVICE_CHECK, 111))
    assert not out[1].any() and out[0].any()


@pytest.mark.parametrize("H", [4, 80])
def test_attend_large_scores_and_one_hot_rows(H):
    """Scores of some hundred: one token takes all; no overflow, no NaN."""
    p = Pair(B=1, H=H, H_kv=1, d=128, max_blocks=6, kind=INT8, seed=11)
    p.fill([333], std=8.0)
    q = p.queries(1, std=100.0)
    out = p.attend(q)
    want, mag, _ = p.o.attend(f64(q), p.lens, [1], None, 0)
    # scores near 2^14 have errors up to 2^14 * 2^-22 = 2^-8 absolute where tokens compete
    # a weight is held as fp16 of 2^8 times it at least, the row's largest taken as 1: its step is
    # 2^-24 / 2^8 at least, so each of the 333 is off by up to half of that, 2^-33, and one below
    # it counts as 0. Where the one token that takes all has value 0 in a column, that is all
    # there is
    floor = 333 * 2.0 ** -33 * np.abs(p.o.rows(0, 0, 333)[1]).max()
    assert np.all(np.abs(f64(out) - want) <= (2.0 ** -8 + 2.0 ** -7) * mag + floor)


@pytest.mark.parametrize("lo,hi", [(-100, -90), (-60, 60), (90, 110)])
@pytest.mark.parametrize("H", [4, 66])
def test_attend_scales_far_apart(lo, hi, H):
    """Pages whose value scales differ by many binades, and tiny or huge values."""
    p = Pair(B=1, H=H, H_kv=1, d=64, max_blocks=4, kind=E4M3, seed=12)
    for j, e in enumerate((lo, hi, lo)):
        k, v = p.kv(64)
        p.append(k, (v.float() * 2.0 ** e).bfloat16())
    p.check()
    q = p.queries(1)
    out = p.attend(q, weight=False)
    want, mag, _ = p.o.attend(f64(q), p.lens, [1], None, 0)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)


@pytest.mark.parametrize("std", [2.0 ** -40, 2.0 ** 40])
@pytest.mark.parametrize("H", [4, 140])
def test_attend_query_magnitudes(std, H):
    """Tiny queries give equal weights; huge ones one token's value. Rows differ in magnitude."""
    p = Pair(B=1, H=H, H_kv=2, d=64, max_blocks=3, seed=13)
    p.fill([150])
    q = p.queries(1)
    q[0, 1] = (q[0, 1].float() * std).bfloat16()
    q[0, 2] = 0
    out = p.attend(q, weight=False)
    want, mag, _ = p.o.attend(f64(q), p.lens, [1], None, 0)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag
    assert np.all(np.abs(f64(out) - want) <= tol)


@pytest.mark.parametrize("H", [8, 68])
def test_attend_nan_query_stays_in_its_row(H):
    p = Pair(B=2, H=H, H_kv=2, d=64, seed=14)
    p.fill([100, 100])
    q = p.queries(2)
    want = p.attend(q, weight=False)
    q2 = q.clone()
    q2[0, 3, 1, 5], q2[1, 6, 0, 2] = float("nan"), float("inf")
    out = p.attend(q2, weight=False)
    rest = torch.ones(2, H, 2, dtype=torch.bool)
    rest[0, 3, 1] = rest[1, 6, 0] = False
    assert torch.equal(out[rest], want[rest])
    assert torch.isnan(out[0, 3, 1]).all() and torch.isnan(out[1, 6, 0]).all()


def test_attend_nan_query_adds_no_weight():
    p = Pair(B=2, H=4, H_kv=2, d=64, seed=19)
    p.fill([100, 70])
    p.c.weight.zero_()
    q = p.queries(2)
    p.attend(q)
    want = p.c.weight.clone()
    q[0, 1, 0, 3] = float("nan")
    p.c.weight.zero_()
    p.attend(q)
    assert torch.isfinite(p.c.weight).all()
    assert torch.equal(p.c.weight[0, 1], want[0, 1]) and torch.equal(p.c.weight[1], want[1])
    # three of the four rows of the KV head are left
    assert abs(p.c.weight[0, 0].sum().item() - 3) < 3e-5 and abs(want[0, 0].sum().item() - 4) < 4e-5


@pytest.mark.parametrize("H,T", [(4, 1), (5, 3), (68, 1), (30, 3)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attend_infinite_query_beside_keys_of_one_sign(H, T, sign):
    """All its scores are +inf or all -inf; one key, some, many parts, none."""
    p = Pair(B=4, H=H, H_kv=1, d=64, max_blocks=32, seed=24)
    k, v = p.kv(2000)
    k[..., 7] = k[..., 7].abs() + 0.5
    p.append(k, v, [T, 100, 2000, 0])
    p.c.weight.zero_()
    n_new = [T, T, T, 0]
    q = p.queries(T)
    want = p.attend(q, n_new)
    weight = p.c.weight.clone()
    bad = q.clone()
    for b in range(4):
        bad[b, 1, T - 1, 7] = sign * float("inf")
    p.c.weight.zero_()
    out = p.attend(bad, n_new)
    p.status()
    assert torch.isnan(out[:3, 1, T - 1]).all() and not out[3].any()
    rest = torch.ones(4, H, T, dtype=torch.bool)
    rest[:, 1, T - 1] = False
    assert torch.equal(out[rest], want[rest])
    # the row's share is missing, and nothing else
    lost = (weight - p.c.weight).sum(dim=(1, 2)).tolist()
    assert all(abs(x - y) <= 2.0 ** -16 * H * T for x, y in zip(lost, (1, 1, 1, 0)))


def test_attend_shared_pages():
    """Sequences may share pages that are only read."""
    p = Pair(B=3, H=4, H_kv=2, d=64, max_blocks=4, seed=15)
    p.fill([256, 256, 256])
    p.table[1, :2] = p.table[0, :2]
    p.table[2] = p.table[0]
    p.o.table = p.table
    p.c.block_table.copy_(i32(p.table))
    p.check_attend(p.queries(1))


@pytest.mark.parametrize("H,T", [(3, 1), (30, 7)])
def test_attend_many_sequences(H, T):
    p = Pair(B=300, H=H, H_kv=3, d=64, max_blocks=2, kind=INT8, seed=16)
    p.fill(np.arange(300) % 128)
    p.check_attend(p.queries(T))
    # most lists empty: many neighbouring segments without a page
    sel = np.full((300, 3, 2), -1)
    sel[::37, 1, 0] = 0
    sel[p.lens == 0] = -1
    p.check_attend(p.queries(T), sel=sel)


def test_attend_many_rows():
    """T * H / H_kv = 1024 rows a KV head, the largest step."""
    p = Pair(B=1, H=16, H_kv=1, d=128, max_blocks=4, seed=17)
    p.fill([190])
    p.check_attend(p.queries(64))


LONGEST = 4096 * 64


@pytest.mark.parametrize("T,H", [(1, 2), (1, 16), (2, 70)])
def test_attend_longest_sequence(T, H):
    """4096 blocks, the last one open, beside a sequence of one token; the long one's pages repeat."""
    p = Pair(B=2, H=H, H_kv=2 if H == 2 else 1, d=64, max_blocks=4096, kind=INT8, seed=20, garbage=False)
    p.c.k.view(torch.uint8).zero_(), p.c.v.view(torch.uint8).zero_()
    few = np.arange(7)
    p.table[0], p.table[1, 0] = few[np.arange(4096) % 7], 7
    p.o.table = p.table
    p.c.block_table.copy_(i32(p.table))
    rng = np.random.default_rng(1)
    for name in ("k", "v"):
        codes = rng.integers(-60, 61, getattr(p.o, name)[:8].shape)
        getattr(p.o, name)[:8] = codes
        getattr(p.c, name)[:8] = torch.from_numpy(codes.astype(np.int8)).cuda()
    for name, dev in (("ks", p.c.k_scale), ("vs", p.c.v_scale)):
        getattr(p.o, name)[:] = 2.0 ** -5
        dev.fill_(2.0 ** -5)
    p.c.weight.zero_()
    p.lens = np.array([LONGEST - 5, 1])
    p.check_attend(p.queries(T), n_new=[T, min(T, 1)])


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("H,d", [(4, 64), (66, 64), (16, 128), (66, 128)])
def test_attend_many_values_of_the_largest_magnitude(kind, H, d):
    """320 tokens of +-2^120 at equal weights: their unnormalised sum is beyond fp32."""
    p = Pair(B=2, H=H, H_kv=1, d=d, max_blocks=6, kind=kind, seed=25)
    k, v = p.kv(320)
    v[:] = 2.0 ** 120
    v[..., ::2] = -(2.0 ** 120)
    p.append(k, v, [320, 300])
    q = p.queries(1) * 0
    out = p.attend(q, weight=False)
    p.status()
    want, mag, _ = p.o.attend(f64(q), p.lens, [1, 1], None, 0)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)


@pytest.mark.parametrize("H", [2, 16, 70])
def test_attend_longest_sequence_of_the_largest_values(H):
    """262144 tokens of 2^120; the first block of every 28 has scores 2^6.5 below the others, so
    that a maximum taken from it stays behind for the whole run of a CTA."""
    p = Pair(B=1, H=H, H_kv=1, d=64, max_blocks=4096, kind=INT8, seed=26, garbage=False)
    p.table[0] = np.where(np.arange(4096) % 28 == 0, 0, 1)
    p.o.table = p.table
    p.c.block_table.copy_(i32(p.table))
    for name in ("k", "v"):
        codes = np.zeros(getattr(p.o, name)[:2].shape)
        codes[:] = 64
        if name == "k":
            codes[0] = 0
        getattr(p.o, name)[:2] = codes
        getattr(p.c, name)[:2] = torch.from_numpy(codes.astype(np.int8)).cuda()
    p.o.ks[:], p.o.vs[:] = 2.0 ** -6, 2.0 ** 114
    p.c.k_scale.fill_(2.0 ** -6), p.c.v_scale.fill_(2.0 ** 114)
    p.lens = np.array([LONGEST])
    # q . k * scale = 64 * 4.5 / 8 * 1 / 8 = 4.5: e^4.5 is 2^6.5, and the others' k is 0
    q = bf16(np.full((1, H, 1, 64), 4.5 / 8))
    out = p.attend(q, weight=False)
    p.status()
    assert np.all(np.abs(f64(out) - 2.0 ** 120) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * 2.0 ** 120)


@pytest.mark.parametrize("H", [4, 66])
def test_attend_values_of_the_least_scale(H):
    """Pages at the least scale: the output is as good as that of other pages."""
    p = Pair(B=1, H=H, H_kv=1, d=64, max_blocks=6, kind=INT8, seed=27)
    k, v = p.kv(330)
    p.append(k, (v.float() * 2.0 ** -106).bfloat16())
    assert (p.o.vs[p.table] == 2.0 ** -110).all()
    q = p.queries(1)
    out = p.attend(q, weight=False)
    want, mag, _ = p.o.attend(f64(q), p.lens, [1], None, 0)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)


@pytest.mark.parametrize("T", [2, 9])
def test_attend_writes_the_same_bits_again(T):
    p = Pair(B=4, H=16, H_kv=2, d=128, max_blocks=40, seed=18)
    p.fill([2500, 1, 700, 1300])
    q = p.queries(T)
    p.c.weight.zero_()
    a = p.attend(q)
    w = p.c.weight.clone()
    for _ in range(3):
        p.c.weight.zero_()
        b = p.attend(q)
        assert torch.equal(a, b) and torch.equal(w, p.c.weight)


# ---------------------------------------------------------------------------
# route
# ---------------------------------------------------------------------------

def run_route(p, q, top_n, n_new=None):
    sel = torch.full((p.cfg.B, p.cfg.H_kv, top_n), -7, dtype=torch.int32, device="cuda")
    sla.sla_cache_route(q, p.cfg, p.c, i32(p.lens), None if n_new is None else i32(n_new), sel)
    return sel.cpu().numpy()


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("d,H,H_kv,T,top_n", [(64, 1, 1, 1, 1), (128, 8, 2, 1, 4), (128, 20, 1, 3, 16), (64, 6, 2, 64, 64),
                                              (128, 96, 2, 2, 7)])
def test_route_picks_the_definitions_blocks(kind, d, H, H_kv, T, top_n):
    p = Pair(B=5, H=H, H_kv=H_kv, d=d, max_blocks=40, kind=kind, seed=H)
    p.fill([T, 64, 64 + T, 1000, 40 * 64])
    for n_new in ([T] * 5, [1, T, 0, (T + 1) // 2, T]):
        q = p.queries(T, std=2.0)
        want, gap = p.o.route(f64(q), p.lens, n_new, top_n)
        assert gap > 1e-9
        np.testing.assert_array_equal(run_route(p, q, top_n, n_new), want)
    p.status()


def test_route_long_context():
    p = Pair(B=1, H=4, H_kv=1, d=64, max_blocks=4096, seed=21, garbage=False)
    p.c.k_mean.normal_()
    p.o.mean = f64(p.c.k_mean)
    p.lens = np.array([4096 * 64])
    q = p.queries(1)
    want, gap = p.o.route(f64(q), p.lens, [1], 64)
    assert gap > 1e-9
    np.testing.assert_array_equal(run_route(p, q, 64), want)


def test_route_equal_blocks_by_lower_index():
    p = Pair(B=1, H=2, H_kv=1, d=64, max_blocks=20, seed=22, garbage=False)
    p.c.k_mean.zero_()
    p.c.k_mean[p.table[0, 11]] = 1.0
    p.lens = np.array([20 * 64])
    q = bf16(np.full((1, 2, 1, 64), 0.5))
    assert run_route(p, q, 4).tolist() == [[[0, 1, 2, 11]]]
    # far behind the best: probabilities of exactly 0 are equal too
    p.c.k_mean[p.table[0, 11]] = 1e6
    assert run_route(p, q, 3).tolist() == [[[0, 1, 11]]]


def test_route_scale_is_not_rounded():
    """1 / sqrt(128) rounded to fp32 is off by 1.7e-8 of it, which would change the order of two
    blocks whose sums are closer than that. The heads' scores are (x, 0, 9) and (0, 1, 0): where
    x = 8.45 or so, blocks 0 and 1 have equal sums. x is put halfway between the places where the
    two scales find them equal."""
    p = Pair(B=1, H=2, H_kv=1, d=128, max_blocks=4, seed=28, garbage=False)
    exact, rounded = 1 / np.sqrt(128.0), float(np.float32(1) / np.sqrt(np.float32(128)))
    q = np.zeros((1, 2, 1, 128))
    q[0, 0, 0, 0], q[0, 1, 0, 1], q[0, 0, 0, 2] = 8.0, 8.0, 2.0 ** -10
    mean = np.zeros((4, 128), np.float32)
    mean[2, 0], mean[1, 1] = 9 / (8 * exact), 1 / (8 * exact)

    def ahead(at, x, scale):
        """Sum of block 0 less that of block 1 with mean[0, at] = x."""
        m = mean[:3].astype(np.float64)
        m[0, at] = x
        e = [np.exp(m @ q[0, h, 0] * scale) for h in range(2)]
        return sum((t[0] - t[1]) / t.sum() for t in e)

    def equal(at, scale, lo, hi):
        assert ahead(at, lo, scale) < 0 < ahead(at, hi, scale)
        for _ in range(100):
            mid = (lo + hi) / 2
            lo, hi = (mid, hi) if ahead(at, mid, scale) < 0 else (lo, mid)
        return lo

    mean[0, 0] = equal(0, exact, 0.0, 20.0)
    mean[0, 2] = (equal(2, exact, -1.0, 1.0) + equal(2, rounded, -1.0, 1.0)) / 2
    x = float(mean[0, 2])
    assert (ahead(2, x, exact) < 0) != (ahead(2, x, rounded) < 0)
    p.lens = np.array([3 * 64 + 1])
    p.c.k_mean[torch.from_numpy(p.table[0]).cuda(), 0] = torch.from_numpy(mean).cuda()
    p.o.mean = f64(p.c.k_mean)
    want, gap = p.o.route(q, p.lens, [1], 2)
    assert gap > 1e-9
    np.testing.assert_array_equal(run_route(p, bf16(q), 2), want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_route_picks_nothing_for_a_query_that_is_not_finite(value):
    """Beside means of one sign an infinity makes every score the same infinity."""
    p = Pair(B=2, H=6, H_kv=2, d=64, max_blocks=10, seed=29)
    k, v = p.kv(600)
    k[..., 7] = k[..., 7].abs() + 0.5
    p.append(k, v, [600, 70])
    q = p.queries(2)
    want, gap = p.o.route(f64(q), p.lens, [2, 2], 3)
    assert gap > 1e-9
    q[:, 4, 1, 7] = value           # a head of the second group
    want[:, 1] = -1
    np.testing.assert_array_equal(run_route(p, q, 3), want)
    p.status()


def test_route_leaves_out_bad_pages():
    p = Pair(B=1, H=2, H_kv=1, d=64, max_blocks=6, seed=23)
    p.fill([6 * 64])
    p.c.block_table[0, 2], p.c.block_table[0, 4] = -1, p.cfg.n_pages
    assert run_route(p, p.queries(1), 5).tolist() == [[[0, 1, 3, -1, -1]]]
    p.status((sla.SLA_ERR_DEVICE_CHECK, 110))
    p.lens = np.array([6 * 64 + 1])
    assert run_route(p, p.queries(1), 2).tolist() == [[[-1, -1]]]
    p.status((sla.SLA_ERR_DEVICE_CHECK, 111))


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------

def run_evict(p, budget, n_sink, n_recent, in_place):
    """Evicts on both sides; returns (table, kept)."""
    B, nd = p.cfg.B, -(-budget // 64)
    dst = p.table[:, :nd].copy() if in_place else p.spare[:B * nd].reshape(B, nd)
    weight_out = p.c.weight if in_place else torch.full_like(p.c.weight, 7.5)
    kept = torch.full((B, p.cfg.H_kv, budget), -9, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.full((sla.sla_cache_evict_workspace_bytes(p.cfg, budget),), 0xff, dtype=torch.uint8, device="cuda")
    old = {n: getattr(p.c, n).view(torch.uint8).clone() for n in ("k", "v")}
    want_w = f64(weight_out)
    sla.sla_cache_evict(p.cfg, p.c, i32(p.lens), budget, n_sink, n_recent, i32(dst), weight_out, kept, lens_out, ws)
    p.status()
    want = p.o.evict(p.lens, budget, n_sink, n_recent, dst, want_w)
    np.testing.assert_array_equal(kept.cpu().numpy(), want)
    np.testing.assert_array_equal(f64(weight_out), want_w)
    p.o.weight = want_w
    if not in_place:
        untouched = torch.ones(p.cfg.n_pages, dtype=torch.bool, device="cuda")
        untouched[torch.from_numpy(dst).cuda()] = False
        for n in old:
            assert torch.equal(getattr(p.c, n).view(torch.uint8)[untouched], old[n][untouched])
        p.c.weight.copy_(weight_out)
    p.lens = np.minimum(p.lens, budget)
    assert lens_out.tolist() == p.lens.tolist()
    return dst, want


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("d,budget,n_sink,n_recent", [(64, 1, 0, 0), (128, 64, 4, 16), (128, 100, 0, 100),
                                                      (64, 321, 2, 63), (128, 500, 0, 0), (64, 640, 640, 0)])
def test_evict_keeps_the_heaviest(kind, d, budget, n_sink, n_recent, in_place):
    p = Pair(B=4, H=2, H_kv=2, d=d, max_blocks=12, kind=kind, spare=48, seed=budget)
    p.fill([0, 90, 700, 768], std=2.0)
    p.o.weight[:] = np.random.default_rng(budget).integers(0, 40, p.o.weight.shape) / 8.0    # many equal
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, _ = run_evict(p, budget, n_sink, n_recent, in_place)
    p.check(dst)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,max_blocks", [(5, 36), (75, 36), (5, 32), (5, 33)])
def test_evict_few_and_many_heads(B, max_blocks, in_place):
    """One CTA or a cluster selects, whatever the lengths are; many equal weights."""
    p = Pair(B=B, H=1, H_kv=1, d=64, max_blocks=max_blocks, kind=INT8, spare=6 * B, seed=B + max_blocks)
    p.fill([max_blocks * 64, 0, 1, 333, 334] + [(97 * i) % 1500 for i in range(B - 5)], std=2.0)
    p.o.weight[:] = np.random.default_rng(B).integers(0, 30, p.o.weight.shape) / 8.0
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, _ = run_evict(p, 333, 3, 70, in_place)
    p.check(dst)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_odd_weights(in_place):
    p = Pair(B=1, H=1, H_kv=1, d=64, max_blocks=4, spare=8, seed=31)
    p.fill([250])
    w = np.zeros(256, np.float32)
    w[10], w[20], w[30], w[40], w[50] = np.nan, np.inf, -np.inf, -1.0, -0.0
    w[60:70] = 1e-40
    w[70:75] = 3e38
    p.o.weight[0, 0] = w
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    run_evict(p, 248, 0, 3, in_place)


def test_evict_drops_non_finite_last():
    """NaN counts as -inf: the lower slot of the two stays longer."""
    p = Pair(B=1, H=1, H_kv=1, d=64, max_blocks=2, spare=4, seed=32)
    p.fill([100])
    p.o.weight[0, 0, :100] = 1.0
    p.o.weight[0, 0, [5, 9]] = [-np.inf, np.nan]
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    _, kept = run_evict(p, 99, 0, 0, False)
    assert 5 in kept and 9 not in kept


def test_evict_long():
    p = Pair(B=1, H=2, H_kv=2, d=64, max_blocks=300, spare=0, seed=33)
    p.fill([300 * 64 - 7])
    p.o.weight[:] = np.random.default_rng(5).random(p.o.weight.shape).astype(np.float32) ** 8
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, _ = run_evict(p, 5000, 4, 128, True)
    p.check(dst)


def test_evict_longest():
    """262144 slots: every weight of a CTA's run in shared memory."""
    p = Pair(B=1, H=1, H_kv=1, d=64, max_blocks=4096, spare=8, seed=36, garbage=False)
    p.lens = np.array([4096 * 64])
    p.o.ks[:], p.o.vs[:] = 1.0, 1.0
    p.c.k_scale.fill_(1.0), p.c.v_scale.fill_(1.0)
    codes = np.random.default_rng(6).integers(0, 120, p.o.k.shape)      # e4m3 bytes of positive numbers
    p.o.k, p.o.v = co.code_table(E4M3)[codes], co.code_table(E4M3)[codes[::-1]]
    p.c.k.view(torch.uint8).copy_(torch.from_numpy(codes.astype(np.uint8)))
    p.c.v.view(torch.uint8).copy_(torch.from_numpy(codes[::-1].astype(np.uint8)))
    p.o.weight[:] = np.random.default_rng(7).integers(0, 5000, p.o.weight.shape) / 64.0
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, _ = run_evict(p, 500, 4, 100, False)
    p.check(dst)


def fill_with_outliers(p, big):
    """130 tokens whose first two blocks each hold one element `big` in every KV head, of keys and
    of values: their other rows are rounded to 0. Returns the outliers' slots."""
    k, v = p.kv(130)
    for at, d in ((5, 3), (70, 40)):
        k[:, :, at, d] = big
        v[:, :, at, d + 1] = -big
    p.append(k, v)
    p.status((0, 0) if np.isfinite(big) else (sla.SLA_ERR_DEVICE_CHECK, 113))
    assert not p.o.k[p.table[0, :2]][:, :, :5].any() and not p.o.v[p.table[0, :2]][:, :, :5].any()
    return [5, 70]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("big", [2.0 ** 30, float("inf")])
@pytest.mark.parametrize("budget", [20, 64, 70])
def test_evict_of_an_outlier_leaves_the_zeros_beside_it(kind, big, budget, in_place):
    """New blocks of zero codes only, from pages of a large scale: the least scale, codes of 0."""
    p = Pair(B=1, H=2, H_kv=2, d=64, max_blocks=3, kind=kind, seed=41)
    gone = fill_with_outliers(p, big)
    w = np.random.default_rng(budget).integers(1, 40, p.o.weight.shape).astype(np.float64)
    w[:, :, gone] = w[:, :, 128:] = 0
    p.o.weight[:] = w
    p.c.weight.copy_(torch.from_numpy(w))
    dst, kept = run_evict(p, budget, 0, 0, in_place)
    assert not np.isin(kept, gone).any()
    p.check(dst)


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_evict_joins_zeros_of_a_large_scale_and_tiny_numbers(kind):
    """Zero codes of a page of scale 2^112 or so move into a block whose scale is the least one."""
    p = Pair(B=1, H=1, H_kv=1, d=64, max_blocks=2, kind=kind, seed=42)
    k, v = p.kv(128)
    for x in (k, v):
        x[:, :, 64:] = (x[:, :, 64:].float() * 2.0 ** -111).bfloat16()
        x[:, :, 9, 1] = 2.0 ** 120
    p.append(k, v)
    p.status()
    p.o.weight[:] = 1.0
    p.o.weight[0, 0, 9] = 0
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, kept = run_evict(p, 127, 0, 0, False)
    assert 9 not in kept and p.o.k[dst[0, 0], 0, 63].any() and not p.o.k[dst[0, 0], 0, :63].any()
    p.check(dst)


@pytest.mark.parametrize("same_weights", [True, False])
@pytest.mark.parametrize("own", [[0, 2], [1, 3], [3], [0, 1, 2]])
def test_evict_some_blocks_in_place(own, same_weights):
    """Blocks packed where they are beside blocks that move to new pages; weights in place or not."""
    p = Pair(B=2, H=3, H_kv=3, d=64, max_blocks=12, kind=INT8, spare=8, seed=43)
    p.fill([768, 500])
    p.o.weight[:] = np.random.default_rng(len(own)).integers(0, 40, p.o.weight.shape) / 8.0
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst = p.spare.reshape(2, 4).copy()
    dst[:, own] = p.table[:, own]
    weight_out = p.c.weight if same_weights else torch.full_like(p.c.weight, 7.5)
    kept = torch.zeros(2, 3, 250, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.full((sla.sla_cache_evict_workspace_bytes(p.cfg, 250),), 0xff, dtype=torch.uint8, device="cuda")
    want_w = f64(weight_out)
    sla.sla_cache_evict(p.cfg, p.c, i32(p.lens), 250, 2, 30, i32(dst), weight_out, kept, lens_out, ws)
    p.status()
    np.testing.assert_array_equal(kept.cpu().numpy(), p.o.evict(p.lens, 250, 2, 30, dst, want_w))
    np.testing.assert_array_equal(f64(weight_out), want_w)
    p.lens, p.o.weight = np.array([250, 250]), want_w
    p.c.weight.copy_(weight_out)
    p.check(dst)


def test_evict_in_a_captured_graph():
    """Replayed twice on the same cache, other weights each time, in place and packed again."""
    p = Pair(B=2, H=2, H_kv=2, d=64, max_blocks=10, kind=INT8, spare=0, seed=37)
    p.fill([600, 333])
    budget, nd = 200, 4
    lens, lens_out = i32(p.lens), torch.zeros(2, dtype=torch.int32, device="cuda")
    dst = i32(p.table[:, :nd])
    kept = torch.zeros(2, 2, budget, dtype=torch.int32, device="cuda")
    ws = torch.empty(sla.sla_cache_evict_workspace_bytes(p.cfg, budget), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        sla.sla_cache_evict(p.cfg, p.c, lens, budget, 4, 50, dst, p.c.weight, kept, lens_out, ws)
    for step in range(2):
        w = np.random.default_rng(step).random(p.o.weight.shape).astype(np.float32)
        p.o.weight[:] = w
        p.c.weight.copy_(torch.from_numpy(w))
        lens.copy_(i32(p.lens))
        g.replay()
        out = p.o.weight.copy()
        want = p.o.evict(p.lens, budget, 4, 50, p.table[:, :nd], out)
        np.testing.assert_array_equal(kept.cpu().numpy(), want)
        p.o.weight = out
        p.lens = np.minimum(p.lens, budget)
        p.check()
        p.append(*p.kv(130))
        p.check()
    p.status()


def test_evict_reports_bad_pages_and_lengths():
    p = Pair(B=3, H=1, H_kv=1, d=64, max_blocks=4, spare=6, seed=34)
    p.fill([200, 200, 200])
    p.c.weight.fill_(1.0)
    before = p.c.k.view(torch.uint8).clone()
    dst = np.array([[-1, p.cfg.n_pages]] * 3)
    kept = torch.zeros(3, 1, 100, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(sla.sla_cache_evict_workspace_bytes(p.cfg, 100), dtype=torch.uint8, device="cuda")
    w = torch.zeros_like(p.c.weight)
    sla.sla_cache_evict(p.cfg, p.c, i32(p.lens), 100, 0, 0, i32(dst), w, kept, lens_out, ws)
    p.status((sla.SLA_ERR_DEVICE_CHECK, 110))
    assert torch.equal(p.c.k.view(torch.uint8), before)
    # a source page out of range: its tokens become 0, the others move
    good = p.spare.reshape(3, 2)
    p.c.block_table[1, 0] = p.cfg.n_pages
    sla.sla_cache_evict(p.cfg, p.c, i32(p.lens), 100, 0, 100, i32(good), w, kept, lens_out, ws)
    p.status()                                   # the kept tokens are in blocks 1 to 3
    sla.sla_cache_evict(p.cfg, p.c, i32(p.lens), 100, 100, 0, i32(good), w, kept, lens_out, ws)
    p.status((sla.SLA_ERR_DEVICE_CHECK, 110))
    moved = codes_of(p.c.k)[good]
    assert not moved[1, 0].any() and moved[1, 1, :, :36].any() and moved[0, 0].any() and moved[2, 0].any()
    p.c.block_table.copy_(i32(p.table))
    before = p.c.k.view(torch.uint8).clone()
    sla.sla_cache_evict(p.cfg, p.c, i32([-1, 257, 0]), 100, 0, 0, i32(dst), w, kept, lens_out, ws)
    p.status((sla.SLA_ERR_DEVICE_CHECK, 111))
    assert lens_out.tolist() == [0, 0, 0] and (kept == -1).all()
    assert torch.equal(p.c.k.view(torch.uint8), before)


def test_calls_without_means_or_weights():
    """k_mean and weight may be left out where a call does not need them."""
    p = Pair(B=2, H=2, H_kv=2, d=64, max_blocks=4, spare=8, seed=44)
    names = ("k", "v", "k_scale", "v_scale", "block_table", "status")
    bare = sla.SlaCache(**{n: getattr(p.c, n) for n in names}, k_mean=None, weight=None)
    weighted = sla.SlaCache(**{n: getattr(p.c, n) for n in names}, k_mean=None, weight=p.c.weight)
    k, v = p.kv(200)
    sla.sla_cache_append(k, v, p.cfg, bare, i32([0, 0]), i32([200, 100]))
    p.lens = p.o.append(f64(k), f64(v), p.lens, [200, 100])
    assert torch.isnan(p.c.k_mean).all() and torch.isnan(p.c.weight).all()
    p.o.weight[:] = np.random.default_rng(1).random(p.o.weight.shape).astype(np.float32)
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, want_w = p.spare[:6].reshape(2, 3), p.o.weight.copy()
    kept = torch.zeros(2, 2, 130, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(sla.sla_cache_evict_workspace_bytes(p.cfg, 130), dtype=torch.uint8, device="cuda")
    sla.sla_cache_evict(p.cfg, weighted, i32(p.lens), 130, 1, 1, i32(dst), p.c.weight, kept, lens_out, ws)
    p.status()
    np.testing.assert_array_equal(kept.cpu().numpy(), p.o.evict(p.lens, 130, 1, 1, dst, want_w))
    p.lens, p.o.weight = np.array([130, 100]), want_w
    assert torch.isnan(p.c.k_mean).all()
    p.o.mean[:] = np.nan
    p.check(dst)
    with pytest.raises(sla.SlaError):
        sla.sla_cache_route(p.queries(1), p.cfg, bare, i32(p.lens), None, torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(sla.SlaError):
        sla.sla_cache_evict(p.cfg, bare, i32(p.lens), 130, 1, 1, i32(dst), p.c.weight, kept, lens_out, ws)


@pytest.mark.parametrize("H", [4, 132])
def test_a_scale_of_the_callers(H):
    p = Pair(B=2, H=H, H_kv=2, d=128, max_blocks=8, kind=INT8, scale=0.03, seed=45)
    p.fill([500, 77])
    q = p.queries(1, std=2.0)
    p.check_attend(q)
    want, gap = p.o.route(f64(q), p.lens, [1, 1], 3)
    assert gap > 1e-9
    np.testing.assert_array_equal(run_route(p, q, 3), want)


@pytest.mark.parametrize("H,H_kv,d", [(2, 1, 128), (8, 2, 64), (66, 1, 64)])
def test_the_most_sequences(H, H_kv, d):
    """1024 sequences: their lengths alone are 9 KB of every attention CTA's shared memory."""
    p = Pair(B=1024, H=H, H_kv=H_kv, d=d, max_blocks=2, kind=INT8, seed=46)
    p.fill((np.arange(1024) * 7) % 129)
    q = p.queries(1)
    p.check_attend(q)
    want, gap = p.o.route(f64(q), p.lens, np.ones(1024, int), 2)
    assert gap > 1e-9
    np.testing.assert_array_equal(run_route(p, q, 2), want)
    p.o.weight[:] = np.random.default_rng(0).integers(0, 9, p.o.weight.shape)
    p.c.weight.copy_(torch.from_numpy(p.o.weight))
    dst, _ = run_evict(p, 70, 3, 20, True)
    p.check(dst)


@pytest.mark.parametrize("H_kv", [1, 1024])
def test_the_most_heads(H_kv):
    p = Pair(B=2, H=1024, H_kv=H_kv, d=64, max_blocks=2, seed=47)
    p.fill([100, 65])
    q = p.queries(1)
    p.check_attend(q)
    np.testing.assert_array_equal(run_route(p, q, 3), p.o.route(f64(q), p.lens, [1, 1], 3)[0])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind,H,H_kv,d", [(E4M3, 8, 2, 128), (INT8, 4, 4, 64)])
def test_serving_loop(kind, H, H_kv, d):
    """Prompts, steps of (append, route, attend), an eviction, more steps."""
    p = Pair(B=3, H=H, H_kv=H_kv, d=d, max_blocks=10, kind=kind, seed=40)
    p.append(*p.kv(400, mean=0.1), n_new=[400, 77, 1])
    for step in range(8):
        T = 1 + step % 3
        n_new = [T, 1, T - 1]
        p.append(*p.kv(T), n_new=n_new)
        q = p.queries(T)
        sel = run_route(p, q, 3, n_new)
        want, gap = p.o.route(f64(q), p.lens, n_new, 3)
        assert gap > 1e-9
        np.testing.assert_array_equal(sel, want)
        p.check_attend(q, n_new, sel=sel, window=70)
        p.check_attend(q, n_new)
        if step == 4:
            dst, _ = run_evict(p, 150, 4, 32, True)
        p.check()
    p.status()


def test_step_is_the_layers_last_query_block():
    """A step of 64 tokens whose keys and values the codes hold exactly equals the last query
    block of the whole-sequence top-n layer: the same blocks, the same output."""
    N, H, H_kv, d, top_n, window = 1024, 8, 2, 128, 4, 200
    cfg = wl.small_config(N=N, N_valid=N, H=H, H_kv=H_kv, d=d, mode=wl.MODE_TOPN_WINDOW, top_n=top_n, window=window,
                          causal=1, has_proj=0)
    rng = np.random.default_rng(50)
    q = bf16(rng.standard_normal((1, H, N, d)))
    k = bf16(rng.integers(-100, 101, (1, H_kv, N, d)) / 64.0)
    v = bf16(rng.integers(-100, 101, (1, H_kv, N, d)) / 64.0)
    out = torch.empty_like(q)
    ws = torch.empty(sla.sla_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    sla.sla_forward(q, k, v, None, None, cfg, out, None, ws)
    mask = torch.empty(1, H_kv, N // 64, N // 64, dtype=torch.int8, device="cuda")
    crit = torch.empty(1, H_kv, N // 64, top_n, dtype=torch.int32, device="cuda")
    sla.sla_route(q, k, cfg, mask, crit, None, ws)
    assert sla.sla_check_device_status(ws) == (0, 0)

    p = Pair(B=1, H=H, H_kv=H_kv, d=d, max_blocks=N // 64, kind=INT8)
    p.append(k, v)
    step = q[:, :, -64:].contiguous()
    sel = run_route(p, step, top_n)
    np.testing.assert_array_equal(sel[0], crit[0, :, -1].cpu().numpy())
    got = p.check_attend(step, sel=sel, window=window)
    # both round once to bf16 at the end; the layer rounds its probabilities to bf16 (2^-8 of
    # each), this one to fp16
    err = (got.float() - out[:, :, -64:].float()).abs()
    mag = torch.from_numpy(p.o.attend(f64(step), p.lens, [64], sel, window)[1]).cuda()
    assert bool((err <= 2 * 2.0 ** -8 * got.float().abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all())


def test_streams_and_captured_steps():
    """A captured step replays on whatever its buffers hold; two graphs share a workspace."""
    p = Pair(B=2, H=8, H_kv=2, d=64, max_blocks=6, seed=60)
    p.fill([130, 40])
    c, T = p.cfg, 1
    k, v, q = *p.kv(T), p.queries(T)
    lens, new_lens = i32(p.lens), i32(p.lens)
    sel = torch.zeros(2, 2, 2, dtype=torch.int32, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(sla.sla_cache_attend_workspace_bytes(c, T, 2, 64, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=side):
        sla.sla_cache_append(k, v, c, p.c, lens, None, new_lens)
        sla.sla_cache_route(q, c, p.c, new_lens, None, sel)
        sla.sla_cache_attend(q, c, p.c, new_lens, None, sel, 64, out, ws)
        lens.copy_(new_lens)
    with torch.cuda.graph(g2, stream=side):
        sla.sla_cache_attend(q, c, p.c, new_lens, None, sel, 64, out2, ws)
    for step in range(70):
        nk, nv = p.kv(T)
        nq = p.queries(T)
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        weight = p.c.weight.clone()
        g1.replay()
        p.lens = p.o.append(f64(nk), f64(nv), p.lens, [1, 1])
        if step % 10 == 0:
            w1 = p.c.weight.clone()
            g2.replay()
            assert torch.equal(out, out2)
            p.c.weight.copy_(w1)
            want_sel, gap = p.o.route(f64(nq), p.lens, [1, 1], 2)
            assert gap > 1e-9
            np.testing.assert_array_equal(sel.cpu().numpy(), want_sel)
            want, mag, _ = p.o.attend(f64(nq), p.lens, [1, 1], want_sel, 64)
            assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)
    assert lens.tolist() == p.lens.tolist()
    p.status()


@pytest.mark.parametrize("B", [3, 24])
def test_lengths_in_two_buffers_in_turn(B):
    """Steps one behind the other without a copy or a wait between them, the lengths in one of two
    buffers and then the other: every kernel of a step sees its own lengths."""
    p = Pair(B=B, H=16, H_kv=2, d=64, max_blocks=20, kind=INT8, seed=62)

    def kv(T):
        """Every token has the same largest element, so that codes are never rounded again."""
        k, v = (x.clamp(-3.5, 3.5) for x in p.kv(T))
        k[..., 3], v[..., 5] = 4.0, -4.0
        return k, v

    steps = 60
    p.append(*kv(1000), n_new=[(331 * b + 1) % 1001 for b in range(B)])
    news, qs = [kv(1) for _ in range(steps)], [p.queries(1) for _ in range(steps)]
    outs = [torch.empty_like(q) for q in qs]
    lens = [i32(p.lens), torch.zeros(B, dtype=torch.int32, device="cuda")]
    ws = torch.empty(sla.sla_cache_attend_workspace_bytes(p.cfg, 1, 0, 0, True), dtype=torch.uint8, device="cuda")
    p.c.weight.zero_()
    torch.cuda.synchronize()
    for i, ((k, v), q, out) in enumerate(zip(news, qs, outs)):
        old, new = lens[i % 2], lens[1 - i % 2]
        sla.sla_cache_append(k, v, p.cfg, p.c, old, None, new)
        sla.sla_cache_attend(q, p.cfg, p.c, new, None, None, 0, out, ws)
    p.status()
    # every row gave out a weight of 1 a step (rows of sums of 2^-16 relative error)
    got = p.c.weight.sum(dim=2)
    assert bool(((got - 8 * steps).abs() <= 8 * steps * 2.0 ** -16).all())
    first = p.lens.copy()
    for i, (q, out) in enumerate(zip(qs, outs)):
        p.lens = first + i + 1
        assert torch.equal(p.attend(q, weight=False), out), i


def test_captured_beside_copies_and_a_second_stream():
    """Copies before, between and behind the calls, and the routing on a stream of its own that
    the attention waits for: each call sees what was written before it, replay after replay."""
    p = Pair(B=2, H=8, H_kv=2, d=64, max_blocks=8, seed=61)
    p.fill([200, 77])
    c, T = p.cfg, 2
    k, v, q = *p.kv(T), p.queries(T)
    k_in, v_in, q_in = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
    lens, new_lens, lens_b = i32(p.lens), i32(p.lens), i32(p.lens)
    sel, sel_b = (torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda") for _ in range(2))
    out, out_b = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(sla.sla_cache_attend_workspace_bytes(c, T, 3, 64, True), dtype=torch.uint8, device="cuda")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        k_in.copy_(k)
        v_in.copy_(v)
        sla.sla_cache_append(k_in, v_in, c, p.c, lens, None, new_lens)
        lens_b.copy_(new_lens)
        other.wait_stream(side)
        with torch.cuda.stream(other):
            q_in.copy_(q)
            sla.sla_cache_route(q_in, c, p.c, lens_b, None, sel)
            sel_b.copy_(sel)
        lens.copy_(new_lens)
        side.wait_stream(other)
        sla.sla_cache_attend(q_in, c, p.c, lens_b, None, sel_b, 64, out, ws)
        out_b.copy_(out)
    for step in range(20):
        nk, nv = p.kv(T)
        nq = p.queries(T)
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        g.replay()
        p.lens = p.o.append(f64(nk), f64(nv), p.lens, [T, T])
        want_sel, gap = p.o.route(f64(nq), p.lens, [T, T], 3)
        assert gap > 1e-9
        np.testing.assert_array_equal(sel_b.cpu().numpy(), want_sel)
        want, mag, _ = p.o.attend(f64(nq), p.lens, [T, T], want_sel, 64)
        assert np.all(np.abs(f64(out_b) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)
    assert lens.tolist() == p.lens.tolist()
    p.status()


def test_calls_on_a_given_stream():
    """stream= instead of the current one: ordered with work on that stream only."""
    p = Pair(B=2, H=4, H_kv=2, d=64, max_blocks=4, seed=61)
    p.fill([130, 40])
    s = torch.cuda.Stream()
    k, v = p.kv(3)
    q = p.queries(3)
    lens, out, sel = i32(p.lens), torch.empty_like(q), torch.zeros(2, 2, 2, dtype=torch.int32, device="cuda")
    ws = torch.empty(sla.sla_cache_attend_workspace_bytes(p.cfg, 3, 2, 9, True), dtype=torch.uint8, device="cuda")
    new = torch.empty_like(lens)
    torch.cuda.synchronize()
    sla.sla_cache_append(k, v, p.cfg, p.c, lens, None, new, stream=s)
    sla.sla_cache_route(q, p.cfg, p.c, new, None, sel, stream=s.cuda_stream)
    sla.sla_cache_attend(q, p.cfg, p.c, new, None, sel, 9, out, ws, stream=s)
    assert sla.sla_check_device_status(p.c.status, stream=s) == (0, 0)
    p.lens = p.o.append(f64(k), f64(v), p.lens, [3, 3])
    want_sel, gap = p.o.route(f64(q), p.lens, [3, 3], 2)
    assert gap > 1e-9
    np.testing.assert_array_equal(sel.cpu().numpy(), want_sel)
    want, mag, _ = p.o.attend(f64(q), p.lens, [3, 3], want_sel, 9)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * mag)


def test_calls_on_two_streams_at_once():
    ps = [Pair(B=2, H=16, H_kv=2, d=128, max_blocks=20, seed=70 + i) for i in range(2)]
    qs, outs, want = [], [], []
    for p in ps:
        p.fill([1200, 900])
        p.c.weight.zero_()
        qs.append(p.queries(1))
        want.append(p.attend(qs[-1], weight=False))
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for p, q, s in zip(ps, qs, streams):
            with torch.cuda.stream(s):
                outs.append(p.attend(q))
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_python_refusals():
    p = Pair(B=2, H=4, H_kv=2, d=64)
    p.fill([10, 20])
    q, lens = p.queries(1), i32(p.lens)
    out = torch.empty_like(q)
    ws = torch.empty(sla.sla_cache_attend_workspace_bytes(p.cfg, 1, 0, 0, True), dtype=torch.uint8, device="cuda")

    def attend(q=q, cfg=p.cfg, cache=p.c, lens=lens, n_new=None, sel=None, window=0, out=out, ws=ws):
        sla.sla_cache_attend(q, cfg, cache, lens, n_new, sel, window, out, ws)

    for kw in (dict(q=q.float()), dict(q=q[:, :, 0]), dict(q=q.cpu()), dict(q=q[:1]), dict(lens=lens.long()),
               dict(lens=lens[:1]), dict(out=out.transpose(1, 2)), dict(n_new=lens.cpu()),
               dict(sel=torch.zeros(2, 2, dtype=torch.int32, device="cuda")), dict(ws=ws.cpu()),
               dict(cfg=wl.CacheConfig(**{**vars(p.cfg), "n_pages": 3})),
               dict(cfg=wl.CacheConfig(**{**vars(p.cfg), "kind": INT8}))):
        with pytest.raises(ValueError):
            attend(**kw)
    with pytest.raises(sla.SlaError):
        attend(ws=ws[:64])
    with pytest.raises(ValueError):
        sla.SlaCache(k=p.c.k, v=p.c.v.view(torch.int8), **{n: getattr(p.c, n) for n in (
            "k_scale", "v_scale", "k_mean", "weight", "block_table", "status")})
    attend()
    p.status()
