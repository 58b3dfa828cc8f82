"""The serving operators of the top-n mode, as they are measured: a paged cache of keys and
values in 8 bits with one power-of-two scale per page of 64 tokens and KV head, and the
four calls that work on it.

  append   writes new tokens' keys and values into the cache
  route    picks the top_n past blocks of a step's queries (one list per KV group)
  attend   softmax attention of a step's queries over the cache (all of it, the selected
           blocks and the window, or the window alone); adds each slot's attention weight
  evict    keeps the slots of largest accumulated weight and packs them

`run` computes them in plain torch operations, or with `own` through the library.
"""
import math
import random

import torch

own = False

BLOCK = 64
E4M3, INT8 = 0, 1


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    e, i = E4M3, INT8
    return [
        # one short conversation on a small layer: launch latency is what counts
        dict(name="attend_small", op="attend", B=1, H=8, H_kv=2, d=64, len=777, ragged=False, T=1, kind=e,
             top_n=0, window=0, weights=False),
        # a decode step of a few users with the NSA-shaped heads, weights kept for eviction
        dict(name="attend_weights", op="attend", B=8, H=64, H_kv=4, d=128, len=8191, ragged=True, T=1, kind=e,
             top_n=0, window=0, weights=True),
        # one user with a long context, nothing to batch: the length has to be split
        dict(name="attend_long", op="attend", B=1, H=64, H_kv=4, d=128, len=65536, ragged=False, T=1, kind=i,
             top_n=0, window=0, weights=False),
        # a full serving batch: the cache is far larger than L2
        dict(name="attend_batch", op="attend", B=64, H=32, H_kv=8, d=128, len=16384, ragged=True, T=1, kind=e,
             top_n=0, window=0, weights=False),
        # the top-n mode's own step: 16 selected blocks and the 512-token window of long contexts
        dict(name="attend_topn", op="attend", B=16, H=64, H_kv=4, d=128, len=65536, ragged=True, T=1, kind=e,
             top_n=16, window=512, weights=False),
        # eight tokens a step (drafted tokens checked at once): 128 query rows a KV head
        dict(name="attend_draft", op="attend", B=8, H=64, H_kv=4, d=128, len=16001, ragged=True, T=8, kind=e,
             top_n=0, window=0, weights=False),
        # the step's new token of every user
        dict(name="append_step", op="append", B=64, H=32, H_kv=8, d=128, len=1500, ragged=True, T=1, kind=e),
        # prompts of up to the 32760 tokens of the video layer written behind a few cached tokens
        dict(name="append_prompt", op="append", B=2, H=12, H_kv=12, d=128, len=100, ragged=True, T=32760, kind=i),
        # one user's step
        dict(name="route_small", op="route", B=1, H=64, H_kv=4, d=128, len=5000, ragged=False, T=1, kind=e, top_n=16),
        # a batch with long contexts
        dict(name="route_batch", op="route", B=16, H=64, H_kv=4, d=128, len=65536, ragged=True, T=2, kind=e, top_n=16),
        # one user's long context cut to a quarter
        dict(name="evict_long", op="evict", B=1, H=64, H_kv=4, d=128, len=65536, ragged=False, kind=e,
             budget=16384, sink=4, recent=512),
        # a batch cut to a budget that is no multiple of the page
        dict(name="evict_batch", op="evict", B=8, H=32, H_kv=8, d=128, len=16384, ragged=True, kind=i,
             budget=4001, sink=4, recent=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "route", "evict"])
    kv = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    c = dict(op=op, B=_log_int(rng, 1, 64), H=kv * group, H_kv=kv, d=rng.choice([64, 128, 128]),
             ragged=rng.random() < 0.7, kind=rng.choice([E4M3, INT8]))
    if op == "append":
        c["T"] = _log_int(rng, 1, 32760)
        c["len"] = rng.randrange(0, 2000)
        while c["B"] > 1 and c["B"] * kv * c["T"] > 2 * 12 * 32760:
            c["B"] = (c["B"] + 1) // 2
    else:
        c["len"] = _log_int(rng, 1 if op == "attend" else 64, 65536)
        # at most half the cached tokens of the largest listed case
        while c["B"] * kv * c["len"] > 32 * 8 * 16384 and c["B"] > 1:
            c["B"] = (c["B"] + 1) // 2
    if op == "attend":
        c["T"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        kind = rng.random()
        c["top_n"], c["window"] = (0, 0) if kind < 0.6 else (rng.randrange(1, 33), rng.randrange(0, 1025)) \
            if kind < 0.85 else (0, rng.randrange(1, 4097))
        c["weights"] = rng.random() < 0.4
        # no more products than the listed case with 128 query rows
        while c["B"] * kv * c["len"] * group * c["T"] > 8 * 4 * 16001 * 128:
            c["B"], c["len"] = ((c["B"] + 1) // 2, c["len"]) if c["B"] > 1 else (1, c["len"] // 2)
    if op == "route":
        c["T"] = rng.choice([1, 1, 2, 3, 8])
        c["len"] = max(c["len"], 1000)
        c["top_n"] = rng.randrange(1, 1 + min(64, c["len"] // BLOCK // 2))
    if op == "evict":
        c["sink"] = rng.randrange(0, 9)
        c["recent"] = rng.randrange(0, 1 + c["len"] // 4)
        c["budget"] = max(c["sink"] + c["recent"], 1) + rng.randrange(0, 1 + c["len"] // 2)
    return c


def lengths(case):
    """The cached tokens of each sequence: up to `len`; the first has all of it."""
    top, r = case["len"], random.Random(case["B"] * 1000003 + case["len"])
    if not case["ragged"]:
        return [top] * case["B"]
    return [top] + [r.randint(max(0, top // 4), top) for _ in range(case["B"] - 1)]


def new_tokens(case):
    """The valid new tokens of each sequence: T, or fewer in a ragged batch."""
    T, r = case.get("T", 0), random.Random(case["B"] * 7919 + case["len"] + 17)
    if not case["ragged"]:
        return [T] * case["B"]
    return [T] + [r.randint((T + 1) // 2, T) for _ in range(case["B"] - 1)]


def blocks_of(case):
    """Pages a sequence may hold: its row of the block table."""
    n = case["len"] + (case["T"] if case["op"] == "append" else 0)
    return max(1, -(-n // BLOCK))


def work(case):
    B, H, kv, d = case["B"], case["H"], case["H_kv"], case["d"]
    lens, new = lengths(case), new_tokens(case)
    if case["op"] == "append":
        n = sum(new)
        # a block that was open is read and written whole
        opened = sum(1 for x, y in zip(lens, new) if x % BLOCK and y)
        touched = sum(-(-(x + y) // BLOCK) - x // BLOCK for x, y in zip(lens, new) if y)
        return {"bytes": kv * (n * 2 * d * 3 + opened * BLOCK * d + touched * (8 + 4 * d) + n * 4),
                "flops": 4 * kv * n * d}
    if case["op"] == "route":
        past = [max(0, x - y) // BLOCK for x, y in zip(lens, new)]
        return {"bytes": kv * sum(past) * 4 * d + 2 * B * H * case["T"] * d + B * kv * case["top_n"] * 4,
                "flops": 2 * H * d * sum(past)}
    if case["op"] == "evict":
        m = [min(x, case["budget"]) for x in lens]
        return {"bytes": kv * (sum(lens) * 4 + sum(m) * (4 * d + 8) + 4 * B * case["budget"]), "flops": 4 * kv * sum(m) * d}
    seen = 0
    for x, y in zip(lens, new):
        if case["top_n"]:
            win = min(x, case["window"] + y - 1) if case["window"] else 0
            seen += min(x, min(case["top_n"], max(0, x - y) // BLOCK) * BLOCK + win)
        elif case["window"]:
            seen += min(x, case["window"] + y - 1)
        else:
            seen += x
    rows = H // kv * case["T"]
    return {"bytes": kv * seen * (2 * d + (8 if case["weights"] else 0)) + 4 * B * H * case["T"] * d,
            "flops": 4 * d * rows * kv * seen}


# ---------------------------------------------------------------------------
# the number formats, in plain operations
# ---------------------------------------------------------------------------

def pow2_scale(amax, kind):
    """The least power of two s with amax <= 448 s (e4m3) or 127 s (int8); 1 where amax is 0."""
    mant, e = torch.frexp(amax)
    if kind == E4M3:
        e = e - 9 + (mant > 0.875).int()
    else:
        e = e - 7 + (mant > 0.9921875).int()
    s = torch.ldexp(torch.ones_like(amax), e.clamp(-110, 120))
    return torch.where(amax == 0, torch.ones_like(s), s)


def to_codes(x, kind):
    """Nearest codes (ties to even) of x, already divided by its scale, as bytes."""
    if kind == E4M3:
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().to(torch.int8).view(torch.uint8)


def of_codes(c, kind):
    return c.view(torch.float8_e4m3fn if kind == E4M3 else torch.int8).float()


def as_values(c, kind):
    """The bytes as what they stand for, in units of their page's scale (a view)."""
    return c.view(torch.float8_e4m3fn if kind == E4M3 else torch.int8)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

class State:
    pass


def _fill_pages(codes, scale, mean, gen, kind, drift):
    """Random pages: each page and head has a mean of its own (drift) and unit noise."""
    n, kv, _, d = codes.shape
    step = max(1, (1 << 26) // (kv * BLOCK * d))
    for a in range(0, n, step):
        b = min(n, a + step)
        x = torch.randn(b - a, kv, BLOCK, d, device="cuda", generator=gen)
        if drift:
            x += drift * torch.randn(b - a, kv, 1, d, device="cuda", generator=gen)
        x = x.bfloat16().float()
        s = pow2_scale(x.abs().amax((2, 3)), kind)
        c = to_codes(x / s[:, :, None, None], kind)
        codes[a:b], scale[a:b] = c, s
        if mean is not None:
            mean[a:b] = of_codes(c, kind).mean(2) * s[:, :, None]


def prepare(case, seed):
    s = State()
    B, H, kv, d, kind = case["B"], case["H"], case["H_kv"], case["d"], case["kind"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev = torch.device("cuda")
    nb = blocks_of(case)
    extra = -(-case["budget"] // BLOCK) if case["op"] == "evict" else 0
    pages = B * (nb + extra)
    s.case, s.kind, s.nb = case, kind, nb
    s.lens = torch.tensor(lengths(case), dtype=torch.int32, device=dev)
    s.n_new = torch.tensor(new_tokens(case), dtype=torch.int32, device=dev)
    s.k = torch.empty(pages, kv, BLOCK, d, dtype=torch.uint8, device=dev)
    s.v = torch.empty_like(s.k)
    s.k_scale = torch.empty(pages, kv, device=dev)
    s.v_scale = torch.empty(pages, kv, device=dev)
    s.k_mean = torch.empty(pages, kv, d, device=dev)
    _fill_pages(s.k, s.k_scale, s.k_mean, gen, kind, 0.5)
    _fill_pages(s.v, s.v_scale, None, gen, kind, 0.0)
    order = torch.randperm(pages, device=dev, generator=gen).int()
    s.table = order[: B * nb].reshape(B, nb).contiguous()
    s.weight = torch.rand(B, kv, nb * BLOCK, device=dev, generator=gen).square() * 2
    s.status = torch.zeros(64, dtype=torch.int32, device=dev)
    if case["op"] in ("attend", "route"):
        s.q = torch.randn(B, H, case["T"], d, device=dev, generator=gen).bfloat16()
    if case["op"] == "append":
        s.new_k = torch.randn(B, kv, case["T"], d, device=dev, generator=gen).bfloat16()
        s.new_v = torch.randn(B, kv, case["T"], d, device=dev, generator=gen).bfloat16()
        s.lens_out = torch.empty_like(s.lens)
    if case["op"] == "route":
        s.sel = torch.empty(B, kv, case["top_n"], dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        s.out = torch.empty_like(s.q)
        s.sel = None
        if case["top_n"]:  # a router's lists: ascending past blocks, -1 behind the last
            past = (s.lens - s.n_new).clamp(min=0) // BLOCK
            key = torch.rand(B, kv, nb, device=dev, generator=gen)
            key = key.masked_fill(torch.arange(nb, device=dev) >= past[:, None, None], 2.0)
            top, at = key.sort(-1)
            n = min(nb, case["top_n"])
            at = torch.where(top[..., :n] < 2, at[..., :n], nb).sort(-1).values
            s.sel = torch.full((B, kv, case["top_n"]), -1, dtype=torch.int32, device=dev)
            s.sel[..., :n] = torch.where(at < nb, at, -1)
    if case["op"] == "evict":
        s.dst = order[B * nb:].reshape(B, extra).contiguous()
        s.weight_out = torch.zeros_like(s.weight)
        s.kept = torch.empty(B, kv, case["budget"], dtype=torch.int32, device=dev)
        s.lens_out = torch.empty_like(s.lens)
    if own:
        import block_sparse_linear_sm_b200 as sla
        from block_sparse_linear_sm_b200 import workloads as wl
        s.cfg = sla.make_cache_config(wl.CacheConfig(B=B, H=H, H_kv=kv, d=d, n_pages=pages, max_blocks=nb, kind=kind))
        weighted = case["op"] != "attend" or case["weights"]
        s.cache = sla.SlaCache(k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale, k_mean=s.k_mean,
                               weight=s.weight if weighted else None, block_table=s.table, status=s.status)
        if case["op"] == "attend":
            n = sla.sla_cache_attend_workspace_bytes(s.cfg, case["T"], case["top_n"], case["window"], case["weights"])
            s.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        if case["op"] == "evict":
            n = sla.sla_cache_evict_workspace_bytes(s.cfg, case["budget"])
            s.ws = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"append": run_append, "route": run_route, "attend": run_attend, "evict": run_evict}[s.case["op"]](s)


def run_append(s):
    if own:
        import block_sparse_linear_sm_b200 as sla
        sla.sla_cache_append(s.new_k, s.new_v, s.cfg, s.cache, s.lens, s.n_new, s.lens_out)
    else:
        B, kv, T, d = s.new_k.shape
        dev = s.lens.device
        start, stop = s.lens.long(), (s.lens + s.n_new).long()
        nt = min(s.nb, (T + BLOCK - 1) // BLOCK + 1)                       # blocks a sequence may touch
        blk = (start // BLOCK)[:, None] + torch.arange(nt, device=dev)      # [B, nt]
        touched = (blk * BLOCK < stop[:, None]) & (blk < s.nb) & (s.n_new > 0)[:, None]
        page = s.table.long().gather(1, blk.clamp(max=s.nb - 1))
        slot = blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)    # [B, nt, 64]
        old = (slot < start[:, None, None])[:, :, None, :, None]
        new = ((slot >= start[:, None, None]) & (slot < stop[:, None, None]))[:, :, None, :, None]
        at = (slot - start[:, None, None]).clamp(0, T - 1).reshape(B, 1, nt * BLOCK, 1).expand(B, kv, nt * BLOCK, d)
        opened = (blk[:, :, None] * BLOCK < start[:, None, None])           # [B, nt, 1]

        def write(x, codes, scale, mean):
            y = x.gather(2, at).reshape(B, kv, nt, BLOCK, d).transpose(1, 2).float()
            y = torch.where(new, y, 0.0)
            fresh = pow2_scale(y.abs().amax((3, 4)), s.kind)                # [B, nt, kv]
            was = scale[page]
            to = torch.where(opened, torch.maximum(was, fresh), fresh)
            kept = of_codes(codes[page], s.kind) * (was / to)[..., None, None]
            c = to_codes(torch.where(old, kept, y / to[..., None, None]), s.kind)
            codes[page[touched]] = c[touched]
            scale[page[touched]] = to[touched]
            if mean is not None:
                full = touched & ((blk + 1) * BLOCK <= stop[:, None])
                mean[page[full]] = (of_codes(c, s.kind).mean(3) * to[..., None])[full]

        write(s.new_k, s.k, s.k_scale, s.k_mean)
        write(s.new_v, s.v, s.v_scale, None)
        every = torch.arange(s.nb * BLOCK, device=dev)
        s.weight.masked_fill_(((every >= start[:, None]) & (every < stop[:, None]))[:, None], 0.0)
        s.lens_out.copy_(s.lens + s.n_new)
    return {"k": as_values(s.k, s.kind), "v": as_values(s.v, s.kind), "k_scale": s.k_scale, "v_scale": s.v_scale,
            "k_mean": s.k_mean, "weight": s.weight, "lens": s.lens_out}


def run_route(s):
    if own:
        import block_sparse_linear_sm_b200 as sla
        sla.sla_cache_route(s.q, s.cfg, s.cache, s.lens, s.n_new, s.sel)
        return s.sel
    B, H, T, d = s.q.shape
    kv, n = s.k.shape[1], s.sel.shape[2]
    dev = s.q.device
    live = (torch.arange(T, device=dev) < s.n_new[:, None])[:, None, :, None]
    # in 64 bits: the order of nearly equal blocks decides
    qbar = torch.where(live, s.q.double(), 0.0).sum(2) / s.n_new.clamp(min=1)[:, None, None]
    mean = s.k_mean[s.table.long()].double()                                # [B, nb, kv, d]
    score = torch.einsum("bkgd,bnkd->bkgn", qbar.reshape(B, kv, H // kv, d), mean) / math.sqrt(d)
    past = ((s.lens - s.n_new).clamp(min=0) // BLOCK)[:, None, None]
    is_past = torch.arange(s.nb, device=dev) < past                         # [B, 1, nb]
    score = score.masked_fill(~is_past[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-300)).sum(2)              # [B, kv, nb]
    p = p.masked_fill(~is_past, -1.0)
    val, at = p.sort(dim=-1, descending=True, stable=True)
    m = min(n, s.nb)
    at = torch.where(val[..., :m] >= 0, at[..., :m], s.nb).sort(-1).values
    s.sel.fill_(-1)
    s.sel[..., :m] = torch.where(at < s.nb, at, -1)
    return s.sel


def run_attend(s):
    if own:
        import block_sparse_linear_sm_b200 as sla
        sla.sla_cache_attend(s.q, s.cfg, s.cache, s.lens, s.n_new, s.sel, s.case["window"], s.out, s.ws)
    else:
        B, H, T, d = s.q.shape
        kv, dev, window = s.k.shape[1], s.q.device, s.case["window"]
        g, L = H // kv, s.nb * BLOCK
        table = s.table.long()

        def whole(codes, scale):
            x = of_codes(codes[table], s.kind) * scale[table][..., None, None]
            return x.permute(0, 2, 1, 3, 4).reshape(B, kv, L, d)

        score = s.q.float().reshape(B, kv, g * T, d) @ whole(s.k, s.k_scale).transpose(2, 3)
        score = score.reshape(B, kv, g, T, L) * (1.0 / math.sqrt(d))
        t = torch.arange(T, device=dev)
        pos = (s.lens - s.n_new)[:, None] + t                                # [B, T]
        slot = torch.arange(L, device=dev)
        sees = ((slot <= pos[..., None]) & (t < s.n_new[:, None])[..., None])[:, None, None]   # [B, 1, 1, T, L]
        near = (slot > pos[..., None] - window)[:, None, None]
        if s.sel is not None:
            chosen = torch.zeros(B, kv, s.nb + 1, dtype=torch.bool, device=dev)
            chosen.scatter_(2, torch.where(s.sel >= 0, s.sel, s.nb).long(), True)
            sees = sees & (chosen[..., :-1].repeat_interleave(BLOCK, -1)[:, :, None, None] | near)
        elif window:
            sees = sees & near
        score = score.masked_fill_(~sees, -math.inf)
        top = score.amax(-1, keepdim=True)
        score = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = score.sum(-1, keepdim=True)
        score = score.div_(torch.where(total == 0, 1.0, total))
        out = score.reshape(B, kv, g * T, L) @ whole(s.v, s.v_scale)
        s.out.copy_(out.reshape(B, H, T, d))
        if s.case["weights"]:
            s.weight += score.sum((2, 3))
    return {"out": s.out, "weight": s.weight} if s.case["weights"] else {"out": s.out}


def run_evict(s):
    budget, sink, recent = s.case["budget"], s.case["sink"], s.case["recent"]
    if own:
        import block_sparse_linear_sm_b200 as sla
        sla.sla_cache_evict(s.cfg, s.cache, s.lens, budget, sink, recent, s.dst, s.weight_out, s.kept, s.lens_out, s.ws)
    else:
        B, kv, L = s.weight.shape
        d, dev = s.k.shape[3], s.k.device
        lens = s.lens.long()[:, None, None]
        slot = torch.arange(L, device=dev)
        live = slot < lens
        held = live & ((slot < sink) | (slot >= lens - recent))
        key = s.weight.masked_fill(held, math.inf).masked_fill(~live, -math.inf)
        order = key.sort(dim=-1, descending=True, stable=True).indices
        m = lens.clamp(max=budget)                                            # [B, 1, 1]
        n = min(budget, L)
        at = torch.where(torch.arange(n, device=dev) < m, order[..., :n], L).sort(-1).values   # ascending slots
        is_kept = at < L
        s.kept.fill_(-1)
        s.kept[..., :n] = torch.where(is_kept, at, -1)
        s.lens_out.copy_(m.reshape(-1))
        s.weight_out[..., :n] = torch.where(is_kept, s.weight.gather(2, at.clamp(max=L - 1)), s.weight_out[..., :n])
        nd = s.dst.shape[1]
        src = torch.zeros(B, kv, nd * BLOCK, dtype=torch.long, device=dev)
        src[..., :n] = at.clamp(max=L - 1)
        good = torch.zeros(B, kv, nd * BLOCK, dtype=torch.bool, device=dev)
        good[..., :n] = is_kept
        page = s.table.long()[:, None].expand(B, kv, s.nb).gather(2, src // BLOCK)
        head = torch.arange(kv, device=dev)[None, :, None]
        dst = s.dst.long()[:, None].expand(B, kv, nd)
        used = (torch.arange(nd, device=dev) * BLOCK < m).expand(B, kv, nd)
        full = ((torch.arange(nd, device=dev) + 1) * BLOCK <= m).expand(B, kv, nd)
        hd = head.expand(B, kv, nd)

        def move(codes, scale, mean):
            x = of_codes(codes[page, head, src % BLOCK], s.kind) * scale[page, head][..., None]
            x = torch.where(good[..., None], x, 0.0).reshape(B, kv, nd, BLOCK, d)
            to = pow2_scale(x.abs().amax((3, 4)), s.kind)
            c = to_codes(x / to[..., None, None], s.kind)
            codes[dst[used], hd[used]] = c[used]
            scale[dst[used], hd[used]] = to[used]
            if mean is not None:
                mean[dst[full], hd[full]] = (of_codes(c, s.kind).mean(3) * to[..., None])[full]

        move(s.k, s.k_scale, s.k_mean)
        move(s.v, s.v_scale, None)
    return {"k": as_values(s.k, s.kind), "v": as_values(s.v, s.kind), "k_scale": s.k_scale, "v_scale": s.v_scale,
            "k_mean": s.k_mean, "weight": s.weight_out, "kept": s.kept, "lens": s.lens_out}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def _values64(codes, scale, kind):
    """The numbers that codes stand for, decoded from their bits."""
    u = codes.to(torch.int64)
    if kind == INT8:
        return torch.where(u > 127, u - 256, u).double() * scale.double()
    e, m = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(u >= 128, -mag, mag) * scale.double()


def _scale64(x, kind):
    a = float(x.abs().max()) if x.numel() else 0.0
    if a == 0:
        return 1.0
    top = 448.0 if kind == E4M3 else 127.0
    e = math.floor(math.log2(a / top)) - 1
    while top * 2.0 ** e < a:
        e += 1
    return 2.0 ** min(120, max(-110, e))


def _rounded64(x, kind):
    """x to the nearest value of the format, ties to even, in units of the scale."""
    if kind == INT8:
        return torch.round(x)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.pow(2.0, e + 1) <= x.abs(), e + 1, e)
    e = torch.where((torch.pow(2.0, e) > x.abs()) & (e > -6), e - 1, e)
    step = torch.pow(2.0, e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    lens, new = lengths(case), new_tokens(case)
    if case["op"] == "route" or (case["op"] in ("append", "evict") and case["B"] * case["H_kv"] * blocks_of(case) > 40000):
        return None
    s = prepare(case, seed)
    kind, d, kv = s.kind, case["d"], case["H_kv"]
    table = s.table.tolist()
    if case["op"] == "attend":
        g, T = case["H"] // kv, case["T"]
        out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
        weight = s.weight.double()
        for b in range(case["B"]):
            n = lens[b]
            if n == 0:
                continue
            pages = s.table[b, : -(-n // BLOCK)].long()
            slots = torch.arange(n, device="cuda")
            for h in range(kv):
                K = _values64(s.k[pages, h], s.k_scale[pages, h][:, None, None], kind).reshape(-1, d)[:n]
                V = _values64(s.v[pages, h], s.v_scale[pages, h][:, None, None], kind).reshape(-1, d)[:n]
                chosen = None
                if s.sel is not None:
                    mine = [j for j in s.sel[b, h].tolist() if j >= 0]
                    chosen = torch.zeros(len(pages) + 1, dtype=torch.bool, device="cuda")
                    chosen[mine] = True
                    chosen = chosen[slots // BLOCK]
                for t in range(new[b]):
                    pos = n - new[b] + t
                    if pos < 0:
                        continue
                    ok = slots <= pos
                    if chosen is not None:
                        ok &= chosen | (slots > pos - case["window"])
                    elif case["window"]:
                        ok &= slots > pos - case["window"]
                    if not bool(ok.any()):
                        continue
                    p = torch.softmax(s.q[b, h * g:(h + 1) * g, t].double() @ K[ok].T / math.sqrt(d), -1)
                    out[b, h * g:(h + 1) * g, t] = p @ V[ok]
                    weight[b, h, :n][ok] += p.sum(0)
        return {"out": out, "weight": weight} if case["weights"] else {"out": out}
    k, v = (_values64(c, torch.ones(1, device="cuda"), kind).cpu() for c in (s.k, s.v))
    ks, vs, km = s.k_scale.double().cpu(), s.v_scale.double().cpu(), s.k_mean.double().cpu()
    if case["op"] == "append":
        weight = s.weight.double().cpu()
        nk, nv = s.new_k.double().cpu(), s.new_v.double().cpu()
        for b in range(case["B"]):
            a, z = lens[b], lens[b] + new[b]
            if z == a:
                continue
            weight[b, :, a:z] = 0
            for j in range(a // BLOCK, -(-z // BLOCK)):
                lo, hi, pg = max(a, j * BLOCK), min(z, (j + 1) * BLOCK), table[b][j]
                keep = lo - j * BLOCK
                for h in range(kv):
                    for x, code, scale, mean in ((nk, k, ks, km), (nv, v, vs, None)):
                        rows = x[b, h, lo - a: hi - a]
                        to = _scale64(rows, kind)
                        if keep:
                            to = max(to, float(scale[pg, h]))
                        full = torch.zeros(BLOCK, d, dtype=torch.float64)
                        full[:keep] = _rounded64(code[pg, h, :keep] * (float(scale[pg, h]) / to), kind)
                        full[keep: keep + hi - lo] = _rounded64(rows / to, kind)
                        code[pg, h], scale[pg, h] = full, to
                        if mean is not None and hi == (j + 1) * BLOCK:
                            mean[pg, h] = full.mean(0) * to
    else:
        weight = s.weight_out.double().cpu()
        old = s.weight.cpu()
        dst = s.dst.tolist()
        k0, v0, ks0, vs0 = k.clone(), v.clone(), ks.clone(), vs.clone()
        for b in range(case["B"]):
            n, m = lens[b], min(lens[b], case["budget"])
            pages = torch.tensor(table[b])
            for h in range(kv):
                w = old[b, h, :n].tolist()
                held = [i for i in range(n) if i < case["sink"] or i >= n - case["recent"]]
                rest = sorted((i for i in range(case["sink"], n - case["recent"])), key=lambda i: (-w[i], i))
                if n <= m:
                    keep = list(range(n))
                else:
                    keep = sorted(held + rest[: m - len(held)])
                at = torch.tensor(keep, dtype=torch.long)
                weight[b, h, :m] = old[b, h, at].double()
                pg = pages[at // BLOCK]
                for code0, scale0, code, scale, mean in ((k0, ks0, k, ks, km), (v0, vs0, v, vs, None)):
                    x = code0[pg, h, at % BLOCK] * scale0[pg, h][:, None]
                    for j in range(-(-m // BLOCK)):
                        rows = x[j * BLOCK:(j + 1) * BLOCK]
                        to = _scale64(rows, kind)
                        full = torch.zeros(BLOCK, d, dtype=torch.float64)
                        full[: len(rows)] = _rounded64(rows / to, kind)
                        code[dst[b][j], h], scale[dst[b][j], h] = full, to
                        if mean is not None and len(rows) == BLOCK:
                            mean[dst[b][j], h] = full.mean(0) * to
    if kind == INT8:  # whole numbers: compared as they are
        k = v = None
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "k_mean": km, "weight": weight, "lens": None,
            **({"kept": None} if case["op"] == "evict" else {})}
