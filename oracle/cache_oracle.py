"""Float64 statement of the paged 8-bit cache (test infrastructure; shares no code with the
kernels): the two number formats, append, route, attend and evict as include/sla.h defines
them, one sequence, head and block at a time.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
E4M3, INT8 = 0, 1
MAX_ABS = 2.0 ** 120


def code_table(kind: int) -> np.ndarray:
    """The number each of the 256 code bytes stands for (e4m3: 0x7f and 0xff are NaN)."""
    u = np.arange(256)
    if kind == INT8:
        return np.where(u > 127, u - 256, u).astype(np.float64)
    sign, e, m = np.where(u > 127, -1.0, 1.0), (u >> 3) & 15, u & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    mag[(u & 127) == 127] = np.nan
    return sign * mag


def scale_of(a: float, kind: int) -> float:
    """The least power of two s >= 2^-110 with a <= top * s."""
    top = 448.0 if kind == E4M3 else 127.0
    s = 2.0 ** -110
    if a > top * s:
        s = 2.0 ** (math.frexp(a / top)[1] - 2)
        while a > top * s:
            s *= 2.0
    return s


def round_codes(x: np.ndarray, kind: int) -> np.ndarray:
    """Nearest code values, ties to even (x already divided by its scale, in range)."""
    if kind == INT8:
        return np.rint(x)
    _, e = np.frexp(x)
    step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)  # 3 mantissa bits, least normal 2^-6
    return np.rint(x / step) * step


class Cache:
    """Values of a cache: codes as numbers [n_pages, H_kv, 64, d], scales [n_pages, H_kv]."""

    def __init__(self, cfg, table):
        self.cfg, self.kind = cfg, cfg.kind
        shape = (cfg.n_pages, cfg.H_kv, BLOCK, cfg.d)
        self.k, self.v = np.zeros(shape), np.zeros(shape)
        self.ks, self.vs = np.zeros(shape[:2]), np.zeros(shape[:2])
        self.mean = np.zeros((cfg.n_pages, cfg.H_kv, cfg.d))
        self.weight = np.zeros((cfg.B, cfg.H_kv, cfg.max_blocks * BLOCK))
        self.table = np.array(table)
        self.scale = cfg.scale if cfg.scale > 0 else 1.0 / math.sqrt(cfg.d)

    # -- append ----------------------------------------------------------------
    def append(self, k, v, lens, n_new):
        k, v = (np.clip(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf), -MAX_ABS, MAX_ABS)
                for x in (k, v))
        for b, (a, n) in enumerate(zip(lens, n_new)):
            for j in range(a // BLOCK, -(-(a + n) // BLOCK) if n else a // BLOCK):
                lo, hi = max(a, j * BLOCK), min(a + n, (j + 1) * BLOCK)
                pg, r = self.table[b, j], lo - j * BLOCK
                for h in range(self.cfg.H_kv):
                    for x, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                        rows = x[b, h, lo - a:hi - a]
                        to = scale_of(np.abs(rows).max(), self.kind)
                        if r:
                            to = max(to, scales[pg, h])
                            codes[pg, h, :r] = round_codes(codes[pg, h, :r] * (scales[pg, h] / to), self.kind)
                        codes[pg, h, r:] = 0
                        codes[pg, h, r:r + hi - lo] = round_codes(rows / to, self.kind)
                        scales[pg, h] = to
                    self.weight[b, h, lo:hi] = 0
                    if hi == (j + 1) * BLOCK:
                        self.mean[pg, h] = self.k[pg, h].mean(0) * self.ks[pg, h]
        return np.array(lens) + np.array(n_new)

    # -- reading ----------------------------------------------------------------
    def rows(self, b, h, n):
        """Keys and values [n, d] of the first n slots."""
        pg = self.table[b, :-(-n // BLOCK)]
        K = (self.k[pg, h] * self.ks[pg, h][:, None, None]).reshape(-1, self.cfg.d)[:n]
        V = (self.v[pg, h] * self.vs[pg, h][:, None, None]).reshape(-1, self.cfg.d)[:n]
        return K, V

    def route(self, q, lens, n_new, top_n):
        """(lists [B, H_kv, top_n], relative gap between the last block in and the first out)."""
        c, g = self.cfg, self.cfg.H // self.cfg.H_kv
        sel = np.full((c.B, c.H_kv, top_n), -1)
        gap = np.inf
        for b in range(c.B):
            past = max(0, lens[b] - n_new[b]) // BLOCK if n_new[b] else 0
            if not past:
                continue
            for h in range(c.H_kv):
                m = self.mean[self.table[b, :past], h]
                p = np.zeros(past)
                for i in range(g):
                    s = m @ q[b, h * g + i, :n_new[b]].mean(0) * self.scale
                    e = np.exp(s - s.max())
                    p += e / e.sum()
                order = np.argsort(-p, kind="stable")
                top = np.sort(order[:top_n])
                sel[b, h, :len(top)] = top
                if past > top_n:
                    x, y = p[order[top_n - 1]], p[order[top_n]]
                    gap = min(gap, (x - y) / x)
        return sel, gap

    def attend(self, q, lens, n_new, sel, window, add_weight=False):
        """(out, sum of p |v| for each output, added weight)."""
        c, g = self.cfg, self.cfg.H // self.cfg.H_kv
        out, mag = np.zeros(q.shape), np.zeros(q.shape)
        got = np.zeros_like(self.weight)
        for b in range(c.B):
            n = lens[b]
            slots = np.arange(n)
            for h in range(c.H_kv):
                K, V = self.rows(b, h, n)
                chosen = np.isin(slots // BLOCK, [j for j in sel[b, h] if j >= 0]) if sel is not None else None
                for t in range(n_new[b]):
                    pos = n - n_new[b] + t
                    ok = slots <= pos
                    if chosen is not None:
                        ok &= chosen | (slots > pos - window)
                    elif window:
                        ok &= slots > pos - window
                    if not ok.any():
                        continue
                    s = q[b, h * g:(h + 1) * g, t] @ K[ok].T * self.scale
                    p = np.exp(s - s.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    out[b, h * g:(h + 1) * g, t] = p @ V[ok]
                    mag[b, h * g:(h + 1) * g, t] = p @ np.abs(V[ok])
                    got[b, h, :n][ok] += p.sum(0)
        if add_weight:
            self.weight += got
        return out, mag, got

    # -- evict ------------------------------------------------------------------
    def evict(self, lens, budget, n_sink, n_recent, dst, weight_out):
        """kept [B, H_kv, budget]; the kept slots move to dst, their weights into weight_out."""
        c = self.cfg
        kept = np.full((c.B, c.H_kv, budget), -1)
        old = {n: getattr(self, n).copy() for n in ("k", "v", "ks", "vs", "weight")}
        for b in range(c.B):
            n, m = lens[b], min(lens[b], budget)
            for h in range(c.H_kv):
                w = old["weight"][b, h, :n].copy()
                w[np.isnan(w)] = -np.inf
                if n <= budget:
                    keep = np.arange(n)
                else:
                    mid = np.arange(n_sink, n - n_recent)
                    best = mid[np.argsort(-w[mid], kind="stable")][:budget - n_sink - n_recent]
                    keep = np.sort(np.concatenate([np.arange(n_sink), best, np.arange(n - n_recent, n)])).astype(int)
                kept[b, h, :m] = keep
                weight_out[b, h, :m] = old["weight"][b, h, keep]
                pg = self.table[b, keep // BLOCK]
                for codes, scales in (("k", "ks"), ("v", "vs")):
                    x = old[codes][pg, h, keep % BLOCK] * old[scales][pg, h][:, None]
                    for j in range(-(-m // BLOCK)):
                        rows = x[j * BLOCK:(j + 1) * BLOCK]
                        to = scale_of(np.abs(rows).max(), self.kind)
                        getattr(self, codes)[dst[b, j], h] = 0
                        getattr(self, codes)[dst[b, j], h, :len(rows)] = round_codes(rows / to, self.kind)
                        getattr(self, scales)[dst[b, j], h] = to
                        if codes == "k" and len(rows) == BLOCK:
                            self.mean[dst[b, j], h] = self.k[dst[b, j], h].mean(0) * to
        return kept
