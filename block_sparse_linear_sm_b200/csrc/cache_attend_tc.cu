// sla_cache_attend for many query rows of a KV head: T * H / H_kv of several dozen to 1024.
//
// With R rows a cached key byte takes 2 R multiplications and so does a value byte: from some
// dozen rows on the products, not the cache's bytes, set the time, and a page should be
// decoded once for all rows. So the rows form groups of 128, the M of tcgen05.mma, and the
// tile is one page for one group; the line of tiles is cut into runs as in the kernel for few
// rows, one CTA an SM. In a CTA
//   warp 0          looks the run's tiles up, 32 at a time, and loads their pages by TMA;
//   warps 8 - 11    turn a page's codes into fp16 (exactly) in the layouts that the products
//                   read, K [slot][d] and V [slot][d] (N-major), 128-byte swizzle;
//   warp 1          issues S = Q K^T (M 128, N 64) and, one page behind, P V (M 128, N d) with
//                   P as the operand in TMEM;
//   warps 4 - 7     own a row a thread: maximum, P = 2^(S - m + 8) as fp16 back to TMEM, and, a
//                   page behind, O = O + 2^-8 v_scale * (P V) in fp32 registers (times 2^-18,
//                   kOutShift).
// Each page's P V goes to a buffer of its own (two, in turn) instead of accumulating in TMEM:
// pages have value scales of their own, and with O in registers neither they nor a new maximum
// need a pass over TMEM. m is raised, and O scaled, only when a maximum exceeds it by 2^7, so
// that P stays below 2^15; a weight below 2^-33 of m's may round to 0. Q is scaled as in the
// kernel for few rows. S and P are double buffered, so that the softmax of one page runs while
// the products of the next are issued.
// What bounds it: the row warps' chain, about 2600 cycles a page (maximum 450, exponentials 690,
// P V 630, barriers and descriptions 700, read from the clock in an instrumented copy); the
// products need about 520 of them, the page's bytes 710. 8 sequences of up to 16001 tokens, 4 KV
// heads, 128 rows: 66 us on the device. No pipe is near full (profiles/cache_calls.md: tensor
// 13 %, exponentials and conversions 16 %, 29 % of the issue slots). Splitting the row work over
// two warpgroups, by pages (two outputs merged at the end) or by kind (softmax apart from O), did
// not shorten it: each part then took almost twice as long, for a reason that was not found.
#include "cache_attend.cuh"

namespace sla {
namespace {

using namespace attend;

constexpr int kThreads = 384;
constexpr int kRaw = 4;     // pages of codes in flight, keys and values together
constexpr int kInfo = 16;   // described tiles
constexpr float kTcShift = 8.f, kTcSlack = 7.f;

struct __align__(16) Info {
  int seg;      // segment of the line, -1: the run is over
  int real;     // 0: the segment has no page in this run (seg only)
  int block, tile, chosen, live;  // live: slots that hold tokens
  float ks, vs;
};

template <int D>
struct Smem {
  static constexpr int kPage = kBlock * D;      // bytes of codes
  static constexpr int kHalf = kBlock * D * 2;  // the same in fp16
  static constexpr int off_q = 0;               // [D / 64][128 rows][128 bytes]
  static constexpr int off_k = off_q + kTcGroupRows * D * 2;
  static constexpr int off_v = off_k + 2 * kHalf;
  static constexpr int off_raw = off_v + 2 * kHalf;
  static constexpr int off_misc = off_raw + kRaw * 2 * kPage;
  static constexpr int kMisc = 2048;
  static constexpr int off_lines = off_misc + kMisc;
  static size_t bytes(int B) { return off_lines + lines_bytes(B); }
};

struct __align__(16) Misc {
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], s_empty[2], p_full[2], o_full[2], o_empty[2];
  uint64_t q_full, info_full[kInfo], info_empty[kInfo];
  Info info[kInfo];
  int warp_sums[kThreads / 32];
  uint32_t tmem;
  int abort, never;
};

// TMEM columns
template <int D>
struct Cols {
  static constexpr int s = 0, p = 128, acc = 192;  // S 2 x 64, P 2 x 32, P V 2 x D
};

// instruction descriptor of kind::f16 with fp16 A and B and fp32 D (the bf16 one without its
// two type bits)
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return tc::idesc_bf16(M, N, false, b_mn) & ~((1u << 7) | (1u << 10));
}

// Waits as a warp; false (for all lanes) when the wait ran out or another warp gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, unsigned phase, Misc& mi) {
  return __all_sync(0xffffffffu, tc::mbar_wait(smem_u32(bar), phase & 1, &mi.abort));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(smem_u32(bar));
}
// Reads entry e; every reader's warps give it back.
__device__ __forceinline__ bool read_info(Misc& mi, unsigned e, int lane, Info* out) {
  if (!wait_all(&mi.info_full[e % kInfo], e / kInfo, mi)) return false;
  const int4* p = reinterpret_cast<const int4*>(&mi.info[e % kInfo]);
  const int4 x = p[0], y = p[1];
  out->seg = x.x;
  out->real = x.y;
  out->block = x.z;
  out->tile = x.w;
  out->chosen = y.x;
  out->live = y.y;
  out->ks = __int_as_float(y.z);
  out->vs = __int_as_float(y.w);
  arrive_warp(&mi.info_empty[e % kInfo], lane);
  return true;
}

// Block of tile idx of (b, hk), for one lane by itself; -1 where it is none.
__device__ int lane_block(const CacheView& c, const Step& a, int b, int hk, int idx, int L, int n, bool* chosen) {
  const int first = first_block(a, L, n);
  *chosen = a.window == 0;
  if (a.sel == nullptr) return first + idx;
  const int32_t* list = a.sel + ((size_t)b * c.H_kv + hk) * a.top_n;
  const int listed = listed_tiles(a, L), j = first + idx - listed, blocks = (L + kBlock - 1) / kBlock;
  int top = -1, valid = 0, entry = -1;  // entry: the valid one that idx of them are before
  bool bad = false, twice = false;      // twice: j is in the list
  for (int i = 0; i < a.top_n; ++i) {
    const int e = list[i];
    if (e > top && e < blocks) {
      if (valid++ == idx) entry = e;
      if (e == j) twice = true;
    } else if (e >= 0) {
      bad = true;
    }
    top = max(top, e);
  }
  if (bad) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheSel);
  *chosen = idx < listed;
  if (*chosen) return entry;
  return twice ? -1 : j;
}

// ---------------------------------------------------------------------------
// warp 0: tiles and pages
// ---------------------------------------------------------------------------
template <int D>
__device__ bool produce(const CacheView& c, const Step& a, const Lines& l, Misc& mi, char* smem,
                        const CUtensorMap* kmap, const CUtensorMap* vmap, unsigned lo, unsigned hi, int lane,
                        unsigned* issued) {
  using Sm = Smem<D>;
  const unsigned per = c.H_kv * a.groups;
  unsigned e = 0;
  auto put = [&](const Info& x) -> bool {
    if (e >= kInfo && !wait_all(&mi.info_empty[e % kInfo], e / kInfo - 1, mi)) return false;
    if (lane == 0) {
      mi.info[e % kInfo] = x;
      tc::mbar_arrive(smem_u32(&mi.info_full[e % kInfo]));
    }
    __syncwarp();
    ++e;
    return true;
  };
  Segment sg;
  sg.b = find_sequence(l, c.B, lo, per);
  sg.nb = l.cum[sg.b + 1] - l.cum[sg.b];
  sg.sr = (int)((lo - (unsigned)l.cum[sg.b] * per) / sg.nb);
  sg.lo = (unsigned)l.cum[sg.b] * per + sg.sr * sg.nb;
  for (;;) {
    const int L = l.len[sg.b], n = l.fresh[sg.b], hk = sg.sr / a.groups, seg = sg.b * (int)per + sg.sr;
    const int i0 = (int)(max(lo, sg.lo) - sg.lo), i1 = (int)(min(hi, sg.lo + sg.nb) - sg.lo);
    bool any = false;
    for (int base = i0; base < i1; base += 32) {
      const int idx = base + lane;
      bool chosen = false;
      int j = -1, page = -1;
      float ks = 0.f, vs = 0.f;
      if (idx < i1) j = lane_block(c, a, sg.b, hk, idx, L, n, &chosen);
      if (j >= 0) page = checked_page(c, sg.b, j);
      const int ph = page * c.H_kv + hk;
      if (page >= 0) {
        ks = c.k_scale[ph];
        vs = c.v_scale[ph];
      }
      uint32_t todo = __ballot_sync(0xffffffffu, page >= 0);
      for (; todo != 0; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        Info x;
        x.seg = seg;
        x.real = 1;
        x.block = __shfl_sync(0xffffffffu, j, src);
        x.tile = l.cum[sg.b] * c.H_kv + hk * (int)sg.nb + base + src;
        x.chosen = __shfl_sync(0xffffffffu, (int)chosen, src);
        x.live = min(kBlock, L - x.block * kBlock);
        x.ks = __shfl_sync(0xffffffffu, ks, src);
        x.vs = __shfl_sync(0xffffffffu, vs, src);
        const int row = __shfl_sync(0xffffffffu, ph, src) * kBlock;
        const unsigned i = *issued, stage = i % kRaw;
        if (i >= kRaw && !wait_all(&mi.raw_empty[stage], i / kRaw - 1, mi)) return false;
        if (lane == 0) {
          const uint32_t dst = smem_u32(smem + Sm::off_raw) + stage * 2 * Sm::kPage, bar = smem_u32(&mi.raw_full[stage]);
          tc::mbar_expect_tx(bar, 2 * Sm::kPage);
          tma_load_rows(dst, kmap, bar, row);
          tma_load_rows(dst + Sm::kPage, vmap, bar, row);
        }
        ++*issued;
        if (!put(x)) return false;
        any = true;
      }
    }
    if (!any) {
      Info x = {};
      x.seg = seg;
      if (!put(x)) return false;
    }
    if (sg.lo + sg.nb >= hi) break;
    next_segment(sg, l, per);
  }
  Info x = {};
  x.seg = -1;
  return put(x);
}

// ---------------------------------------------------------------------------
// warp 1: products
// ---------------------------------------------------------------------------
// *pages: pages whose S was issued; *outputs: those whose P V was.
template <int D>
__device__ bool multiply(Misc& mi, char* smem, uint32_t tmem, int lane, unsigned* pages, unsigned* outputs) {
  using Sm = Smem<D>;
  constexpr uint32_t kIdS = idesc_f16(128, 64, false), kIdO = idesc_f16(128, D, true);
  const uint64_t dq = tc::sw128_desc(smem_u32(smem + Sm::off_q), 16, 1024);
  const uint64_t dk = tc::sw128_desc(smem_u32(smem + Sm::off_k), 16, 1024);
  const uint64_t dv = tc::sw128_desc(smem_u32(smem + Sm::off_v), 8192, 1024);
  unsigned page = 0, segs = 0;
  int seg = -1;
  bool owed = false;  // P V of page - 1
  auto values = [&](unsigned i) -> bool {
    const unsigned b = i & 1;
    if (!wait_all(&mi.v_full[b], i >> 1, mi) || !wait_all(&mi.p_full[b], i >> 1, mi) ||
        (i >= 2 && !wait_all(&mi.o_empty[b], (i >> 1) - 1, mi)))
      return false;
    tc::fence_after_sync();
    if (tc::elect_one()) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc::mma_bf16_ts(tmem + Cols<D>::acc + b * D, tmem + Cols<D>::p + 32 * b + 8 * k,
                        dv + (uint32_t)((b * Sm::kHalf + k * 2048) >> 4), kIdO, k > 0);
      tc::mma_commit(smem_u32(&mi.o_full[b]));
      tc::mma_commit(smem_u32(&mi.v_empty[b]));
    }
    __syncwarp();
    *outputs = i + 1;
    return true;
  };
  for (unsigned e = 0;; ++e) {
    Info x;
    if (!read_info(mi, e, lane, &x)) return false;
    if (x.seg < 0) break;
    if (x.seg != seg) {  // the rows are waiting for the last product of the segment before
      if (owed && !values(page - 1)) return false;
      owed = false;
    }
    if (!x.real) continue;
    if (x.seg != seg) {
      if (!wait_all(&mi.q_full, segs++, mi)) return false;
      seg = x.seg;
    }
    const unsigned b = page & 1;
    if (!wait_all(&mi.k_full[b], page >> 1, mi) || (page >= 2 && !wait_all(&mi.s_empty[b], (page >> 1) - 1, mi)))
      return false;
    tc::fence_after_sync();
    if (tc::elect_one()) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_bf16_ss(tmem + Cols<D>::s + 64 * b, dq + (uint32_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                        dk + (uint32_t)((b * Sm::kHalf + (k >> 2) * 8192 + (k & 3) * 32) >> 4), kIdS, k > 0);
      tc::mma_commit(smem_u32(&mi.s_full[b]));
      tc::mma_commit(smem_u32(&mi.k_empty[b]));
    }
    __syncwarp();
    *pages = page + 1;
    if (owed && !values(page - 1)) return false;
    owed = true;
    ++page;
  }
  return !owed || values(page - 1);
}

// ---------------------------------------------------------------------------
// warps 8 - 11: codes to fp16
// ---------------------------------------------------------------------------
// One page of codes (TMA's swizzle of D-byte rows) to fp16 panels of 64 columns, 128-byte rows
// and swizzle. Eight lanes take 16-byte chunks of two neighbouring rows such that neither the
// loads nor the stores meet in a bank. Rows from `live` on become 0.
template <int KIND, int D>
__device__ __forceinline__ void decode_page(uint32_t src, uint32_t dst, int tid, int live) {
  constexpr int kTurns = D / 64;  // chunk halves of a row
  constexpr int kLanes = 128, kAll = 256 / kLanes * kTurns, kBatch = kAll < 4 ? kAll : 4;
#pragma unroll
  for (int i0 = 0; i0 < kAll; i0 += kBatch) {
    uint4 x[kBatch];
    int row[kBatch], ch[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {  // the loads of a batch together: each is waited for once
      const int i = i0 + k, o = (tid + kLanes * (i / kTurns)) >> 3, w = tid & 7, turn = i % kTurns;
      row[k] = 2 * o + (w >> 2);
      ch[k] = D == 128 ? (w & 3) + 4 * (turn ^ (w >> 2)) : w & 3;
      x[k] = lds128(src + row[k] * D + ((ch[k] ^ (D == 128 ? (row[k] & 7) : ((row[k] >> 1) & 3))) << 4));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      uint32_t h[8];
      decode4_f16<KIND>(x[k].x, h[0], h[1]);
      decode4_f16<KIND>(x[k].y, h[2], h[3]);
      decode4_f16<KIND>(x[k].z, h[4], h[5]);
      decode4_f16<KIND>(x[k].w, h[6], h[7]);
      if (live < kBlock && row[k] >= live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = 0u;
      }
      const uint32_t at = dst + (ch[k] >> 2) * 8192 + row[k] * 128;
      const int c16 = 2 * (ch[k] & 3);
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((c16 ^ (row[k] & 7)) << 4)), "r"(h[0]),
                   "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((c16 + 1) ^ (row[k] & 7)) << 4)), "r"(h[4]),
                   "r"(h[5]), "r"(h[6]), "r"(h[7])
                   : "memory");
    }
  }
}

template <int KIND, int D>
__device__ bool convert(Misc& mi, char* smem, int tid, int lane) {
  using Sm = Smem<D>;
  unsigned page = 0;
  for (unsigned e = 0;; ++e) {
    Info x;
    if (!read_info(mi, e, lane, &x)) return false;
    if (x.seg < 0) return true;
    if (!x.real) continue;
    const unsigned b = page & 1, stage = page % kRaw;
    const uint32_t raw = smem_u32(smem + Sm::off_raw) + stage * 2 * Sm::kPage;
    if (!wait_all(&mi.raw_full[stage], page / kRaw, mi)) return false;
    if (page >= 2 && !wait_all(&mi.k_empty[b], (page >> 1) - 1, mi)) return false;
    decode_page<KIND, D>(raw, smem_u32(smem + Sm::off_k) + b * Sm::kHalf, tid, x.live);
    tc::fence_async_smem();
    arrive_warp(&mi.k_full[b], lane);
    if (page >= 2 && !wait_all(&mi.v_empty[b], (page >> 1) - 1, mi)) return false;
    decode_page<KIND, D>(raw + Sm::kPage, smem_u32(smem + Sm::off_v) + b * Sm::kHalf, tid, x.live);
    tc::fence_async_smem();
    arrive_warp(&mi.v_full[b], lane);
    arrive_warp(&mi.raw_empty[stage], lane);
    ++page;
  }
}

// ---------------------------------------------------------------------------
// warps 4 - 7: a row a thread
// ---------------------------------------------------------------------------
template <int D>
__device__ bool rows_of_step(const CacheView& c, const Step& a, const Lines& l, Misc& mi, char* smem, uint32_t tmem,
                             unsigned lo, unsigned hi, int warp, int lane) {
  using Sm = Smem<D>;
  const unsigned per = c.H_kv * a.groups;
  const int r = 32 * (warp & 3) + lane;  // row of the group and TMEM lane
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  uint64_t o[D / 2];
  float m = -INFINITY, sum = 0.f, qs = 0.f, owed_vs = 0.f;
  unsigned page = 0;
  int seg = -1, b = 0, L = 0, n = 0, row = 0, pos = -1;
  size_t qrow = 0;
  bool owed = false;  // P V of page - 1

  // O += v_scale * (P V) of page i, with `meanwhile` done while the first columns are on their way
  auto collect = [&](unsigned i, auto meanwhile) -> bool {
    const unsigned k = i & 1;
    if (!wait_all(&mi.o_full[k], i >> 1, mi)) return false;
    tc::fence_after_sync();
    const uint64_t v2 = tc::f2_pack(owed_vs, owed_vs);
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      uint32_t x[32], y[32];
      tc::tmem_ld32(lanes + Cols<D>::acc + k * D + 64 * u, x);
      tc::tmem_ld32(lanes + Cols<D>::acc + k * D + 64 * u + 32, y);
      if (u == 0) meanwhile();
      tc::tmem_ld_wait();
#pragma unroll
      for (int i2 = 0; i2 < 16; ++i2) {
        o[32 * u + i2] = tc::ffma2(v2, (uint64_t)x[2 * i2] | ((uint64_t)x[2 * i2 + 1] << 32), o[32 * u + i2]);
        o[32 * u + 16 + i2] =
            tc::ffma2(v2, (uint64_t)y[2 * i2] | ((uint64_t)y[2 * i2 + 1] << 32), o[32 * u + 16 + i2]);
      }
    }
    tc::fence_before_sync();
    arrive_warp(&mi.o_empty[k], lane);
    return true;
  };

  for (unsigned e = 0;; ++e) {
    Info x;
    if (!read_info(mi, e, lane, &x)) return false;
    if (x.seg != seg) {
      if (owed && !collect(page - 1, [] {})) return false;
      owed = false;
      if (seg >= 0) {
        const int sr = seg % (int)per, nb = l.cum[b + 1] - l.cum[b];
        const unsigned seg_lo = (unsigned)l.cum[b] * per + (unsigned)sr * nb;
        const float all = sum * exp2_int(-(int)kTcShift);
        const bool whole = seg_lo >= lo && seg_lo + nb <= hi;
        const size_t part = (size_t)blockIdx.x + seg;
        if (!whole || a.scores != nullptr) {
          a.part_ml[part * 2 * kTcGroupRows + r] = m;
          a.part_ml[part * 2 * kTcGroupRows + kTcGroupRows + r] = all;
        }
        if (whole) {
          if (row < a.rows) {
            const bool empty = all == 0.f || pos < 0;
            const float inv = 1.f / out_divisor(all);
            uint4* out = reinterpret_cast<uint4*>(a.out + qrow * D);
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = empty ? 0u : pack_bf16(tc::f2_lo(o[4 * u + i]) * inv, tc::f2_hi(o[4 * u + i]) * inv);
              out[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (a.lse != nullptr) a.lse[qrow] = log2_sum(m, all);
          }
        } else {
          ulonglong2* out = reinterpret_cast<ulonglong2*>(a.part_o + (part * kTcGroupRows + r) * D);
#pragma unroll
          for (int u = 0; u < D / 4; ++u) out[u] = make_ulonglong2(o[2 * u], o[2 * u + 1]);
        }
      }
      if (x.seg < 0) return true;
      seg = x.seg;
      b = seg / (int)per;
      const int sr = seg % (int)per, hk = sr / a.groups;
      L = l.len[b];
      n = l.fresh[b];
      row = sr % a.groups * kTcGroupRows + r;
      qrow = ((size_t)b * c.H + (size_t)hk * c.group) * a.T + row;
      const int t = row % a.T;
      pos = row < a.rows && t < n ? L - n + t : -1;
      m = -INFINITY;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < D / 2; ++i) o[i] = 0ull;
      if (x.real) {  // Q's row, all earlier products with the old ones being done
        uint4 w[D / 8];
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          w[u] = row < a.rows ? reinterpret_cast<const uint4*>(a.q + qrow * D)[u] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16(ws[i]);
            top = tc::fmax3(top, fabsf(f.x), fabsf(f.y));
          }
        }
        const int ex = max((int)(__float_as_uint(top) >> 23) - 127, -100);
        const float up = row_factor(top, ex);
        qs = exp2_int(ex - 14) * (c.scale * 1.4426950408889634f);
        const uint32_t at = smem_u32(smem + Sm::off_q) + r * 128;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16(ws[i]);
            h[i] = pack_f16(f.x * up, f.y * up);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (u >> 3) * 16384 + (((u & 7) ^ (r & 7)) << 4)),
                       "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
        }
        tc::fence_async_smem();
        arrive_warp(&mi.q_full, lane);
      }
    }
    if (!x.real) continue;

    const unsigned k = page & 1;
    if (!wait_all(&mi.s_full[k], page >> 1, mi)) return false;
    tc::fence_after_sync();
    float s[64];
    {
      uint32_t s0[32], s1[32];
      tc::tmem_ld32(lanes + Cols<D>::s + 64 * k, s0);
      tc::tmem_ld32(lanes + Cols<D>::s + 64 * k + 32, s1);
      tc::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        s[i] = __uint_as_float(s0[i]);
        s[32 + i] = __uint_as_float(s1[i]);
      }
    }
    tc::fence_before_sync();
    arrive_warp(&mi.s_empty[k], lane);
    const int j0 = x.block * kBlock;
    if (j0 + kBlock - 1 > L - n || (!x.chosen && j0 <= L - 1 - a.window)) {
      const int last = pos - j0, first = x.chosen ? -1 : pos - a.window - j0;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (i > last || i <= first) s[i] = -INFINITY;
    }
    const float f = fmaxf(qs * x.ks, 1e-37f);
    if (a.scores != nullptr && row < a.rows) {
      float* p = a.scores + (size_t)x.tile * kBlock * a.score_rows + row;
#pragma unroll
      for (int i = 0; i < 64; ++i) p[(size_t)i * a.score_rows] = s[i] * f;
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int i = 4; i < 64; i += 8)
#pragma unroll
      for (int u = 0; u < 4; ++u) mx[u] = i + 4 + u < 64 ? tc::fmax3(mx[u], s[i + u], s[i + 4 + u]) : fmaxf(mx[u], s[i + u]);
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    // x = (s - page's maximum) * f + (its scaled value - m) + shift, with m raised first where
    // the value exceeds it by the slack
    const float low = top == -INFINITY ? 0.f : top, scaled = __fmul_rn(top, f);
    const bool raise = scaled > m + kTcSlack;
    const float alpha = raise ? tc::ex2_approx(m - scaled) : 1.f;
    const bool any_raise = __any_sync(0xffffffffu, raise);
    m = raise ? scaled : m;
    sum *= alpha;
    const float off = (scaled == -INFINITY ? 0.f : scaled - (m == -INFINITY ? 0.f : m)) + kTcShift;
    const uint64_t f2 = tc::f2_pack(f, f), l2 = tc::f2_pack(low, low), o2 = tc::f2_pack(off, off);
    uint32_t pk[32];
    uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint64_t y = tc::ffma2(tc::fsub2(tc::f2_pack(s[2 * i], s[2 * i + 1]), l2), f2, o2);
      const float p0 = tc::ex2_approx(tc::f2_lo(y)), p1 = tc::ex2_approx(tc::f2_hi(y));
      s2[i & 1] = tc::fadd2(s2[i & 1], tc::f2_pack(p0, p1));
      pk[i] = pack_f16(p0, p1);
    }
    s2[0] = tc::fadd2(s2[0], s2[1]);
    sum += tc::f2_lo(s2[0]) + tc::f2_hi(s2[0]);
    // this buffer's P was read by the product that was collected a page ago
    tc::tmem_st32(lanes + Cols<D>::p + 32 * k, pk);
    auto hand_over = [&] {
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive_warp(&mi.p_full[k], lane);
    };
    if (!owed) hand_over();
    else if (!collect(page - 1, hand_over)) return false;
    if (any_raise) {
      const uint64_t a2 = tc::f2_pack(alpha, alpha);
#pragma unroll
      for (int i = 0; i < D / 2; ++i) o[i] = tc::fmul2(o[i], a2);
    }
    owed = true;
    owed_vs = x.vs * exp2_int(-(int)kTcShift - kOutShift);
    ++page;
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const CacheView c, const Step a) {
  using Sm = Smem<D>;
  extern __shared__ __align__(1024) char smem[];
  static_assert(sizeof(Misc) <= Sm::kMisc, "misc");
  Misc& mi = *reinterpret_cast<Misc*>(smem + Sm::off_misc);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    mi.abort = mi.never = 0;
    auto init = [](uint64_t* bar, int n, int count) {
      for (int i = 0; i < n; ++i) tc::mbar_init(smem_u32(bar + i), count);
    };
    init(mi.raw_full, kRaw, 1);
    init(mi.raw_empty, kRaw, 4);
    init(mi.k_full, 2, 4);
    init(mi.k_empty, 2, 1);
    init(mi.v_full, 2, 4);
    init(mi.v_empty, 2, 1);
    init(mi.s_full, 2, 1);
    init(mi.s_empty, 2, 4);
    init(mi.p_full, 2, 4);
    init(mi.o_full, 2, 1);
    init(mi.o_empty, 2, 4);
    init(&mi.q_full, 1, 4);
    init(mi.info_full, kInfo, 1);
    init(mi.info_empty, kInfo, 9);  // the product warp, four converting, four row warps
    tc::fence_mbar_init();
    tc::prefetch_tensormap(&kmap);
    tc::prefetch_tensormap(&vmap);
  }
  Lines l;
  wait_for_previous();
  scan_lines(c, a, smem + Sm::off_lines, &l, mi.warp_sums);
  let_next_start();
  const unsigned per = c.H_kv * a.groups, total = (unsigned)l.cum[c.B] * per;
  const unsigned run = run_length(a, total, c.B * per, gridDim.x);
  const unsigned lo = min(total, blockIdx.x * run), hi = min(total, lo + run);
  if (lo >= hi) return;
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&mi.tmem), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = mi.tmem;

  // registers of the three warpgroups: 80 + 240 + 120 a thread of the launch's 3 x 168
  bool ok = true;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) {
      unsigned issued = 0;
      ok = produce<D>(c, a, l, mi, smem, &kmap, &vmap, lo, hi, lane, &issued);
      if (!ok) mi.abort = 1;
      // loads on their way land before the block's memory is given back
      for (unsigned i = issued > kRaw ? issued - kRaw : 0; i < issued; ++i)
        tc::mbar_wait(smem_u32(&mi.raw_full[i % kRaw]), (i / kRaw) & 1, &mi.never);
    } else if (warp == 1) {
      unsigned pages = 0, outputs = 0;
      ok = multiply<D>(mi, smem, tmem, lane, &pages, &outputs);
      if (!ok) mi.abort = 1;
      // products on their way end before TMEM and the block's memory are given back, also where
      // another wait ran out
      for (unsigned i = pages > 2 ? pages - 2 : 0; i < pages; ++i)
        ok = tc::mbar_wait(smem_u32(&mi.k_empty[i & 1]), (i >> 1) & 1, &mi.never) && ok;
      for (unsigned i = outputs > 2 ? outputs - 2 : 0; i < outputs; ++i)
        ok = tc::mbar_wait(smem_u32(&mi.v_empty[i & 1]), (i >> 1) & 1, &mi.never) && ok;
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    ok = rows_of_step<D>(c, a, l, mi, smem, tmem, lo, hi, warp, lane);
    if (!ok) tc::tmem_st_wait();  // P, which was not handed over
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    ok = convert<KIND, D>(mi, smem, tid & 127, lane);
  }
  if (!ok) {
    mi.abort = 1;
    if (lane == 0) report(c.status, SLA_ERR_DEVICE_TIMEOUT, kDetailTimeout);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

template <int KIND, int D>
cudaError_t launch(const CacheView& c, const Step& a, int ctas, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)c.n_pages * c.H_kv * kBlock;
  if (!make_tmap_rows_u8(&kmap, c.k, rows, D, kBlock) || !make_tmap_rows_u8(&vmap, c.v, rows, D, kBlock))
    return cudaErrorInvalidValue;
  auto kernel = attend_tc_kernel<KIND, D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D>::bytes(kCacheMaxB));
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, dim3(ctas), kThreads, Smem<D>::bytes(c.B), s, kmap, vmap, c, a);
}

}  // namespace

cudaError_t launch_attend_tc(const CacheView& c, const attend::Step& a, int ctas, cudaStream_t s) {
  if (c.kind == SLA_CACHE_E4M3)
    return c.d == 128 ? launch<SLA_CACHE_E4M3, 128>(c, a, ctas, s) : launch<SLA_CACHE_E4M3, 64>(c, a, ctas, s);
  return c.d == 128 ? launch<SLA_CACHE_INT8, 128>(c, a, ctas, s) : launch<SLA_CACHE_INT8, 64>(c, a, ctas, s);
}

}  // namespace sla
