// What the two attention kernels over the 8-bit cache share: a step's arguments, the line of
// tiles that the CTAs cut into runs, and a few instructions.
#pragma once
#include <cuda.h>

#include "cache.cuh"
#include "tc.cuh"

namespace sla {
namespace attend {

// P is 2^(score - maximum + kShift) in fp16
constexpr float kShift = 15.f;

// The unnormalised output is held times 2^-kOutShift in fp32: values are up to 2^120, a sequence
// has up to 2^18 tokens, and the kernel for many rows lets a weight be up to 2^7, so the sum is
// below 2^128 with 2^-18 and would not be without. At the other end an addition is off by 2^-150
// at most, which is 2^-132 of output, below bf16's least normal number by 2^6.
constexpr int kOutShift = 18;
// what such a sum is divided by: the row's sum of weights, l
__device__ __forceinline__ float out_divisor(float l) { return l * exp2_int(-kOutShift); }

struct Step {
  const __nv_bfloat16* q;
  const int32_t *lens, *n_new, *sel;
  __nv_bfloat16* out;
  float* part_ml;   // [slots][2][rows of a group]: m, l of a partial
  float* part_o;    // [slots][rows of a group][D], times 2^-kOutShift
  float* lse;       // [B, H, T] log2-sum-exp (with weights)
  float* scores;    // [tiles of all (sequence, KV head)][64][score_rows] (with weights)
  int T, top_n, window, rows, groups;  // rows = T * group of a KV head, in groups of group_rows
  int group_rows;
  unsigned round;                      // tiles that a CTA works on at once
  int score_rows;                      // rows rounded up to 8
};

// ---------------------------------------------------------------------------
// the line of tiles
// ---------------------------------------------------------------------------
// Tiles of one (sequence, KV head): the list's valid entries first, as many as there can be in
// a list of top_n and a sequence of L, then the window's (or all) blocks.
__device__ __forceinline__ int listed_tiles(const Step& a, int L) { return min(a.top_n, (L + kBlock - 1) / kBlock); }
__device__ __forceinline__ int first_block(const Step& a, int L, int n) {
  return a.window > 0 ? max(0, L - n - a.window + 1) / kBlock : 0;
}
__device__ __forceinline__ int tile_count(const Step& a, int L, int n) {
  if (n == 0 || L == 0) return 0;
  const int range = (L + kBlock - 1) / kBlock - first_block(a, L, n);
  return a.sel == nullptr ? range : listed_tiles(a, L) + (a.window > 0 ? range : 0);
}

struct Lines {  // in shared memory
  int* cum;     // [B + 1]: tiles of one KV head of the sequences before
  int* len;     // [B]
  uint8_t* fresh;  // [B]: valid query rows of a head
};
__host__ __device__ inline size_t lines_bytes(int B) { return align_up((size_t)(2 * B + 1) * 4 + B, 16); }

// All threads of the block; ends with a barrier. The lengths are read from L2: join_kernel and
// weight_kernel look at them before they wait (what wrote them was complete when the attention
// kernel let them start), and a line in L1 may be older.
static __device__ void scan_lines(const CacheView& c, const Step& a, char* smem, Lines* out, int* warp_sums) {
  Lines l;
  l.cum = reinterpret_cast<int*>(smem);
  l.len = l.cum + c.B + 1;
  l.fresh = reinterpret_cast<uint8_t*>(l.len + c.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int per = (c.B + blockDim.x - 1) / blockDim.x, b0 = tid * per;
  int mine = 0;
  for (int b = b0; b < min(c.B, b0 + per); ++b) {
    bool bad = false;
    const int L = in_range(__ldcg(a.lens + b), c.cap, &bad);
    const int n = a.n_new == nullptr ? a.T : in_range(__ldcg(a.n_new + b), a.T, &bad);
    if (bad && blockIdx.x == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
    l.len[b] = L;
    l.fresh[b] = (uint8_t)n;
    const int t = tile_count(a, L, n);
    l.cum[b] = t;
    mine += t;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < nw; ++w)
    if (w < warp) before += warp_sums[w];
  for (int b = b0; b < min(c.B, b0 + per); ++b) {
    const int t = l.cum[b];
    l.cum[b] = before;
    before += t;
  }
  if (b0 < c.B && b0 + per >= c.B) l.cum[c.B] = before;
  __syncthreads();
  *out = l;
}

// Tiles a CTA's run has. Whole rounds leave fewer parts to join; where segments (segs of them)
// are shorter than a round, it counts as no longer than they are on average: a CTA's segments
// come one after another, and 432 of one tile each would else keep 108 of 296 CTAs busy.
__device__ __forceinline__ unsigned run_length(const Step& a, unsigned total, unsigned segs, unsigned ctas) {
  const unsigned unit = max(1u, min(a.round, total / segs));
  return unit * ((total + ctas * unit - 1) / (ctas * unit));
}

// Sequence that holds tile t of the line (per: segments a KV-head line of a sequence has).
__device__ __forceinline__ int find_sequence(const Lines& l, int B, unsigned t, unsigned per) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((unsigned)l.cum[mid] * per <= t) lo = mid;
    else hi = mid - 1;
  }
  // sequences without tiles share their number with the next: the last of them was found
  return lo;
}

// The entries of (b, hk)'s list that count, lane and lane + 32, -1 for the others: those above
// every earlier one and inside the sequence. Called by a whole warp, which reports the rest.
__device__ __forceinline__ void valid_entries(const CacheView& c, const Step& a, int b, int hk, int L, int lane, int& e0,
                                              int& e1) {
  const int32_t* list = a.sel + ((size_t)b * c.H_kv + hk) * a.top_n;
  e0 = lane < a.top_n ? list[lane] : -1;
  e1 = lane + 32 < a.top_n ? list[lane + 32] : -1;
  int p0 = e0, p1 = e1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, p0, o), y1 = __shfl_up_sync(0xffffffffu, p1, o);
    if (lane >= o) {
      p0 = max(p0, y0);
      p1 = max(p1, y1);
    }
  }
  const int all0 = __shfl_sync(0xffffffffu, p0, 31);
  int before0 = __shfl_up_sync(0xffffffffu, p0, 1), before1 = __shfl_up_sync(0xffffffffu, p1, 1);
  if (lane == 0) before0 = before1 = -1;
  before1 = max(before1, all0);
  const int blocks = (L + kBlock - 1) / kBlock;
  const bool bad0 = e0 >= 0 && (e0 <= before0 || e0 >= blocks), bad1 = e1 >= 0 && (e1 <= before1 || e1 >= blocks);
  if (bad0 || bad1) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheSel);
  if (bad0 || e0 < 0) e0 = -1;
  if (bad1 || e1 < 0) e1 = -1;
}

// Block of tile idx of a sequence whose list's valid entries the warp holds; -1 where it is
// none. *chosen: the window does not limit it.
__device__ __forceinline__ int listed_block(const Step& a, int idx, int L, int first, int lane, int e0, int e1,
                                            bool* chosen) {
  const int listed = listed_tiles(a, L);
  *chosen = idx < listed;
  if (idx < listed) {  // the valid entry that idx of them are before
    const uint32_t m0 = __ballot_sync(0xffffffffu, e0 >= 0), m1 = __ballot_sync(0xffffffffu, e1 >= 0);
    const bool late = idx >= __popc(m0);
    const int e = late ? e1 : e0;
    const int before = late ? __popc(m0) + __popc(m1 & ((1u << lane) - 1)) : __popc(m0 & ((1u << lane) - 1));
    const uint32_t hit = __ballot_sync(0xffffffffu, e >= 0 && before == idx);
    return hit == 0 ? -1 : __shfl_sync(0xffffffffu, e, __ffs(hit) - 1);
  }
  const int j = first + idx - listed;
  return __any_sync(0xffffffffu, e0 == j || e1 == j) ? -1 : j;
}

// The same for a tile by itself.
__device__ __forceinline__ int tile_block(const CacheView& c, const Step& a, int b, int hk, int idx, int L, int n,
                                          int lane, bool* chosen) {
  const int first = first_block(a, L, n);
  if (a.sel == nullptr) {
    *chosen = a.window == 0;
    return first + idx;
  }
  int e0, e1;
  valid_entries(c, a, b, hk, L, lane, e0, e1);
  return listed_block(a, idx, L, first, lane, e0, e1, chosen);
}

// A segment of the line: one row group of one KV head of one sequence, with its tiles.
struct Segment {
  int b, sr;         // sequence, number in it
  unsigned lo, nb;   // first tile of the line, tiles
};
__device__ __forceinline__ void next_segment(Segment& s, const Lines& l, unsigned per) {
  s.lo += s.nb;
  if (++s.sr == (int)per) {
    s.sr = 0;
    do ++s.b;
    while (l.cum[s.b + 1] == l.cum[s.b]);  // there is a tile ahead, so there is such a sequence
    s.nb = l.cum[s.b + 1] - l.cum[s.b];
  }
}

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row)
      : "memory");
}
// What a query row of largest magnitude `top`, exponent ex, is multiplied by for fp16. NaN where
// it holds an infinity: the row's scores are to be NaN, and minus infinity means masked.
__device__ __forceinline__ float row_factor(float top, int ex) {
  return top < INFINITY ? exp2_int(14 - ex) : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ float log2_sum(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }


}  // namespace attend

// The kernel for many query rows (cache_attend_tc.cu): groups of 128 rows on `ctas` CTAs that
// take at least one tile each.
constexpr int kTcGroupRows = 128;
cudaError_t launch_attend_tc(const CacheView& c, const attend::Step& a, int ctas, cudaStream_t s);

}  // namespace sla
