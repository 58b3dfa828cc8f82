// sla_cache_attend: softmax attention of a step's queries over the paged 8-bit cache.
//
// A step has few query rows (T * H / H_kv of a KV head) and a long cache, so each cached
// key and value is wanted once, by all rows at a time, and the work is spread along the
// cache. The unit is a tile: one page of one KV head, for up to 16 query rows. All tiles of
// all sequences and heads, one (sequence, head, row group) segment after the other, form one
// line that the CTAs cut into equal runs, so a batch of ragged lengths loads every SM alike
// and one long sequence uses the whole device. The cut depends on the lengths, which only
// the device knows: every CTA scans them first. A CTA takes its run with four warps, each
// of them every fourth tile with its own ring of TMA-loaded pages; at the end of a segment
// the warps' (max, sum, output) are merged through shared memory and either written out
// (the CTA had the whole segment) or left as a partial that join_kernel adds up.
//
// A warp's tile, by mma.sync m16n8k16 on fp16 (codes are fp16 numbers exactly), with the
// cache as the 16-row operand and the query rows as the 8 columns, so that up to 8 rows cost
// half of what 16 do:
//   S^T[64 slots x rows] = K Q^T; the scales of page, row and softmax in fp32;
//   m' = max(m, colmax S^T), P = 2^(S - m' + 15) as fp16, l = l 2^(m - m') + 2^-15 sum P;
//   O^T[d x rows] = O^T 2^(m - m') + 2^-15 v_scale * (V^T P^T), held times 2^-18 (kOutShift).
// The 15 keeps P's smallest terms out of fp16's subnormals: a weight of 2^-29 still has 11
// bits. Q is scaled by a power of two a row so that its largest element is in [2^14, 2^15):
// bf16 elements down to 2^-28 of it are then fp16 numbers exactly.
// K Q^T runs over a permuted d (a lane's 16-byte loads of a key row are its k indices of
// consecutive steps) with Q permuted alike. V^T comes from ldmatrix's transpose of bytes,
// which hands slots out in another order; the rows of S^T take their keys in that order, and
// movmatrix turns P's 8 x 8 pieces into the second product's operand.
//
// What bounds it. A large batch: HBM (64 sequences of up to 16384 tokens, 8 KV heads, 4 rows
// each: 189 us on the device for 1.25 GB, 6.6 TB/s, the measured copy rate; with the
// rows as the 16-row operand, 4 rows padded to 16, it was 240). A few sequences: latency. A
// warp's tile takes some 4000 cycles (products 1300 and 1500, softmax 1000, read from the clock in
// an instrumented copy), and 296 CTAs leave it three or four tiles behind a start of 3 us
// (lengths, table, page): 65536 tokens of one sequence, 16 rows, 20 us. More than 16 rows read a
// page once a group of 16, from L2: 128 rows were bound by that (5.9 TB/s of L2 reads), hence
// the other kernel. Twelve warps an SM instead of eight, at 168 registers, were 12 % slower. The
// lengths of more than 650 sequences leave room for one CTA an SM instead of two (9 to 16 rows,
// d 128): the second half of the CTAs then comes in a second wave.
#include <cuda.h>

#include <algorithm>

#include "cache_attend.cuh"

namespace sla {
namespace {

using namespace attend;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlots = 2;       // pages in a warp's ring: keys and values of a tile
constexpr int kCtasPerSm = 2;
// More rows of a KV head go to the tcgen05 kernel, whose time hardly depends on their number: 8
// sequences of up to 16001 tokens, 4 KV heads, took this kernel 42, 53, 63 and 88 us at 32, 48,
// 64 and 96 rows, the other 68 to 70 us; 65536 tokens of one sequence 52 and 59 us at 64.
constexpr int kFewRows = 64;

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two 16 x 16 byte matrices, transposed: lane (g = lane / 4, q = lane % 4) gets in r[2 i]
// rows 4 q .. 4 q + 3 of column g of matrix i and in r[2 i + 1] of column g + 8. Lanes
// 0 - 15 give the row addresses of matrix 0, the others of matrix 1.
__device__ __forceinline__ void ldmatrix_trans_b8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// ---------------------------------------------------------------------------
// a warp's ring
// ---------------------------------------------------------------------------
// All of it is the same in every lane.
struct Tile {
  int seg, block;  // segment of the line, block of the sequence
  int tile;        // number of the tile among those of all (sequence, KV head)
  bool chosen;     // the window does not limit it
};

template <int D>
struct Ring {
  static constexpr int kPage = kBlock * D;  // bytes of a page of one head
  uint32_t data, bars;                      // shared addresses: kSlots pages, kSlots barriers
  unsigned issued, used;                    // pages requested and released (K and V of a tile in turn)
  unsigned next, end;                       // tiles of the line not yet looked at
  // where tile `next` is: its sequence, KV head, segment, number in it, the segment's tiles
  int b, hk, seg, idx, nb;
  int2* list;   // shared, a lane's pair: the valid list entries of (sequence, KV head) number list_of
  int list_of;
  int vrow;  // first row of the values requested next
  // the tile whose pages are requested, and the one after it, whose table entry is being loaded
  Tile req, ahead;
  int ahead_page, ahead_hk;
  float req_ks, req_vs;
  bool has_req, has_ahead;
};

// Places the ring's `next` in its segment.
template <int D>
__device__ __forceinline__ void locate(Ring<D>& r, const CacheView& c, const Step& a, const Lines& l) {
  const unsigned per = c.H_kv * a.groups;
  while ((unsigned)l.cum[r.b + 1] * per <= r.next) ++r.b;
  r.nb = l.cum[r.b + 1] - l.cum[r.b];
  const unsigned in = r.next - (unsigned)l.cum[r.b] * per, sr = in / (unsigned)r.nb;
  r.hk = a.groups == 1 ? (int)sr : (int)sr / a.groups;
  r.idx = (int)(in - sr * r.nb);
  r.seg = r.b * (int)per + (int)sr;
}

template <int D>
__device__ __forceinline__ void request(Ring<D>& r, const CUtensorMap* map, int row, int lane) {
  const uint32_t slot = r.issued % kSlots;
  if (lane == 0) {
    tc::mbar_expect_tx(r.bars + 8 * slot, Ring<D>::kPage);
    tma_load_rows(r.data + slot * Ring<D>::kPage, map, r.bars + 8 * slot, row);
  }
  ++r.issued;
}

// Finds the run's next tile that names a block and starts to load its table entry.
template <int D>
__device__ __forceinline__ void look_ahead(Ring<D>& r, const CacheView& c, const Step& a, const Lines& l, int lane) {
  r.has_ahead = false;
  while (r.next < r.end && !r.has_ahead) {
    if (r.idx >= r.nb) locate(r, c, a, l);
    const int first = first_block(a, l.len[r.b], l.fresh[r.b]);
    bool chosen = a.window == 0;
    int j = first + r.idx;
    if (a.sel != nullptr) {
      if (r.list_of != r.b * c.H_kv + r.hk) {
        r.list_of = r.b * c.H_kv + r.hk;
        int2 e;
        valid_entries(c, a, r.b, r.hk, l.len[r.b], lane, e.x, e.y);
        r.list[lane] = e;
      }
      const int2 e = r.list[lane];
      j = listed_block(a, r.idx, l.len[r.b], first, lane, e.x, e.y, &chosen);
    }
    if (j >= 0) {
      r.ahead.seg = r.seg;
      r.ahead.block = j;
      r.ahead.tile = l.cum[r.b] * c.H_kv + r.hk * r.nb + r.idx;
      r.ahead.chosen = chosen;
      r.ahead_hk = r.hk;
      r.ahead_page = c.table[(size_t)r.b * c.max_blocks + j];
      r.has_ahead = true;
    }
    r.next += kWarps;
    r.idx += kWarps;
  }
}

// Requests the keys of the tile ahead, if there is one, and looks for the one after it.
template <int D>
__device__ __forceinline__ void request_keys(Ring<D>& r, const CacheView& c, const Step& a, const Lines& l,
                                             const CUtensorMap* kmap, int lane) {
  r.has_req = false;
  while (r.has_ahead) {
    const int page = r.ahead_page;
    if (page >= 0 && page < c.n_pages) {
      const int ph = page * c.H_kv + r.ahead_hk;
      request(r, kmap, ph * kBlock, lane);
      r.vrow = ph * kBlock;
      r.req = r.ahead;
      r.req_ks = c.k_scale[ph];
      r.req_vs = c.v_scale[ph];
      r.has_req = true;
      look_ahead(r, c, a, l, lane);
      return;
    }
    if (lane == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCachePage);
    look_ahead(r, c, a, l, lane);
  }
}

// Waits for the ring's oldest page as a warp. Where the wait runs out the ring requests nothing
// more: a barrier whose copy has not landed takes no second one, and the run ends.
template <int D>
__device__ __forceinline__ bool wait_page(Ring<D>& r, volatile int* abort) {
  const uint32_t slot = r.used % kSlots;
  if (__all_sync(0xffffffffu, tc::mbar_wait(r.bars + 8 * slot, (r.used / kSlots) & 1, abort))) return true;
  r.next = r.end;
  r.has_ahead = r.has_req = false;
  return false;
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
template <int D, int NR>
struct Smem {
  static constexpr int kPitch = D + 4;  // words of a merged row: lanes of a store hit all banks
  static constexpr int kRing = kWarps * kSlots * kBlock * D;
  static constexpr int kMerge = kWarps * 8 * NR * kPitch * 4;  // the warps' outputs
  static constexpr int kQ = 8 * NR * D * 2;                    // Q's fragments; the next segment's rows
  static constexpr int off_merge = kRing, off_q = off_merge + kMerge, off_next_q = off_q + kQ, off_misc = off_next_q + kQ;
  static constexpr int kMisc = 2304;
  static constexpr int off_lines = off_misc + kMisc;
  static size_t bytes(int B) { return off_lines + lines_bytes(B); }
};

// NR: query rows of a segment in eights.
template <int KIND, int D, int NR>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const CacheView c,
                  const Step a) {
  constexpr int KS = D / 16;  // k steps of K Q^T; words of codes a lane holds of a key row
  constexpr int MT = D / 16;  // row tiles of O^T
  constexpr int kRows = 8 * NR;
  using Sm = Smem<D, NR>;
  extern __shared__ __align__(1024) char smem[];  // TMA's swizzle goes by address bits
  struct Misc {
    uint64_t bars[kWarps][kSlots];
    float m[kWarps][kRows], l[kWarps][kRows];
    int2 list[kWarps][32];
    float qs[kRows];  // what a row's scores are multiplied by
    float top[kRows], all[kRows];  // the segment's
    int warp_sums[kWarps];
    int abort, never;
  };
  static_assert(sizeof(Misc) <= Sm::kMisc, "misc");
  Misc& mi = *reinterpret_cast<Misc*>(smem + Sm::off_misc);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;

  if (tid == 0) {
    mi.abort = mi.never = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kSlots; ++i) tc::mbar_init(smem_u32(&mi.bars[w][i]), 1);
    tc::fence_mbar_init();
    tc::prefetch_tensormap(&kmap);
    tc::prefetch_tensormap(&vmap);
  }
  Lines l;
  wait_for_previous();
  scan_lines(c, a, smem + Sm::off_lines, &l, mi.warp_sums);
  let_next_start();

  // this CTA's run of the line
  const unsigned per = c.H_kv * a.groups, total = (unsigned)l.cum[c.B] * per;
  const unsigned run = run_length(a, total, c.B * per, gridDim.x);
  const unsigned lo = min(total, blockIdx.x * run), hi = min(total, lo + run);
  if (lo >= hi) return;

  Ring<D> ring;
  ring.data = smem_u32(smem) + warp * kSlots * Ring<D>::kPage;
  ring.bars = smem_u32(&mi.bars[warp][0]);
  ring.issued = ring.used = 0;
  ring.next = lo + warp;
  ring.end = hi;
  Segment sg;
  sg.b = find_sequence(l, c.B, lo, per);
  sg.nb = l.cum[sg.b + 1] - l.cum[sg.b];
  sg.sr = (int)((lo - (unsigned)l.cum[sg.b] * per) / sg.nb);
  sg.lo = (unsigned)l.cum[sg.b] * per + sg.sr * sg.nb;
  // rows of Q, eight by a warp: lane (g, q4) copies row g's elements q4 * D / 4 .. for itself
  const uint32_t my_q = smem_u32(smem + Sm::off_next_q) + (warp * 32 + lane) * (D / 2);
  auto fetch_q = [&](const Segment& s) {
    const int hk = a.groups == 1 ? s.sr : s.sr / a.groups, grp = s.sr - hk * a.groups;
    const int r = grp * kRows + 8 * warp + g;
    if (warp < NR && r < a.rows) {
      const __nv_bfloat16* p = a.q + (((size_t)s.b * c.H + (size_t)hk * c.group) * a.T + r) * D + q4 * (D / 4);
#pragma unroll
      for (int u = 0; u < D / 32; ++u) cp_async16(my_q + 16 * u, p + 8 * u, 16);
    }
    cp_async_commit();
  };
  fetch_q(sg);
  ring.b = sg.b;
  ring.idx = ring.nb = 0;  // locate it first
  ring.list = mi.list[warp];
  ring.list_of = -1;
  // the first tile's keys and values
  look_ahead(ring, c, a, l, lane);
  request_keys(ring, c, a, l, &kmap, lane);
  if (ring.has_req) request(ring, &vmap, ring.vrow, lane);

  float* merge = reinterpret_cast<float*>(smem + Sm::off_merge);
  bool dead = false;
  while (sg.lo < hi) {
    const int L = l.len[sg.b], n = l.fresh[sg.b], seg = sg.b * (int)per + sg.sr;
    const int hk = a.groups == 1 ? sg.sr : sg.sr / a.groups, row0 = (sg.sr - hk * a.groups) * kRows;
    const unsigned seg_lo = sg.lo, seg_hi = sg.lo + sg.nb;
    const size_t qrow0 = ((size_t)sg.b * c.H + (size_t)hk * c.group) * a.T;

    // Q^T's columns go where the product's lanes find them
    uint2* qf = reinterpret_cast<uint2*>(smem + Sm::off_q);  // [NR][KS][32]
    cp_async_wait<0>();
    if (warp < NR) {
      const bool there = row0 + 8 * warp + g < a.rows;
      float x[D / 4], top = 0.f;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        const uint4 w = lds128(my_q + 16 * u);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16(there ? ws[e] : 0u);
          x[8 * u + 2 * e] = f.x;
          x[8 * u + 2 * e + 1] = f.y;
          top = tc::fmax3(top, fabsf(f.x), fabsf(f.y));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max((int)(__float_as_uint(top) >> 23) - 127, -100);
      const float up = row_factor(top, ex);
      if (q4 == 0) mi.qs[8 * warp + g] = exp2_int(ex - 14) * (c.scale * 1.4426950408889634f);
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qf[(warp * KS + s) * 32 + lane] =
            make_uint2(pack_f16(x[4 * s] * up, x[4 * s + 1] * up), pack_f16(x[4 * s + 2] * up, x[4 * s + 3] * up));
    }
    __syncthreads();
    if (seg_hi < hi) {
      next_segment(sg, l, per);
      fetch_q(sg);
    } else {
      sg.lo = hi;
    }
    float qs[NR][2];  // of the rows whose scores this lane gets: 8 i + 2 q4 + e
    int pos[NR][2];   // the slots such a row sees end here
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * i + 2 * q4 + e, rc = row0 + col, t = a.T == 1 ? 0 : rc % a.T;
        qs[i][e] = mi.qs[col];
        pos[i][e] = rc < a.rows && t < n ? L - n + t : -1;
      }

    float o[MT][NR][4], m[NR][2], sum[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      sum[i][0] = sum[i][1] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }

    while (ring.has_req && ring.req.seg == seg) {
      const Tile cur = ring.req;
      const int j0 = cur.block * kBlock;
      const bool chosen = cur.chosen;
      const float ks = ring.req_ks, vs = ring.req_vs * exp2_int(-(int)kShift - kOutShift);
      const uint32_t kbase = ring.data + ring.used % kSlots * Ring<D>::kPage;
      if (!wait_page(ring, &mi.abort)) {
        dead = true;
        break;
      }

      // scores: row g (+ 8) of tile t is slot 16 t + 4 (g / 2) + g % 2 (+ 2)
      float s[4][NR][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < NR; ++i) s[t][i][0] = s[t][i][1] = s[t][i][2] = s[t][i][3] = 0.f;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        uint2 qk[NR][4];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) qk[i][k] = qf[(i * KS + 4 * u + k) * 32 + lane];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = 16 * t + 4 * (g >> 1) + (g & 1);
          uint4 x, y;
          if (D == 128) {
            x = lds128(kbase + row * 128 + (((2 * q4 + u) ^ (row & 7)) << 4));
            y = lds128(kbase + (row + 2) * 128 + (((2 * q4 + u) ^ ((row + 2) & 7)) << 4));
          } else {
            x = lds128(kbase + row * 64 + ((q4 ^ ((row >> 1) & 3)) << 4));
            y = lds128(kbase + (row + 2) * 64 + ((q4 ^ (((row + 2) >> 1) & 3)) << 4));
          }
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[4];
            decode4_f16<KIND>(xs[k], f[0], f[2]);
            decode4_f16<KIND>(ys[k], f[1], f[3]);
#pragma unroll
            for (int i = 0; i < NR; ++i) mma_f16(s[t][i], f, qk[i][k].x, qk[i][k].y);
          }
        }
      }
      ++ring.used;
      __syncwarp();  // every lane has finished with the keys
      request_keys(ring, c, a, l, &kmap, lane);

      // rows that do not see the whole page: its end, the window's start
      if (j0 + kBlock - 1 > L - n || (!chosen && j0 <= L - 1 - a.window)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int slot = j0 + 16 * t + 4 * (g >> 1) + (g & 1) + (e & 2), p = pos[i][e & 1];
              if (slot > p || (!chosen && slot <= p - a.window)) s[t][i][e] = -INFINITY;
            }
      }
      uint32_t pf[4][NR][2];  // P^T as the second operand of V^T P^T
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        // the scale stays positive (a product that underflows would turn a masked score into NaN)
        const float f[2] = {fmaxf(qs[i][0] * ks, 1e-37f), fmaxf(qs[i][1] * ks, 1e-37f)};
        // x = (s - tile's maximum) * f + (its scaled value - m') + shift: the largest exponent is
        // the shift exactly, however large the scores
        float low[2], off[2], alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[0][i][e], s[0][i][e + 2]);
#pragma unroll
          for (int t = 1; t < 4; ++t) top = tc::fmax3(top, s[t][i][e], s[t][i][e + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          low[e] = top == -INFINITY ? 0.f : top;
          const float scaled = __fmul_rn(top, f[e]), next = fmaxf(m[i][e], scaled);
          const float base = next == -INFINITY ? 0.f : next;
          off[e] = (scaled == -INFINITY ? 0.f : scaled - base) + kShift;
          alpha[e] = tc::ex2_approx(m[i][e] - base);
          m[i][e] = next;
          sum[i][e] *= alpha[e];
        }
        if (a.scores != nullptr && row0 + 8 * i + 2 * q4 < a.score_rows) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int slot = 16 * t + 4 * (g >> 1) + (g & 1) + 2 * h;
              *reinterpret_cast<float2*>(a.scores + ((size_t)cur.tile * kBlock + slot) * a.score_rows + row0 + 8 * i + 2 * q4) =
                  make_float2(s[t][i][2 * h] * f[0], s[t][i][2 * h + 1] * f[1]);
            }
        }
        const uint64_t f2 = tc::f2_pack(f[0], f[1]), l2 = tc::f2_pack(low[0], low[1]), o2 = tc::f2_pack(off[0], off[1]);
        uint64_t s2 = tc::f2_pack(sum[i][0], sum[i][1]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float p[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t x = tc::ffma2(tc::fsub2(tc::f2_pack(s[t][i][2 * h], s[t][i][2 * h + 1]), l2), f2, o2);
            p[2 * h] = tc::ex2_approx(tc::f2_lo(x));
            p[2 * h + 1] = tc::ex2_approx(tc::f2_hi(x));
            s2 = tc::fadd2(s2, tc::f2_pack(p[2 * h], p[2 * h + 1]));
          }
          pf[t][i][0] = transpose_8x8(pack_f16(p[0], p[1]));
          pf[t][i][1] = transpose_8x8(pack_f16(p[2], p[3]));
        }
        sum[i][0] = tc::f2_lo(s2);
        sum[i][1] = tc::f2_hi(s2);
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[t][i][0] *= alpha[0];
            o[t][i][1] *= alpha[1];
            o[t][i][2] *= alpha[0];
            o[t][i][3] *= alpha[1];
          }
        }
      }

      const uint64_t vs2 = tc::f2_pack(vs, vs);
      const uint32_t vbase = ring.data + ring.used % kSlots * Ring<D>::kPage;
      if (!wait_page(ring, &mi.abort)) {
        dead = true;
        break;
      }
      if (j0 + kBlock > L) {  // codes of slots behind the last token are whatever they are: they count as 0
        for (int e = (L - j0) * (D / 16) + lane; e < kBlock * (D / 16); e += 32) sts128(vbase + e * 16, 0u);
        __syncwarp();
      }
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        float acc[2][NR][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < NR; ++i) acc[h][i][0] = acc[h][i][1] = acc[h][i][2] = acc[h][i][3] = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = 16 * t + (lane & 15), ch = 2 * cc + (lane >> 4);
          uint32_t w[4];
          ldmatrix_trans_b8(w, vbase + row * D + ((ch ^ (D == 128 ? (row & 7) : ((row >> 1) & 3))) << 4));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t f[4];
            decode4_f16<KIND>(w[2 * h], f[0], f[2]);
            decode4_f16<KIND>(w[2 * h + 1], f[1], f[3]);
#pragma unroll
            for (int i = 0; i < NR; ++i) mma_f16(acc[h][i], f, pf[t][i][0], pf[t][i][1]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              float(&y)[4] = o[2 * cc + h][i];
              const uint64_t z = tc::ffma2(vs2, tc::f2_pack(acc[h][i][e], acc[h][i][e + 1]), tc::f2_pack(y[e], y[e + 1]));
              y[e] = tc::f2_lo(z);
              y[e + 1] = tc::f2_hi(z);
            }
      }
      ++ring.used;
      if (j0 + kBlock > L) tc::fence_async_smem();  // the zeros come before the page that is loaded next
      __syncwarp();
      if (ring.has_req) request(ring, &vmap, ring.vrow, lane);
    }

    // the warps' parts of the segment become one
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = sum[i][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          mi.m[warp][8 * i + 2 * q4 + e] = m[i][e];
          mi.l[warp][8 * i + 2 * q4 + e] = x * exp2_int(-(int)kShift);
        }
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * i + 2 * q4 + e;
        float top = mi.m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, mi.m[w][r]);
        const float f = tc::ex2_approx(m[i][e] - (top == -INFINITY ? 0.f : top));
        float* p = merge + (warp * kRows + r) * Sm::kPitch + g;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          p[16 * t] = o[t][i][e] * f;
          p[16 * t + 8] = o[t][i][e + 2] * f;
        }
        if (warp == kWarps - 1 && g == 0) {
          float all = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) all += mi.l[w][r] * tc::ex2_approx(mi.m[w][r] - (top == -INFINITY ? 0.f : top));
          mi.top[r] = top;
          mi.all[r] = all;
        }
      }
    __syncthreads();
    const bool whole = seg_lo >= lo && seg_hi <= hi;
    const size_t part = (size_t)blockIdx.x + seg;
    for (int e = tid; e < kRows * D / 4; e += kThreads) {
      const int r = e / (D / 4), d4 = e % (D / 4);
      float4 y = *reinterpret_cast<const float4*>(merge + r * Sm::kPitch + 4 * d4);
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * kRows + r) * Sm::kPitch + 4 * d4);
        y.x += x.x;
        y.y += x.y;
        y.z += x.z;
        y.w += x.w;
      }
      const float top = mi.top[r], all = mi.all[r];
      if (d4 == 0 && (!whole || a.scores != nullptr)) {
        a.part_ml[part * 2 * kRows + r] = top;
        a.part_ml[part * 2 * kRows + kRows + r] = all;
      }
      if (!whole) {
        reinterpret_cast<float4*>(a.part_o)[part * (kRows * D / 4) + e] = y;
      } else if (row0 + r < a.rows) {
        const bool empty = all == 0.f || (row0 + r) % a.T >= n;
        const float inv = 1.f / out_divisor(all);
        *reinterpret_cast<uint2*>(a.out + (qrow0 + row0 + r) * D + 4 * d4) =
            empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
        if (d4 == 0 && a.lse != nullptr) a.lse[qrow0 + row0 + r] = log2_sum(top, all);
      }
    }
    // what is written here is written again behind the next segment's first barrier
  }
  if (dead) {
    mi.abort = 1;
    if (lane == 0) report(c.status, SLA_ERR_DEVICE_TIMEOUT, kDetailTimeout);
    // copies still on their way land before the block's memory is given back
    for (unsigned i = ring.issued > kSlots ? ring.issued - kSlots : 0; i < ring.issued; ++i)
      tc::mbar_wait(ring.bars + 8 * (i % kSlots), (i / kSlots) & 1, &mi.never);
  }
}

// ---------------------------------------------------------------------------
// weights: weight[b, hk, s] += sum over rows of 2^(score - lse), rows in order
// ---------------------------------------------------------------------------
// A CTA of `ctas` takes an equal run of the tiles, which are few: a CTA's warps wait for one
// another's loads of scores (a slot's rows are a line), yet share the parts of their rows. A
// warp a tile (list entries that name no block are passed over), a lane two slots. lse: this
// warp's place for the log2-sum-exp of the tile's rows, put together from the parts of its
// segments (run: tiles of a part), or taken from a.lse where run is 0; infinite for rows that
// add nothing. Bound by the chain of loads (8 sequences of up to 8191 tokens, 4 KV heads, 16
// rows: 5 to 8 us beside the join): what can start before the rows' sums does.
__device__ void weigh(const CacheView& c, const Step& a, const Lines& l, unsigned cta, unsigned ctas, unsigned warp,
                      unsigned warps, int lane, float* lse, unsigned run) {
  const unsigned per = c.H_kv, total = (unsigned)l.cum[c.B] * per;
  int have = -1;  // (sequence, KV head) whose rows lse holds
  const unsigned mine = (total + ctas - 1) / ctas, end = min(total, (cta + 1) * mine);
  for (unsigned t = cta * mine + warp; t < end; t += warps) {
    const int b = find_sequence(l, c.B, t, per), nb = l.cum[b + 1] - l.cum[b], L = l.len[b], n = l.fresh[b];
    const unsigned in = t - (unsigned)l.cum[b] * per;
    const int hk = (int)(in / (unsigned)nb);
    bool chosen;
    const int j = tile_block(c, a, b, hk, (int)(in - (unsigned)hk * nb), L, n, lane, &chosen);
    if (j < 0) continue;
    const int page = c.table[(size_t)b * c.max_blocks + j];
    float* w = c.weight + ((size_t)b * c.H_kv + hk) * c.cap + j * kBlock + lane;
    const bool live0 = j * kBlock + lane < L, live1 = j * kBlock + lane + 32 < L;
    const float w0 = live0 ? w[0] : 0.f, w1 = live1 ? w[32] : 0.f;
    if (have != b * c.H_kv + hk) {
      have = b * c.H_kv + hk;
      __syncwarp();
      for (int r = lane; r < a.score_rows; r += 32) {
        float z = -INFINITY;
        if (r < a.rows && r % a.T < n) {
          if (run == 0) {
            z = a.lse[((size_t)b * c.H + (size_t)hk * c.group) * a.T + r];
          } else {
            const int grp = r / a.group_rows, seg = have * a.groups + grp, at = r - grp * a.group_rows;
            const unsigned lo = (unsigned)l.cum[b] * per * a.groups + (unsigned)(hk * a.groups + grp) * nb;
            float m = -INFINITY, sum = 0.f;
#pragma unroll 4
            for (unsigned i = lo / run; i <= (lo + nb - 1) / run; ++i) {
              const float* ml = a.part_ml + ((size_t)i + seg) * 2 * a.group_rows + at;
              const float x = ml[0], y = ml[a.group_rows], next = fmaxf(m, x), base = next == -INFINITY ? 0.f : next;
              sum = sum * tc::ex2_approx(m - base) + y * tc::ex2_approx(x - base);
              m = next;
            }
            z = log2_sum(m, sum);
          }
        }
        lse[r] = z > -INFINITY ? z : INFINITY;  // neither a row that sees nothing nor one that is NaN
      }
      __syncwarp();
    }
    if (page < 0 || page >= c.n_pages) continue;  // reported by the attention kernel
    const float4* s = reinterpret_cast<const float4*>(a.scores + ((size_t)t * kBlock + lane) * a.score_rows);
    const int half = 32 * a.score_rows / 4;  // from slot lane to slot lane + 32
    float x = 0.f, y = 0.f;
#pragma unroll 2
    for (int r = 0; r < a.score_rows; r += 8) {
      const float4 u0 = s[r / 4], u1 = s[r / 4 + 1], v0 = s[r / 4 + half], v1 = s[r / 4 + 1 + half];
      const float us[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
      const float vs[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = lse[r + e];
        x += z < INFINITY ? tc::ex2_approx(us[e] - z) : 0.f;
        y += z < INFINITY ? tc::ex2_approx(vs[e] - z) : 0.f;
      }
    }
    if (live0) w[0] = w0 + x;
    if (live1) w[32] = w1 + y;
  }
}

// By itself: behind join_kernel, which has left lse.
__global__ void __launch_bounds__(kThreads) weight_kernel(const CacheView c, const Step a) {
  extern __shared__ __align__(1024) char smem[];
  __shared__ int warp_sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Lines l;
  scan_lines(c, a, smem, &l, warp_sums);
  wait_for_previous();
  weigh(c, a, l, blockIdx.x, gridDim.x, warp, kWarps, lane,
        reinterpret_cast<float*>(smem + lines_bytes(c.B)) + warp * a.score_rows, 0);
}

// ---------------------------------------------------------------------------
// segments that several CTAs worked on, or none
// ---------------------------------------------------------------------------
// PW warps a row take the partials in turn, a lane D / 32 columns; a CTA has 8 / PW rows. CTAs
// before the segments' add the weights, whose chain is the longer one. Launched while the attention kernel runs
// (programmatic dependent launch), so that only its loads wait. Bound by their latency: 4 to 8
// us, the longer for the 64 parts of a segment spread over the device.
constexpr int kJoinThreads = 256;

template <int D, int PW>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const CacheView c, const Step a, unsigned ctas, int segs) {
  constexpr int E = D / 32, W = kJoinThreads / 32;
  extern __shared__ __align__(1024) char smem[];
  __shared__ int warp_sums[W];
  __shared__ float s_l[W], s_o[PW > 1 ? W : 1][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part_warp = warp % PW;
  Lines l;
  scan_lines(c, a, smem, &l, warp_sums);
  const unsigned per = c.H_kv * a.groups, total = (unsigned)l.cum[c.B] * per;
  const unsigned run = run_length(a, total, c.B * per, ctas);
  const int weighing = gridDim.x - segs;
  if (blockIdx.x < weighing) {
    wait_for_previous();
    weigh(c, a, l, blockIdx.x * gridDim.y + blockIdx.y, weighing * gridDim.y, warp, W, lane,
          reinterpret_cast<float*>(smem + lines_bytes(c.B)) + warp * a.score_rows, run);
    return;
  }
  const int rows = a.group_rows, seg = blockIdx.x - weighing, b = seg / (int)per, sr = seg % (int)per, hk = sr / a.groups;
  const int r = blockIdx.y * (W / PW) + warp / PW, row = sr % a.groups * rows + r;
  const int nb = l.cum[b + 1] - l.cum[b];
  const unsigned lo = (unsigned)l.cum[b] * per + (unsigned)sr * nb, hi = lo + nb;
  const unsigned c0 = nb ? lo / run : 0, c1 = nb ? (hi - 1) / run : 0;
  const size_t qrow = ((size_t)b * c.H + (size_t)hk * c.group) * a.T + row;
  wait_for_previous();
  let_next_start();
  if (nb != 0 && c0 == c1) return;  // written by the CTA that had all of it
  const bool there = r < rows && row < a.rows;
  float m = -INFINITY, sum = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (nb != 0 && there) {
    for (unsigned i = c0 + lane; i <= c1; i += 32) m = fmaxf(m, a.part_ml[((size_t)i + seg) * 2 * rows + r]);
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float top = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (unsigned i = c0 + part_warp; i <= c1; i += PW) {
      const size_t part = (size_t)i + seg;
      const float f = tc::ex2_approx(a.part_ml[part * 2 * rows + r] - top);
      sum += a.part_ml[part * 2 * rows + rows + r] * f;
      const float* p = a.part_o + (part * rows + r) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += p[e] * f;
    }
  }
  if (PW > 1) {
    if (lane == 0) s_l[warp] = sum;
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[PW > 1 ? warp : 0][lane * E + e] = o[e];
    __syncthreads();
    if (part_warp != 0) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < PW; ++w) sum += s_l[warp + w];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < PW; ++w) o[e] += s_o[PW > 1 ? warp + w : 0][lane * E + e];
    }
  }
  if (!there) return;
  const bool valid = row % a.T < l.fresh[b] && sum != 0.f;
  const float by = out_divisor(sum);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + qrow * D + lane * E + e) = valid ? pack_bf16(o[e] / by, o[e + 1] / by) : 0u;
  if (lane == 0 && a.lse != nullptr) a.lse[qrow] = log2_sum(m, sum);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

constexpr int kMaxCtas = kCtasPerSm * 148;  // a workspace is sized for this grid, whatever device is current

struct Layout {
  size_t ml, o, lse, scores, total;
  int64_t tiles;  // at most, of all KV heads
  int rows, group_rows, groups;
};

// Most tiles that a (sequence, KV head) can have.
int most_tiles(const sla_cache_config* c, int T, int top_n, int window) {
  const int64_t range = window > 0 ? ((int64_t)window + T - 2) / kBlock + 2 : c->max_blocks;
  const int blocks = (int)(range < c->max_blocks ? range : c->max_blocks);
  return top_n > 0 ? top_n + (window > 0 ? blocks : 0) : blocks;
}

sla_status plan_step(const sla_cache_config* c, int32_t T, int32_t top_n, int32_t window, bool weights, Layout* p) {
  const sla_status st = sla_cache_validate_config(c);
  if (st != SLA_OK) return st;
  if (T < 1 || top_n < 0 || window < 0) return SLA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)T * (c->H / c->H_kv);
  if (T > kCacheMaxT || rows > kCacheMaxRows || top_n > kCacheMaxSel) return SLA_ERR_UNSUPPORTED;
  p->rows = (int)rows;
  p->group_rows = p->rows <= 8 ? 8 : p->rows <= kFewRows ? 16 : kTcGroupRows;
  p->groups = (p->rows + p->group_rows - 1) / p->group_rows;
  const int64_t segs = (int64_t)c->B * c->H_kv * p->groups;
  const int64_t tiles = p->tiles = (int64_t)c->B * c->H_kv * most_tiles(c, T, top_n, window);
  if (tiles * p->groups >= ((int64_t)1 << 31)) return SLA_ERR_UNSUPPORTED;  // the line is counted in 32 bits
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t parts = kMaxCtas + (size_t)segs;
  p->ml = take(parts * 2 * p->group_rows * 4);
  p->o = take(parts * p->group_rows * c->d * 4);
  p->lse = take(weights ? (size_t)c->B * c->H * T * 4 : 0);
  p->scores = take(weights ? (size_t)tiles * align_up(p->rows, 8) * kBlock * 4 : 0);
  p->total = off;
  return SLA_OK;
}

template <int KIND, int D, int NR>
cudaError_t launch(const CacheView& c, const Step& a, int ctas, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)c.n_pages * c.H_kv * kBlock;
  if (!make_tmap_rows_u8(&kmap, c.k, rows, D, kBlock) || !make_tmap_rows_u8(&vmap, c.v, rows, D, kBlock))
    return cudaErrorInvalidValue;
  auto attend = attend_kernel<KIND, D, NR>;
  const cudaError_t e =
      cudaFuncSetAttribute(attend, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D, NR>::bytes(kCacheMaxB));
  if (e != cudaSuccess) return e;
  return launch_overlapped(attend, dim3(ctas), kThreads, Smem<D, NR>::bytes(c.B), s, kmap, vmap, c, a);
}

template <int KIND, int D>
cudaError_t launch_rows(const CacheView& c, const Step& a, int ctas, cudaStream_t s) {
  return a.group_rows == 8 ? launch<KIND, D, 1>(c, a, ctas, s) : launch<KIND, D, 2>(c, a, ctas, s);
}

cudaError_t launch_attend(const CacheView& c, const Step& a, int ctas, cudaStream_t s) {
  if (a.group_rows == kTcGroupRows) return launch_attend_tc(c, a, ctas, s);
  if (c.kind == SLA_CACHE_E4M3)
    return c.d == 128 ? launch_rows<SLA_CACHE_E4M3, 128>(c, a, ctas, s) : launch_rows<SLA_CACHE_E4M3, 64>(c, a, ctas, s);
  return c.d == 128 ? launch_rows<SLA_CACHE_INT8, 128>(c, a, ctas, s) : launch_rows<SLA_CACHE_INT8, 64>(c, a, ctas, s);
}

template <int D>
cudaError_t launch_step(const CacheView& c, const Step& a, int sms, int64_t tiles, cudaStream_t s) {
  const int per_sm = a.group_rows == kTcGroupRows ? 1 : kCtasPerSm;
  const int ctas = per_sm * sms < kMaxCtas ? per_sm * sms : kMaxCtas;
  cudaError_t e = launch_attend(c, a, ctas, s);
  if (e != cudaSuccess) return e;
  const int segs = c.B * c.H_kv * a.groups, most = a.rows < a.group_rows ? a.rows : a.group_rows;
  const int weighing = (int)std::min<int64_t>((c.weight != nullptr ? 4 : 0) * sms, tiles);
  // A warp a row where segments are cut into few parts, eight where one is spread over the
  // device. In the first case the weights' warps can put the parts' sums together themselves and
  // run beside the join; in the second they would each read hundreds of parts.
  if (ctas > 16 * segs) {
    e = launch_overlapped(join_kernel<D, 8>, dim3(segs, most), kJoinThreads, lines_bytes(c.B), s, c, a, (unsigned)ctas, segs);
    if (e != cudaSuccess || c.weight == nullptr) return e;
    return launch_overlapped(weight_kernel, dim3(weighing), kThreads,
                            lines_bytes(c.B) + kWarps * a.score_rows * sizeof(float), s, c, a);
  }
  const int y = (most + 7) / 8, more = (weighing + y - 1) / y;
  const size_t smem = lines_bytes(c.B) + (c.weight != nullptr ? kJoinThreads / 32 * a.score_rows * sizeof(float) : 0);
  return launch_overlapped(join_kernel<D, 1>, dim3(segs + more, y), kJoinThreads, smem, s, c, a, (unsigned)ctas, segs);
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_cache_attend_workspace_bytes(const sla_cache_config* cfg, int32_t T, int32_t top_n, int32_t window,
                                        int32_t with_weight) {
  Layout p;
  return plan_step(cfg, T, top_n, window, with_weight != 0, &p) == SLA_OK ? p.total : 0;
}

sla_status sla_cache_attend(const void* q, const sla_cache_config* cfg, const sla_cache* cache, int32_t T,
                            const int32_t* lens, const int32_t* n_new, const int32_t* sel, int32_t top_n,
                            int32_t window, void* out, void* ws, size_t ws_bytes, void* stream) {
  CacheView c;
  sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  Layout p;
  st = plan_step(cfg, T, top_n, window, c.weight != nullptr, &p);
  if (st != SLA_OK) return st;
  if (!q || !lens || !out || q == out || (sel == nullptr) != (top_n == 0)) return SLA_ERR_INVALID_ARG;
  if (((uintptr_t)q % 16) || ((uintptr_t)out % 16) || ((uintptr_t)lens % 4) || ((uintptr_t)n_new % 4) ||
      ((uintptr_t)sel % 4))
    return SLA_ERR_INVALID_ARG;
  if (!ws || ((uintptr_t)ws % 256) || ws_bytes < p.total) return SLA_ERR_WORKSPACE;
  Step a;
  a.q = (const __nv_bfloat16*)q;
  a.lens = lens;
  a.n_new = n_new;
  a.sel = sel;
  a.out = (__nv_bfloat16*)out;
  a.part_ml = (float*)((char*)ws + p.ml);
  a.part_o = (float*)((char*)ws + p.o);
  a.lse = c.weight ? (float*)((char*)ws + p.lse) : nullptr;
  a.scores = c.weight ? (float*)((char*)ws + p.scores) : nullptr;
  a.T = T;
  a.top_n = top_n;
  a.window = window < c.cap + kCacheMaxT ? window : c.cap + kCacheMaxT;  // more sees no more
  a.rows = p.rows;
  a.groups = p.groups;
  a.group_rows = p.group_rows;
  a.round = p.group_rows == kTcGroupRows ? 1 : kWarps;
  a.score_rows = (int)align_up(p.rows, 8);
  const int sms = sm_count();
  if (sms < 1) return SLA_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = c.d == 128 ? launch_step<128>(c, a, sms, p.tiles, s) : launch_step<64>(c, a, sms, p.tiles, s);
  return e == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

}  // extern "C"
