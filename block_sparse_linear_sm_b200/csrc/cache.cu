// The 8-bit paged cache: argument checks, sla_cache_append and sla_cache_evict.
//
// A page holds 64 slots of one KV head after the other, codes [H_kv][64][d], so that the
// page of one head is one contiguous run of 64 * d bytes.
#include <math.h>

#include <algorithm>

#include "cache.cuh"
#include "tc.cuh"

namespace sla {

static bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Whether two arrays of B lengths share memory: lengths are written while other blocks read.
static bool lengths_overlap(const int32_t* a, const int32_t* b, int B) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b, n = (uintptr_t)B * sizeof(int32_t);
  return a && b && x < y + n && y < x + n;
}

static sla_status check_sizes(const sla_cache_config* c) {
  if (c == nullptr) return SLA_ERR_INVALID_ARG;
  if (c->B < 1 || c->H < 1 || c->H_kv < 1 || c->d < 1 || c->n_pages < 1 || c->max_blocks < 1)
    return SLA_ERR_INVALID_ARG;
  if (c->H % c->H_kv != 0) return SLA_ERR_INVALID_ARG;
  if (c->kind != SLA_CACHE_E4M3 && c->kind != SLA_CACHE_INT8) return SLA_ERR_INVALID_ARG;
  if (!(c->scale >= 0.f) || !isfinite(c->scale)) return SLA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SLA_ERR_UNSUPPORTED;
  if (c->B > kCacheMaxB || c->H > 1024 || c->max_blocks > kMaxBlocks) return SLA_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->H_kv * kBlock >= ((int64_t)1 << 31)) return SLA_ERR_UNSUPPORTED;
  return SLA_OK;
}

// Sizes and buffers that every call needs; fills *view.
sla_status check_cache(const sla_cache_config* c, const sla_cache* m, CacheView* view) {
  const sla_status st = check_sizes(c);
  if (st != SLA_OK) return st;
  if (m == nullptr || !m->k || !m->v || !m->k_scale || !m->v_scale || !m->block_table || !m->status)
    return SLA_ERR_INVALID_ARG;
  if (!aligned_to(m->k, 16) || !aligned_to(m->v, 16) || !aligned_to(m->k_scale, 4) || !aligned_to(m->v_scale, 4) ||
      !aligned_to(m->k_mean, 16) || !aligned_to(m->weight, 16) || !aligned_to(m->block_table, 4) ||
      !aligned_to(m->status, 256) || m->k == m->v)
    return SLA_ERR_INVALID_ARG;
  view->k = (uint8_t*)m->k;
  view->v = (uint8_t*)m->v;
  view->k_scale = m->k_scale;
  view->v_scale = m->v_scale;
  view->k_mean = m->k_mean;
  view->weight = m->weight;
  view->table = m->block_table;
  view->status = (int*)m->status;
  view->B = c->B;
  view->H = c->H;
  view->H_kv = c->H_kv;
  view->group = c->H / c->H_kv;
  view->d = c->d;
  view->n_pages = c->n_pages;
  view->max_blocks = c->max_blocks;
  view->cap = c->max_blocks * kBlock;
  view->kind = c->kind;
  view->scale = c->scale > 0.f ? c->scale : 1.f / sqrtf((float)c->d);
  view->scale64 = c->scale > 0.f ? (double)c->scale : 1.0 / sqrt((double)c->d);
  return SLA_OK;
}

namespace {

constexpr int kCta = 256;

// Largest of one unsigned value a thread over the block (all get it). slots: 8 words.
__device__ __forceinline__ uint32_t block_max(uint32_t a, uint32_t* slots) {
  const uint32_t w = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = w;
  __syncthreads();
  uint32_t m = slots[0];
#pragma unroll
  for (int i = 1; i < kCta / 32; ++i) m = max(m, slots[i]);
  return m;
}

// Sixteen codes of 16 values times inv.
template <int KIND>
__device__ __forceinline__ uint4 encode16(const float* x, float inv) {
  uint4 c;
  c.x = encode4<KIND>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  c.y = encode4<KIND>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
  c.z = encode4<KIND>(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv);
  c.w = encode4<KIND>(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv);
  return c;
}
// Codes at a scale `ratio` times as fine (a power of two): rounded again, exact for ratio >= 1.
template <int KIND>
__device__ __forceinline__ uint4 recode16(const uint4& c, float ratio) {
  float y[16];
  decode4<KIND>(c.x, y);
  decode4<KIND>(c.y, y + 4);
  decode4<KIND>(c.z, y + 8);
  decode4<KIND>(c.w, y + 12);
  return encode16<KIND>(y, ratio);
}

// Mean of a page's 64 rows of codes in shared memory, times the scale; all threads. Codes are
// integers times 2^-9 (e4m3) or integers (int8) of at most 19 bits, so 64 of them add up
// exactly, in any order: in fp32, or (int8, offset by 128) four at a time in 16-bit lanes.
template <int KIND, int D>
__device__ __forceinline__ void write_mean(const uint8_t* tile, float scale, float* mean, float4* parts) {
  constexpr int W = D / 4, P = kCta / W, R = kBlock / P;  // words a row, threads a word, rows a thread
  const int w = threadIdx.x % W, p = threadIdx.x / W;
  const uint32_t* word = reinterpret_cast<const uint32_t*>(tile + p * R * D) + w;
  const float f = scale * (1.f / kBlock);
  if (KIND == SLA_CACHE_INT8) {
    uint2* sums = reinterpret_cast<uint2*>(parts);
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t u = word[r * W] ^ 0x80808080u;
      even += u & 0x00ff00ffu;
      odd += (u >> 8) & 0x00ff00ffu;
    }
    sums[threadIdx.x] = make_uint2(even, odd);
    __syncthreads();
    if (threadIdx.x < W) {
#pragma unroll
      for (int i = 1; i < P; ++i) {
        even += sums[i * W + threadIdx.x].x;
        odd += sums[i * W + threadIdx.x].y;
      }
      constexpr int kOff = 128 * kBlock;
      reinterpret_cast<float4*>(mean)[threadIdx.x] =
          make_float4((float)((int)(even & 0xffffu) - kOff) * f, (float)((int)(odd & 0xffffu) - kOff) * f,
                      (float)((int)(even >> 16) - kOff) * f, (float)((int)(odd >> 16) - kOff) * f);
    }
    return;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float x[4];
    decode4<KIND>(word[r * W], x);
    s.x += x[0];
    s.y += x[1];
    s.z += x[2];
    s.w += x[3];
  }
  parts[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < W) {
#pragma unroll
    for (int i = 1; i < P; ++i) {
      const float4 y = parts[i * W + threadIdx.x];
      s.x += y.x;
      s.y += y.y;
      s.z += y.z;
      s.w += y.w;
    }
    reinterpret_cast<float4*>(mean)[threadIdx.x] = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
  }
}

// ---------------------------------------------------------------------------
// append: one CTA a (block that may be written, KV head, sequence), keys and values apart.
// A thread holds its 16-element chunks as the bf16 words that it loaded (8 registers) and
// takes the largest magnitude on their bits, which order like the magnitudes. One pass: a page
// is read, its scale found with one barrier, and written. Bound by HBM for prompts (2 x 12 x
// 32760 rows of 128, int8: 80 us on the device, 5.9 TB/s of the 476 MB it cannot do without),
// by its chain of loads (length, page, rows, barrier) for a step's one token (64 sequences x 8
// heads: 6 us).
// ---------------------------------------------------------------------------
template <int KIND, int D>
__global__ void __launch_bounds__(kCta) append_kernel(const CacheView c, const __nv_bfloat16* __restrict__ k_new,
                                                      const __nv_bfloat16* __restrict__ v_new, int T,
                                                      const int32_t* __restrict__ lens,
                                                      const int32_t* __restrict__ n_new, int32_t* lens_out) {
  constexpr int C = D / 16;             // chunks of 16 elements a row
  constexpr int NT = kBlock * C / kCta;  // chunks a thread
  constexpr uint32_t kTop = 0x7b80;     // 2^120 in bf16
  __shared__ uint32_t slots[kCta / 32];
  __shared__ __align__(16) uint8_t tile[kBlock * D];
  __shared__ float4 parts[kCta];
  const int hk = blockIdx.x % c.H_kv, jj = blockIdx.x / c.H_kv, b = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  wait_for_previous();
  let_next_start();
  const int L = lens[b], n = n_new ? n_new[b] : T;
  const bool bad = L < 0 || L > c.cap || n < 0 || n > T || L + n > c.cap;
  if (blockIdx.x == 0 && is_k && threadIdx.x == 0) {
    if (bad) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
    if (lens_out) lens_out[b] = bad ? L : L + n;
  }
  if (bad) return;
  const int j = L / kBlock + jj, first = j * kBlock;
  if (first >= L + n || n == 0) return;
  const int lo = max(L - first, 0), hi = min(L + n - first, kBlock);  // rows of the page written now
  const int page = checked_page(c, b, j);
  const __nv_bfloat16* src = (is_k ? k_new : v_new) + ((size_t)b * c.H_kv + hk) * T * D;

  uint32_t x[NT][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = threadIdx.x + kCta * i, r = task / C, ch = task % C;
    uint4 u = make_uint4(0u, 0u, 0u, 0u), w = u;
    if (r >= lo && r < hi) {
      const uint4* p = reinterpret_cast<const uint4*>(src + (size_t)(first + r - L) * D + ch * 16);
      u = __ldcs(p);
      w = __ldcs(p + 1);
    }
    x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
    x[i][4] = w.x, x[i][5] = w.y, x[i][6] = w.z, x[i][7] = w.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, x[i][e] & 0x7fff7fffu);
  }
  if (page < 0) return;
  const size_t ph = (size_t)page * c.H_kv + hk;
  uint8_t* codes = (is_k ? c.k : c.v) + ph * kBlock * D;
  float* scale = (is_k ? c.k_scale : c.v_scale) + ph;
  top = max(top & 0xffffu, top >> 16);
  if (top > kTop) {  // NaN becomes 0, larger magnitudes 2^120
    report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheValue);
    top = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t y = 0;
        for (int s = 0; s < 32; s += 16) {
          uint32_t h = (x[i][e] >> s) & 0xffffu, mag = h & 0x7fffu;
          mag = mag > 0x7f80u ? 0u : min(mag, kTop);
          top = max(top, mag);
          y |= ((h & 0x8000u) | mag) << s;
        }
        x[i][e] = y;
      }
  }
  const bool open = lo > 0;
  const float was = open ? *scale : 0.f;
  top = block_max(top, slots);  // every thread has read the old scale behind this barrier
  const float to = fmaxf(was, exp2_int(scale_exponent<KIND>(__uint_as_float(top << 16))));
  const float inv = 1.f / to;
  const bool again = open && to != was;  // the codes held are rounded at the new scale
  const bool full = hi == kBlock && is_k && c.k_mean != nullptr;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = threadIdx.x + kCta * i, r = task / C, ch = task % C;
    uint4* at = reinterpret_cast<uint4*>(codes + r * D + ch * 16);
    uint4 code = make_uint4(0u, 0u, 0u, 0u);
    if (r >= lo) {  // slots behind the last token hold 0
      float y[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[2 * e] = __uint_as_float(x[i][e] << 16);
        y[2 * e + 1] = __uint_as_float(x[i][e] & 0xffff0000u);
      }
      code = encode16<KIND>(y, inv);
      *at = code;
    } else {
      if (again || full) code = *at;
      if (again) {
        code = recode16<KIND>(code, was * inv);
        *at = code;
      }
    }
    if (full) *reinterpret_cast<uint4*>(tile + r * D + ch * 16) = code;
  }
  if (threadIdx.x == 0) *scale = to;
  if (is_k && c.weight != nullptr && threadIdx.x >= lo && threadIdx.x < hi)
    c.weight[((size_t)b * c.H_kv + hk) * c.cap + first + threadIdx.x] = 0.f;
  if (full) {
    __syncthreads();
    write_mean<KIND, D>(tile, to, c.k_mean + ph * D, parts);
  }
}

// ---------------------------------------------------------------------------
// evict, first step: which slots stay (one cluster of eight CTAs a sequence and KV head, or one CTA)
//
// The budget - n_sink - n_recent heaviest of the slots between are those above a threshold
// weight and the first few equal to it. Each CTA keeps its eighth of the weights in shared
// memory as integers of the same order. The threshold is found digit by digit, 8 bits at a
// time: the CTAs' histograms are added through distributed shared memory. Weights crowd in
// few values of the first digit, so there lanes with the same one count together. Then
// every CTA counts its run, takes its place from the counts of those before, and writes its
// kept slots in order, with the pool rows that they are in. Bound by its chain of steps (four
// digits of a pass, a cluster barrier and a scan each), not by the 4 bytes a slot: 65536 slots
// of 4 heads 19 us, up to 16384 of 64 heads 21 us.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at the same place of another CTA's shared memory.
__device__ __forceinline__ int peer_int(const int* p, uint32_t rank) {
  uint32_t addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kSelAlone = 8192;  // slots that one CTA takes by itself at most

// Slots of one CTA's run: a multiple of 32 a warp.
__host__ __device__ inline int select_run(int n, int ctas, int threads) {
  return (int)align_up((size_t)(n + ctas - 1) / ctas, threads);
}

template <int kSelCluster, int kSelThreads>
__global__ void __cluster_dims__(kSelCluster, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const CacheView c, const int32_t* __restrict__ lens, int budget, int n_sink, int n_recent,
                        int32_t* __restrict__ kept, int32_t* lens_out, const int32_t* __restrict__ dst_table,
                        int same_weights, int* __restrict__ flags, int n_flags, int* __restrict__ rows) {
  extern __shared__ uint32_t keys[];  // [select_run(cap)]
  __shared__ int hist[2][256], total[256];
  __shared__ int s_digit, s_rest;
  __shared__ int above[kSelThreads / 32], equal[kSelThreads / 32], mine[2];
  const int bh = blockIdx.x / kSelCluster, b = bh / c.H_kv, hk = bh % c.H_kv;
  const int rank = (int)cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous();
  let_next_start();
  bool bad = false;
  const int n = checked_len(lens, b, c.cap, &bad), m = min(n, budget);
  if (hk == 0 && rank == 0 && tid == 0) {
    if (bad) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
    lens_out[b] = m;
  }
  // what the move's CTAs of this sequence and head count and signal with
  int* flag = flags + (size_t)bh * n_flags;
  for (int i = rank * kSelThreads + tid; i < n_flags - 1; i += kSelCluster * kSelThreads) flag[i] = 0;
  int32_t* out = kept + (size_t)bh * budget;
  rows += (size_t)bh * budget;
  // kept slot i comes from row `slot` of the sequence; rows: where that is in the pool, -1 nowhere
  auto page_of = [&](int slot) { return slot < n ? c.table[(size_t)b * c.max_blocks + slot / kBlock] : 0; };
  auto keep = [&](int i, int slot, int page) {
    out[i] = slot;
    const bool there = page >= 0 && page < c.n_pages;
    if (!there) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCachePage);
    rows[i] = there ? (page * c.H_kv + hk) * kBlock + slot % kBlock : -1;
  };
  for (int i = m + rank * kSelThreads + tid; i < budget; i += kSelCluster * kSelThreads) out[i] = -1;
  // whether the move has to: it packs some block in place, or its weights (one warp)
  auto tell = [&] {
    bool any = same_weights != 0;
    for (int i = lane; i * kBlock < m; i += 32)
      any |= dst_table[(size_t)b * (n_flags - 2) + i] == c.table[(size_t)b * c.max_blocks + i];
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) flag[n_flags - 1] = any;
  };
  const bool teller = rank == kSelCluster - 1 && warp == kSelThreads / 32 - 1;
  if (n <= budget) {  // the same for the whole cluster
    if (teller) tell();
    for (int i = rank * kSelThreads + tid; i < n; i += kSelCluster * kSelThreads) keep(i, i, page_of(i));
    return;
  }
  const float* w = c.weight + (size_t)bh * c.cap;
  const int run = select_run(n, kSelCluster, kSelThreads), a = min(n, rank * run), z = min(n, a + run);
  const int lo = n_sink, hi = n - n_recent;    // n_sink + n_recent <= budget < n: lo < hi
  const int want = budget - n_sink - n_recent;  // of the slots between
  for (int i = a + tid; i < z; i += kSelThreads) keys[i - a] = weight_key(w[i]);
  if (tid < 256) hist[0][tid] = hist[1][tid] = 0;
  __syncthreads();
  int rest = want;  // still to be taken among the keys that match the prefix
  uint32_t prefix = 0;
  if (want > 0) {
    int turn = 0;
    for (int shift = 24; shift >= 0; shift -= 8, turn ^= 1) {
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = a + tid; i - lane < z; i += kSelThreads) {
        uint32_t dig = 256;
        if (i < z && i >= lo && i < hi && (keys[i - a] & mask) == prefix) dig = (keys[i - a] >> shift) & 255u;
        if (shift == 24) {  // sign and exponent: few digits
          const uint32_t same = __match_any_sync(0xffffffffu, dig);
          if (dig < 256 && lane == __ffs(same) - 1) atomicAdd(&hist[turn][dig], __popc(same));
        } else if (dig < 256) {
          atomicAdd(&hist[turn][dig], 1);
        }
      }
      cluster_sync();
      if (tid < 256) {
        int s = 0;
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) s += peer_int(&hist[turn][tid], r);
        total[tid] = s;
        hist[turn ^ 1][tid] = 0;  // read by the others before the barrier above, if at all
      }
      __syncthreads();
      if (warp == 0) {  // digit whose keys, from the largest down, hold the rest-th one
        int v[8], s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = total[255 - 8 * lane - i];
          s += v[i];
        }
        int upto = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        int before = upto - s;
        if (before < rest && upto >= rest) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < rest && before + v[i] >= rest) {
              s_digit = 255 - 8 * lane - i;
              s_rest = rest - before;
              before = 1 << 30;
            } else {
              before += v[i];
            }
          }
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      rest = s_rest;
    }
  }
  // keys above prefix stay, and the first `rest` equal to it (none of either where want is 0)
  const int per = run / (kSelThreads / 32), wa = min(z, a + warp * per), wz = min(z, wa + per);
  int n_above = 0, n_equal = 0;
  for (int i = wa + lane; i - lane < wz; i += 32) {
    const bool held = i < wz && (i < lo || i >= hi), in = i < wz && !held && want > 0;
    const uint32_t key = in ? keys[i - a] : 0u;
    n_above += __popc(__ballot_sync(0xffffffffu, held || (in && key > prefix)));
    n_equal += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
  }
  if (lane == 0) {
    above[warp] = n_above;
    equal[warp] = n_equal;
  }
  __syncthreads();
  if (warp == 0) {
    const bool a_warp = lane < kSelThreads / 32;
    const int x = __reduce_add_sync(0xffffffffu, a_warp ? above[lane] : 0);
    const int y = __reduce_add_sync(0xffffffffu, a_warp ? equal[lane] : 0);
    if (lane == 0) {
      mine[0] = x;
      mine[1] = y;
    }
  }
  cluster_sync();
  int at = 0, eq = 0;
  for (int r = 0; r < rank; ++r) {
    at += peer_int(&mine[0], r);
    eq += peer_int(&mine[1], r);
  }
  cluster_sync();  // no CTA leaves while another reads its counts
  for (int i = 0; i < warp; ++i) {
    at += above[i];
    eq += equal[i];
  }
  at += min(eq, rest);
  if (teller) tell();
  int next_page = page_of(wa + lane);
  for (int i = wa + lane; i - lane < wz; i += 32) {
    const int page = next_page;
    next_page = page_of(i + 32);
    const bool held = i < wz && (i < lo || i >= hi), in = i < wz && !held && want > 0;
    const uint32_t key = in ? keys[i - a] : 0u;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eqs = __ballot_sync(0xffffffffu, in && key == prefix);
    const bool take = held || (in && (key > prefix || (key == prefix && eq + __popc(eqs & below) < rest)));
    const uint32_t takes = __ballot_sync(0xffffffffu, take);
    if (take) keep(at + __popc(takes & below), i, page);
    at += __popc(takes);
    eq += __popc(eqs);
  }
}

// ---------------------------------------------------------------------------
// evict, second step: the kept slots move, one CTA a (new block, KV head, sequence)
//
// A CTA loads its 64 rows of keys and values (16-byte chunks of whole rows, as codes), takes
// the largest magnitudes, and writes the block. Where the new page is the old one of that
// place it still holds rows that other new blocks load: those that keep slots of old block
// j are one or two (kept is ascending and kept[i] >= i), all of them at or before j. So every
// CTA signals when its loads are done, and one that writes in place first waits for those
// few. CTAs of a sequence that is packed in place take their block from a counter when they
// start: one that waits has only such before it that have started, and none of them waits
// before it has signalled. Bound by the latency of the gather (place, rows, barrier, write)
// with 40 KB or so in flight an SM: 8 x 8 heads x 4001 rows 35 us (131 MB, 3.8 TB/s).
// ---------------------------------------------------------------------------
// first i in [0, m) with from[i] >= slot, m if none
__device__ __forceinline__ int first_kept(const int32_t* from, int m, int slot) {
  int lo = 0, hi = m;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (from[mid] < slot) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Old scale / new scale 2^e, a finite number: beside an outlier that is evicted a row may have
// codes of 0 only, and its page's scale times 2^110 can be beyond fp32, which would make them
// NaN. Other codes never ask for more than 2^18: 2^-9 at least, they become 448 at most.
__device__ __forceinline__ float scale_ratio(float old, int e) { return fminf(old * exp2_int(-e), 1048576.f); }

template <int KIND, int D>
__global__ void __launch_bounds__(kCta, 5) evict_move_kernel(const CacheView c, const int32_t* kept,
                                                          const int32_t* lens, int budget, const int32_t* dst_table,
                                                          float* weight_out, int* flags, int n_flags, const int* rows) {
  constexpr int C = D / 16;
  constexpr int NT = kBlock * C / kCta;
  __shared__ uint32_t slots[2][kCta / 32];
  __shared__ __align__(16) uint8_t tile[kBlock * D];
  __shared__ float4 parts[kCta];
  __shared__ int s_row[kBlock];
  __shared__ int s_j, s_late;
  const int tid = threadIdx.x, nd = (budget + kBlock - 1) / kBlock;
  const int bh = blockIdx.x / nd, b = bh / c.H_kv, hk = bh % c.H_kv;
  wait_for_previous();
  let_next_start();
  bool bad = false;
  const int m = min(checked_len(lens, b, c.cap, &bad), budget);
  int* done = flags + (size_t)bh * n_flags;  // [nd] signals, a counter, whether they are needed
  const int32_t* from = kept + (size_t)bh * budget;
  rows += (size_t)bh * budget;
  // the block that the launch order gives is on its way before it is known whether it may be taken
  int j = blockIdx.x - bh * nd;
  const bool ordered = done[nd + 1] != 0;
  if (tid < kBlock) s_row[tid] = j * kBlock + tid < m ? rows[j * kBlock + tid] : -1;
  int to_page = dst_table[(size_t)b * nd + j];
  if (tid == 0) s_late = 0;
  if (ordered) {
    if (tid == 0) s_j = atomicAdd(&done[nd], 1);
    __syncthreads();
    j = s_j;
    if (tid < kBlock) s_row[tid] = j * kBlock + tid < m ? rows[j * kBlock + tid] : -1;
    to_page = dst_table[(size_t)b * nd + j];
  }
  const int first = j * kBlock;
  if (first >= m) return;
  __syncthreads();
  uint4 kc[NT], vc[NT];
  float ks[NT], vs[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = tid + kCta * i, r = task / C, ch = task % C, row = s_row[r];
    kc[i] = vc[i] = make_uint4(0u, 0u, 0u, 0u);
    ks[i] = vs[i] = 0.f;
    if (row >= 0) {
      const size_t at = (size_t)row * D + ch * 16;
      kc[i] = *reinterpret_cast<const uint4*>(c.k + at);
      vc[i] = *reinterpret_cast<const uint4*>(c.v + at);
      ks[i] = c.k_scale[row / kBlock];
      vs[i] = c.v_scale[row / kBlock];
    }
  }
  const size_t wrow = (size_t)bh * c.cap;
  const float w = tid < kBlock && first + tid < m ? c.weight[wrow + from[first + tid]] : 0.f;
  float ka = 0.f, va = 0.f;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    ka = fmaxf(ka, max_magnitude16<KIND>(kc[i]) * ks[i]);
    va = fmaxf(va, max_magnitude16<KIND>(vc[i]) * vs[i]);
  }
  const uint32_t kw = __reduce_max_sync(0xffffffffu, __float_as_uint(ka));
  const uint32_t vw = __reduce_max_sync(0xffffffffu, __float_as_uint(va));
  if ((tid & 31) == 0) {
    slots[0][tid >> 5] = kw;
    slots[1][tid >> 5] = vw;
  }
  __syncthreads();  // every thread has its rows
  uint32_t km = slots[0][0], vm = slots[1][0];
#pragma unroll
  for (int i = 1; i < kCta / 32; ++i) {
    km = max(km, slots[0][i]);
    vm = max(vm, slots[1][i]);
  }
  if (tid == 0) {
    if (ordered) asm volatile("fence.acq_rel.gpu;\n\tst.relaxed.gpu.global.s32 [%0], 1;" ::"l"(done + j) : "memory");
    if (weight_out == c.weight || to_page == c.table[(size_t)b * c.max_blocks + j]) {
      const int i0 = first_kept(from, m, first), i1 = first_kept(from, m, first + kBlock);
      const uint64_t t0 = tc::globaltimer();
      for (int y = i0 / kBlock; y * kBlock < i1 && y < j; ++y) {
        int seen = 0;
        for (;;) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(done + y) : "memory");
          if (seen || tc::globaltimer() - t0 > tc::kTimeoutNs) break;
          __nanosleep(50);
        }
        if (!seen) s_late = 1;
      }
      if (s_late) report(c.status, SLA_ERR_DEVICE_TIMEOUT, kDetailTimeout);
    }
  }
  __syncthreads();
  if (s_late) return;  // the old rows stay as they are
  if (tid < kBlock && first + tid < m) weight_out[wrow + first + tid] = w;
  if (to_page < 0 || to_page >= c.n_pages) {
    if (tid == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCachePage);
    return;
  }
  const size_t ph = (size_t)to_page * c.H_kv + hk;
  const int ke = scale_exponent<KIND>(fminf(__uint_as_float(km), kCacheMaxAbs));
  const int ve = scale_exponent<KIND>(fminf(__uint_as_float(vm), kCacheMaxAbs));
  const float kt = exp2_int(ke), vt = exp2_int(ve);
  const bool full = first + kBlock <= m && c.k_mean != nullptr;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = tid + kCta * i, r = task / C, ch = task % C;
    const size_t at = (ph * kBlock + r) * D + ch * 16;
    if (ks[i] != kt) kc[i] = recode16<KIND>(kc[i], scale_ratio(ks[i], ke));
    if (vs[i] != vt) vc[i] = recode16<KIND>(vc[i], scale_ratio(vs[i], ve));
    *reinterpret_cast<uint4*>(c.k + at) = kc[i];
    *reinterpret_cast<uint4*>(c.v + at) = vc[i];
    if (full) *reinterpret_cast<uint4*>(tile + r * D + ch * 16) = kc[i];
  }
  if (tid == 0) {
    c.k_scale[ph] = kt;
    c.v_scale[ph] = vt;
  }
  if (full) {
    __syncthreads();
    write_mean<KIND, D>(tile, kt, c.k_mean + ph * D, parts);
  }
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

sla_status sla_cache_validate_config(const sla_cache_config* cfg) { return check_sizes(cfg); }

sla_status sla_cache_append(const void* k, const void* v, const sla_cache_config* cfg, const sla_cache* cache,
                            int32_t T, const int32_t* lens, const int32_t* n_new, int32_t* lens_out, void* stream) {
  CacheView c;
  const sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  if (!k || !v || !lens || T < 1) return SLA_ERR_INVALID_ARG;
  if (lengths_overlap(lens_out, lens, c.B) || lengths_overlap(lens_out, n_new, c.B)) return SLA_ERR_INVALID_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(lens, 4) || !aligned_to(n_new, 4) ||
      !aligned_to(lens_out, 4))
    return SLA_ERR_INVALID_ARG;
  if (T > c.cap && !n_new) return SLA_ERR_INVALID_ARG;  // no sequence could take them
  // blocks that the tokens one sequence takes can reach into
  const int most = T < c.cap ? T : c.cap;
  const int touched = std::min((most + kBlock - 2) / kBlock + 1, c.max_blocks);
  const dim3 grid((unsigned)(touched * c.H_kv), (unsigned)c.B, 2);
  cudaStream_t s = (cudaStream_t)stream;
  auto run = [&](auto kernel) {
    return launch_overlapped(kernel, grid, kCta, 0, s, c, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, (int)T, lens,
                             n_new, lens_out);
  };
  cudaError_t e;
  if (c.kind == SLA_CACHE_E4M3) e = c.d == 128 ? run(append_kernel<SLA_CACHE_E4M3, 128>) : run(append_kernel<SLA_CACHE_E4M3, 64>);
  else e = c.d == 128 ? run(append_kernel<SLA_CACHE_INT8, 128>) : run(append_kernel<SLA_CACHE_INT8, 64>);
  return e == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

// ints a (sequence, KV head): a signal of each new block, a counter, whether they are needed
static int evict_flags(int budget) { return (budget + kBlock - 1) / kBlock + 2; }

size_t sla_cache_evict_workspace_bytes(const sla_cache_config* cfg, int32_t budget) {
  if (check_sizes(cfg) != SLA_OK || budget < 1 || budget > cfg->max_blocks * kBlock) return 0;
  return align_up((size_t)cfg->B * cfg->H_kv * ((size_t)evict_flags(budget) + budget) * sizeof(int), 256);
}

sla_status sla_cache_evict(const sla_cache_config* cfg, const sla_cache* cache, const int32_t* lens, int32_t budget,
                           int32_t n_sink, int32_t n_recent, const int32_t* dst_table, float* weight_out,
                           int32_t* kept, int32_t* lens_out, void* ws, size_t ws_bytes, void* stream) {
  CacheView c;
  const sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  if (!lens || !dst_table || !weight_out || !kept || !lens_out || !c.weight || lengths_overlap(lens_out, lens, c.B))
    return SLA_ERR_INVALID_ARG;
  if (!aligned_to(lens, 4) || !aligned_to(dst_table, 4) || !aligned_to(weight_out, 16) || !aligned_to(kept, 4) ||
      !aligned_to(lens_out, 4))
    return SLA_ERR_INVALID_ARG;
  if (budget < 1 || budget > c.cap || n_sink < 0 || n_recent < 0 || n_sink > budget - n_recent)
    return SLA_ERR_INVALID_ARG;
  if ((int64_t)c.B * c.H_kv * (evict_flags(budget) - 2) >= ((int64_t)1 << 31)) return SLA_ERR_UNSUPPORTED;  // grid
  if (!ws || !aligned_to(ws, 256) || ws_bytes < sla_cache_evict_workspace_bytes(cfg, budget))
    return SLA_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  int* flags = (int*)ws;
  const int n_flags = evict_flags(budget), nd = n_flags - 2;
  int* rows = flags + (size_t)c.B * c.H_kv * n_flags;
  // The keys take turns of one a thread: 1024 threads where all CTAs are resident at once with
  // them (65536 slots of 4 heads: 31 us for the call, 35 with 512), else 512 (64 heads of 16384
  // slots: 60 us, 72 with 1024, whose 512 CTAs came in two waves). Up to 2048 slots one CTA is
  // no slower than eight (8 heads of 2048: 13 and 14 us), and up to 8192 it is faster where the
  // eights come in several waves (300 heads of 1025 slots 21 and 68 us, of 8192 104 and 124; 64
  // heads of 8192, in one wave, 40 and 32). The rule goes by the table's length, since the host
  // does not know the sequences': short ones in a table of more than 8192 slots take eight CTAs.
  auto select = [&](auto kernel, int ctas, int threads, int most) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               select_run(most, ctas, threads) * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3(c.B * c.H_kv * ctas), threads,
                             select_run(c.cap, ctas, threads) * sizeof(uint32_t), s, c, lens, (int)budget, (int)n_sink,
                             (int)n_recent, kept, lens_out, dst_table, (int)(weight_out == c.weight), flags, n_flags, rows);
  };
  const int most = kMaxBlocks * kBlock, heads = c.B * c.H_kv;
  const bool alone = c.cap <= 2048 || (c.cap <= kSelAlone && heads * 8 > 4 * 148);
  cudaError_t e = alone                  ? select(evict_select_kernel<1, 512>, 1, 512, kSelAlone)
                  : heads * 8 <= 2 * 148 ? select(evict_select_kernel<8, 1024>, 8, 1024, most)
                                         : select(evict_select_kernel<8, 512>, 8, 512, most);
  if (e != cudaSuccess) return SLA_ERR_CUDA;
  auto run = [&](auto kernel) {
    return launch_overlapped(kernel, dim3((unsigned)(c.B * c.H_kv * nd)), kCta, 0, s, c, (const int32_t*)kept, lens,
                             (int)budget, dst_table, weight_out, flags, n_flags, (const int*)rows);
  };
  if (c.kind == SLA_CACHE_E4M3)
    e = c.d == 128 ? run(evict_move_kernel<SLA_CACHE_E4M3, 128>) : run(evict_move_kernel<SLA_CACHE_E4M3, 64>);
  else
    e = c.d == 128 ? run(evict_move_kernel<SLA_CACHE_INT8, 128>) : run(evict_move_kernel<SLA_CACHE_INT8, 64>);
  return e == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

}  // extern "C"
