// The 8-bit paged cache: argument checks, sla_cache_append and sla_cache_evict.
//
// A page holds 64 slots of one KV head after the other, codes [H_kv][64][d], so that the
// page of one head is one contiguous run of 64 * d bytes.
#include <math.h>

#include "cache.cuh"

namespace sla {

static bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

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
  return SLA_OK;
}

namespace {

// Largest of one non-negative value a thread over the block's 256 threads (all get it).
__device__ __forceinline__ float block_max_256(float a, uint32_t* slots) {
  const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = w;
  __syncthreads();
  uint32_t m = slots[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, slots[i]);
  return __uint_as_float(m);
}

// One 16-element chunk of a row as its 16 code bytes.
template <int KIND>
__device__ __forceinline__ uint4 encode16(const float* x, float inv) {
  uint4 c;
  c.x = encode4<KIND>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  c.y = encode4<KIND>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
  c.z = encode4<KIND>(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv);
  c.w = encode4<KIND>(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv);
  return c;
}
template <int KIND>
__device__ __forceinline__ void decode16(const uint4& c, float* x) {
  decode4<KIND>(c.x, x);
  decode4<KIND>(c.y, x + 4);
  decode4<KIND>(c.z, x + 8);
  decode4<KIND>(c.w, x + 12);
}

// Mean over 64 rows of codes in shared memory, times the scale. Codes are integers times
// 2^-9 (e4m3) or integers (int8) of at most 19 bits, so 64 of them add up exactly in fp32.
template <int KIND, int D>
__device__ __forceinline__ void write_mean(const uint8_t* tile, float scale, float* mean) {
  for (int c = threadIdx.x; c < D / 4; c += blockDim.x) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    for (int r = 0; r < kBlock; ++r) {
      float x[4];
      decode4<KIND>(reinterpret_cast<const uint32_t*>(tile + r * D)[c], x);
      s0 += x[0];
      s1 += x[1];
      s2 += x[2];
      s3 += x[3];
    }
    const float f = scale * (1.f / kBlock);
    reinterpret_cast<float4*>(mean)[c] = make_float4(s0 * f, s1 * f, s2 * f, s3 * f);
  }
}

// ---------------------------------------------------------------------------
// append: one CTA a (block that may be written, KV head, sequence), keys and values apart
// ---------------------------------------------------------------------------
template <int KIND, int D>
__global__ void __launch_bounds__(256) append_kernel(const CacheView c, const __nv_bfloat16* __restrict__ k_new,
                                                     const __nv_bfloat16* __restrict__ v_new, int T,
                                                     const int32_t* __restrict__ lens,
                                                     const int32_t* __restrict__ n_new, int32_t* lens_out) {
  constexpr int C = D / 16;            // chunks of 16 elements a row
  constexpr int NT = kBlock * C / 256;  // chunks a thread
  __shared__ uint32_t slots[8];
  __shared__ __align__(16) uint8_t tile[kBlock * D];
  const int hk = blockIdx.x % c.H_kv, jj = blockIdx.x / c.H_kv, b = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
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
  if (page < 0) return;
  const size_t ph = (size_t)page * c.H_kv + hk;
  uint8_t* codes = (is_k ? c.k : c.v) + ph * kBlock * D;
  float* scale = (is_k ? c.k_scale : c.v_scale) + ph;
  const __nv_bfloat16* src = (is_k ? k_new : v_new) + ((size_t)b * c.H_kv + hk) * T * D;

  float x[NT][16];
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = threadIdx.x + 256 * i, r = task / C, ch = task % C;
    if (r >= lo && r < hi) {
      const uint4* p = reinterpret_cast<const uint4*>(src + (size_t)(first + r - L) * D + ch * 16);
      const uint4 u = p[0], w = p[1];
      const uint32_t words[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = unpack_bf16(words[e]);
        x[i][2 * e] = f.x;
        x[i][2 * e + 1] = f.y;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (!(fabsf(x[i][e]) <= kCacheMaxAbs)) {
          odd = true;
          x[i][e] = isnan(x[i][e]) ? 0.f : copysignf(kCacheMaxAbs, x[i][e]);
        }
        amax = fmaxf(amax, fabsf(x[i][e]));
      }
    }
  }
  if (odd) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheValue);
  const bool open = lo > 0;
  const float was = open ? *scale : 0.f;
  amax = block_max_256(amax, slots);  // every thread has read the old scale behind this barrier
  const float to = fmaxf(was, exp2_int(scale_exponent<KIND>(amax)));
  const float inv = 1.f / to;
  const bool again = open && to != was;  // the codes held are rounded at the new scale
  const bool full = hi == kBlock && is_k && c.k_mean != nullptr;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int task = threadIdx.x + 256 * i, r = task / C, ch = task % C;
    uint4* at = reinterpret_cast<uint4*>(codes + r * D + ch * 16);
    uint4 code = make_uint4(0u, 0u, 0u, 0u);
    if (r >= lo && r < hi) {
      code = encode16<KIND>(x[i], inv);
      *at = code;
    } else if (r < lo) {
      if (again || full) code = *at;
      if (again) {
        float y[16];
        decode16<KIND>(code, y);
        code = encode16<KIND>(y, was * inv);
        *at = code;
      }
    } else {
      *at = code;  // slots behind the last token hold 0
    }
    if (full) *reinterpret_cast<uint4*>(tile + r * D + ch * 16) = code;
  }
  if (threadIdx.x == 0) *scale = to;
  if (is_k && c.weight != nullptr && threadIdx.x >= lo && threadIdx.x < hi)
    c.weight[((size_t)b * c.H_kv + hk) * c.cap + first + threadIdx.x] = 0.f;
  if (full) {
    __syncthreads();
    write_mean<KIND, D>(tile, to, c.k_mean + ph * D);
  }
}

// ---------------------------------------------------------------------------
// evict, first step: which slots stay (one CTA a sequence and KV head)
//
// The budget - n_sink - n_recent heaviest of the slots between are those above a threshold
// weight and the first few equal to it. The threshold is found digit by digit (8 bits of
// the weight's order-preserving integer at a time, a histogram each), then every warp
// counts its run of slots and, after a scan over the warps, writes its kept slots in order.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(1024) evict_select_kernel(const CacheView c, const int32_t* __restrict__ lens,
                                                            int budget, int n_sink, int n_recent,
                                                            int32_t* __restrict__ kept, int32_t* lens_out) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_rest;
  __shared__ int above[32], equal[32];
  const int b = blockIdx.x / c.H_kv, hk = blockIdx.x % c.H_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const int n = checked_len(lens, b, c.cap, &bad), m = min(n, budget);
  if (hk == 0 && tid == 0) {
    if (bad) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
    lens_out[b] = m;
  }
  int32_t* out = kept + (size_t)blockIdx.x * budget;
  for (int i = m + tid; i < budget; i += 1024) out[i] = -1;
  if (n <= budget) {
    for (int i = tid; i < n; i += 1024) out[i] = i;
    return;
  }
  const float* w = c.weight + (size_t)blockIdx.x * c.cap;
  const int lo = n_sink, hi = n - n_recent;  // n_sink + n_recent <= budget < n: lo < hi
  int rest = budget - n_sink - n_recent;     // still to be taken among the keys that match the prefix
  uint32_t prefix = 0;
  if (rest > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = lo + tid; i < hi; i += 1024) {
        const uint32_t key = weight_key(w[i]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = rest, dgt = 255;
        while (hist[dgt] < left) left -= hist[dgt--];  // at least `rest` keys match: ends at dgt >= 0
        s_digit = dgt;
        s_rest = left;
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      rest = s_rest;
    }
  }
  // keys above prefix stay, and the first `rest` equal to it (none of either where rest was 0)
  const bool any = budget - n_sink - n_recent > 0;
  const int per = ((n + 31) / 32 + 31) / 32 * 32, a = min(n, warp * per), z = min(n, a + per);
  int n_above = 0, n_equal = 0;
  for (int i = a + lane; i - lane < z; i += 32) {
    const bool in = i < z && i >= lo && i < hi;
    const bool held = i < z && (i < lo || i >= hi);
    const uint32_t key = in ? weight_key(w[i]) : 0u;
    n_above += __popc(__ballot_sync(0xffffffffu, held || (in && any && key > prefix)));
    n_equal += __popc(__ballot_sync(0xffffffffu, in && any && key == prefix));
  }
  if (lane == 0) {
    above[warp] = n_above;
    equal[warp] = n_equal;
  }
  __syncthreads();
  int at = 0, eq = 0;
  for (int i = 0; i < warp; ++i) {
    at += above[i];
    eq += equal[i];
  }
  at += min(eq, rest);
  for (int i = a + lane; i - lane < z; i += 32) {
    const bool in = i < z && i >= lo && i < hi;
    const bool held = i < z && (i < lo || i >= hi);
    const uint32_t key = in ? weight_key(w[i]) : 0u;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eqs = __ballot_sync(0xffffffffu, in && any && key == prefix);
    const bool take = held || (in && any && (key > prefix || (key == prefix && eq + __popc(eqs & below) < rest)));
    const uint32_t takes = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(takes & below)] = i;
    at += __popc(takes);
    eq += __popc(eqs);
  }
}

// ---------------------------------------------------------------------------
// evict, second step: the kept slots move (one CTA a sequence and KV head, keys and values
// apart, new blocks in ascending order: kept[i] >= i, so a new block's page, where it is
// the old one of that place, holds no slot that a later new block reads)
// ---------------------------------------------------------------------------
template <int KIND, int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const CacheView c, const int32_t* __restrict__ kept,
                                                         const int32_t* __restrict__ lens, int budget,
                                                         const int32_t* __restrict__ dst_table, float* weight_out) {
  constexpr int C = D / 16;
  constexpr int NT = kBlock * C / 256;
  __shared__ uint32_t slots[8];
  __shared__ __align__(16) uint8_t tile[kBlock * D];
  const int b = blockIdx.x / c.H_kv, hk = blockIdx.x % c.H_kv;
  const bool is_k = blockIdx.z == 0;
  bool bad = false;
  const int m = min(checked_len(lens, b, c.cap, &bad), budget);
  const int nd = (budget + kBlock - 1) / kBlock;
  const int32_t* from = kept + (size_t)blockIdx.x * budget;
  const size_t wrow = (size_t)blockIdx.x * c.cap;
  uint8_t* pool = is_k ? c.k : c.v;
  float* scales = is_k ? c.k_scale : c.v_scale;
  for (int j = 0; j * kBlock < m; ++j) {
    float x[NT][16];
    float amax = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int task = threadIdx.x + 256 * i, r = task / C, ch = task % C;
      const int slot = j * kBlock + r < m ? from[j * kBlock + r] : -1;
      const int page = slot < 0 ? -1 : checked_page(c, b, slot / kBlock);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] = 0.f;
      if (page >= 0) {
        const size_t ph = (size_t)page * c.H_kv + hk;
        const uint4 code = *reinterpret_cast<const uint4*>(pool + (ph * kBlock + slot % kBlock) * D + ch * 16);
        const float s = scales[ph];
        decode16<KIND>(code, x[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[i][e] *= s;
          amax = fmaxf(amax, fabsf(x[i][e]));
        }
      }
      if (is_k && ch == 0 && slot >= 0) w = c.weight[wrow + slot];
      if (is_k && ch == 0) {
        // held until every thread has read its sources
        if (slot >= 0) reinterpret_cast<float*>(tile)[r] = w;
      }
    }
    amax = block_max_256(fminf(amax, kCacheMaxAbs), slots);
    if (is_k && threadIdx.x < kBlock && j * kBlock + threadIdx.x < m)
      weight_out[wrow + j * kBlock + threadIdx.x] = reinterpret_cast<const float*>(tile)[threadIdx.x];
    __syncthreads();
    const int page = dst_table[(size_t)b * nd + j];
    if (page < 0 || page >= c.n_pages) {
      if (threadIdx.x == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCachePage);
      continue;
    }
    const size_t ph = (size_t)page * c.H_kv + hk;
    const int ex = scale_exponent<KIND>(amax);
    const float inv = exp2_int(-ex);
    const bool full = (j + 1) * kBlock <= m && is_k && c.k_mean != nullptr;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int task = threadIdx.x + 256 * i, r = task / C, ch = task % C;
      const uint4 code = encode16<KIND>(x[i], inv);
      *reinterpret_cast<uint4*>(pool + (ph * kBlock + r) * D + ch * 16) = code;
      if (full) *reinterpret_cast<uint4*>(tile + r * D + ch * 16) = code;
    }
    if (threadIdx.x == 0) scales[ph] = exp2_int(ex);
    if (full) {
      __syncthreads();
      write_mean<KIND, D>(tile, exp2_int(ex), c.k_mean + ph * D);
    }
    __syncthreads();
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
  if (!k || !v || !lens || T < 1 || lens == lens_out) return SLA_ERR_INVALID_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(lens, 4) || !aligned_to(n_new, 4) ||
      !aligned_to(lens_out, 4))
    return SLA_ERR_INVALID_ARG;
  if (T > c.cap) return SLA_ERR_INVALID_ARG;  // no sequence could take them
  const int touched = (T + kBlock - 2) / kBlock + 1;  // blocks that T tokens can reach into
  const dim3 grid((unsigned)(touched * c.H_kv), (unsigned)c.B, 2);
  cudaStream_t s = (cudaStream_t)stream;
  auto run = [&](auto kernel) {
    kernel<<<grid, 256, 0, s>>>(c, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, T, lens, n_new, lens_out);
  };
  if (c.kind == SLA_CACHE_E4M3) {
    if (c.d == 128) run(append_kernel<SLA_CACHE_E4M3, 128>);
    else run(append_kernel<SLA_CACHE_E4M3, 64>);
  } else {
    if (c.d == 128) run(append_kernel<SLA_CACHE_INT8, 128>);
    else run(append_kernel<SLA_CACHE_INT8, 64>);
  }
  return cudaGetLastError() == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

size_t sla_cache_evict_workspace_bytes(const sla_cache_config* cfg, int32_t budget) {
  if (check_sizes(cfg) != SLA_OK || budget < 1 || budget > cfg->max_blocks * kBlock) return 0;
  return 256;
}

sla_status sla_cache_evict(const sla_cache_config* cfg, const sla_cache* cache, const int32_t* lens, int32_t budget,
                           int32_t n_sink, int32_t n_recent, const int32_t* dst_table, float* weight_out,
                           int32_t* kept, int32_t* lens_out, void* ws, size_t ws_bytes, void* stream) {
  CacheView c;
  const sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  if (!lens || !dst_table || !weight_out || !kept || !lens_out || !c.weight || lens == lens_out)
    return SLA_ERR_INVALID_ARG;
  if (!aligned_to(lens, 4) || !aligned_to(dst_table, 4) || !aligned_to(weight_out, 16) || !aligned_to(kept, 4) ||
      !aligned_to(lens_out, 4))
    return SLA_ERR_INVALID_ARG;
  if (budget < 1 || budget > c.cap || n_sink < 0 || n_recent < 0 || n_sink > budget - n_recent)
    return SLA_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256) || ws_bytes < sla_cache_evict_workspace_bytes(cfg, budget))
    return SLA_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  evict_select_kernel<<<c.B * c.H_kv, 1024, 0, s>>>(c, lens, budget, n_sink, n_recent, kept, lens_out);
  const dim3 grid((unsigned)(c.B * c.H_kv), 1, 2);
  auto run = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(c, kept, lens, budget, dst_table, weight_out); };
  if (c.kind == SLA_CACHE_E4M3) {
    if (c.d == 128) run(evict_move_kernel<SLA_CACHE_E4M3, 128>);
    else run(evict_move_kernel<SLA_CACHE_E4M3, 64>);
  } else {
    if (c.d == 128) run(evict_move_kernel<SLA_CACHE_INT8, 128>);
    else run(evict_move_kernel<SLA_CACHE_INT8, 64>);
  }
  return cudaGetLastError() == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

}  // extern "C"
