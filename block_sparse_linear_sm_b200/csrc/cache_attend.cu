// sla_cache_attend: softmax attention of a step's queries over the paged 8-bit cache.
#include "cache.cuh"

namespace sla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Step {
  const __nv_bfloat16* q;
  const int32_t *lens, *n_new, *sel;
  __nv_bfloat16* out;
  float* lse;  // [B, H, T], natural log; -inf where a row sees nothing
  int T, top_n, window;
};

// Whether block j is in the list, and whether every entry up to its place is in order.
__device__ bool in_list(const int32_t* list, int n, int j) {
  int top = -1;
  for (int i = 0; i < n; ++i) {
    if (list[i] == j && j > top) return true;
    top = max(top, list[i]);
  }
  return false;
}

// Score of one row against slot s of (b, hk): a warp, lane holds d/32 elements of q.
template <int KIND, int D>
__device__ __forceinline__ float score_of(const CacheView& c, size_t ph, int row, const float* q, int lane) {
  constexpr int E = D / 32;
  const uint8_t* p = c.k + (ph * kBlock + row) * D + lane * E;
  float x[4], a = 0.f;
  decode4<KIND>(E == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p), x);
#pragma unroll
  for (int e = 0; e < E; ++e) a += q[e] * x[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a * c.k_scale[ph] * c.scale;
}

// One CTA a query row; its warps take the slots in turn and are merged at the end.
template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(const CacheView c, const Step a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int h = blockIdx.x % c.H, b = blockIdx.x / c.H, t = blockIdx.y, hk = h / c.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  const int L = checked_len(a.lens, b, c.cap, &bad), n = checked_new(a.n_new, b, a.T, &bad);
  if (bad && threadIdx.x == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
  const int pos = t < n ? L - n + t : -1;
  const size_t row = (size_t)blockIdx.x * a.T + t;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row * D + lane * E + e]);
  const int32_t* list = a.sel ? a.sel + ((size_t)b * c.H_kv + hk) * a.top_n : nullptr;
  if (list != nullptr && threadIdx.x == 0)
    for (int i = 0, top = -1; i < a.top_n; ++i) {
      if (list[i] >= 0 && (list[i] <= top || list[i] >= (L + kBlock - 1) / kBlock))
        report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheSel);
      top = max(top, list[i]);
    }
  for (int j = 0; j * kBlock <= pos; ++j) {
    const bool chosen = list ? in_list(list, a.top_n, j) : a.window == 0;
    const int lo = chosen ? 0 : max(0, pos - a.window + 1 - j * kBlock);
    const int hi = min(kBlock, pos - j * kBlock + 1);
    if (lo >= hi) continue;
    const int page = checked_page(c, b, j);
    if (page < 0) continue;
    const size_t ph = (size_t)page * c.H_kv + hk;
    for (int r = lo + warp; r < hi; r += kWarps) {
      const float s = score_of<KIND, D>(c, ph, r, q, lane);
      const float top = fmaxf(m, s), keep = __expf(m - top), p = __expf(s - top);
      const uint8_t* v = c.v + (ph * kBlock + r) * D + lane * E;
      float x[4];
      decode4<KIND>(E == 4 ? *reinterpret_cast<const uint32_t*>(v) : *reinterpret_cast<const uint16_t*>(v), x);
      const float f = p * c.v_scale[ph];
      for (int e = 0; e < E; ++e) o[e] = o[e] * keep + f * x[e];
      l = l * keep + p;
      m = top;
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w) sum += s_l[w] == 0.f ? 0.f : s_l[w] * __expf(s_m[w] - top);  // 0: no slot; NaN stays
  if (threadIdx.x < D) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (s_l[w] != 0.f) y += s_o[w][threadIdx.x] * __expf(s_m[w] - top);
    a.out[row * D + threadIdx.x] = __float2bfloat16(sum == 0.f ? 0.f : y / sum);
  }
  if (threadIdx.x == 0) a.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// weight[b, hk, s] += sum over the group's heads and the step's rows of exp(score - lse).
// One CTA a (block, sequence, KV head); a warp a slot.
template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) weight_kernel(const CacheView c, const Step a) {
  constexpr int E = D / 32;
  const int j = blockIdx.x, b = blockIdx.y / c.H_kv, hk = blockIdx.y % c.H_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  const int L = checked_len(a.lens, b, c.cap, &bad), n = checked_new(a.n_new, b, a.T, &bad);
  if (j * kBlock >= L) return;
  const int page = checked_page(c, b, j);
  if (page < 0) return;
  const size_t ph = (size_t)page * c.H_kv + hk;
  const bool chosen = a.sel ? in_list(a.sel + ((size_t)b * c.H_kv + hk) * a.top_n, a.top_n, j) : a.window == 0;
  for (int r = warp; r < kBlock && j * kBlock + r < L; r += kWarps) {
    const int s = j * kBlock + r;
    float sum = 0.f;
    for (int g = 0; g < c.group; ++g)
      for (int t = 0; t < n; ++t) {
        const int pos = L - n + t;
        if (s > pos || !(chosen || s > pos - a.window)) continue;
        const size_t row = ((size_t)b * c.H + hk * c.group + g) * a.T + t;
        float q[E];
        for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row * D + lane * E + e]);
        sum += __expf(score_of<KIND, D>(c, ph, r, q, lane) - a.lse[row]);
      }
    if (lane == 0) c.weight[((size_t)b * c.H_kv + hk) * c.cap + s] += sum;
  }
}

sla_status check_step(const sla_cache_config* c, int32_t T, int32_t top_n, int32_t window) {
  const sla_status st = sla_cache_validate_config(c);
  if (st != SLA_OK) return st;
  if (T < 1 || top_n < 0 || window < 0) return SLA_ERR_INVALID_ARG;
  if (T > kCacheMaxT || (int64_t)T * (c->H / c->H_kv) > kCacheMaxRows || top_n > kCacheMaxSel)
    return SLA_ERR_UNSUPPORTED;
  return SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_cache_attend_workspace_bytes(const sla_cache_config* cfg, int32_t T, int32_t top_n, int32_t window,
                                        int32_t with_weight) {
  if (check_step(cfg, T, top_n, window) != SLA_OK) return 0;
  return align_up((size_t)cfg->B * cfg->H * T * sizeof(float), 256);
}

sla_status sla_cache_attend(const void* q, const sla_cache_config* cfg, const sla_cache* cache, int32_t T,
                            const int32_t* lens, const int32_t* n_new, const int32_t* sel, int32_t top_n,
                            int32_t window, void* out, void* ws, size_t ws_bytes, void* stream) {
  CacheView c;
  sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  st = check_step(cfg, T, top_n, window);
  if (st != SLA_OK) return st;
  if (!q || !lens || !out || q == out || (sel == nullptr) != (top_n == 0)) return SLA_ERR_INVALID_ARG;
  if (((uintptr_t)q % 16) || ((uintptr_t)out % 16) || ((uintptr_t)lens % 4) || ((uintptr_t)n_new % 4) ||
      ((uintptr_t)sel % 4))
    return SLA_ERR_INVALID_ARG;
  if (!ws || ((uintptr_t)ws % 256) ||
      ws_bytes < sla_cache_attend_workspace_bytes(cfg, T, top_n, window, c.weight != nullptr))
    return SLA_ERR_WORKSPACE;
  Step a;
  a.q = (const __nv_bfloat16*)q;
  a.lens = lens;
  a.n_new = n_new;
  a.sel = sel;
  a.out = (__nv_bfloat16*)out;
  a.lse = (float*)ws;
  a.T = T;
  a.top_n = top_n;
  a.window = window;
  cudaStream_t s = (cudaStream_t)stream;
  auto run = [&](auto attend, auto weigh) {
    attend<<<dim3(c.B * c.H, T), kThreads, 0, s>>>(c, a);
    if (c.weight != nullptr) weigh<<<dim3(c.max_blocks, c.B * c.H_kv), kThreads, 0, s>>>(c, a);
  };
  if (c.kind == SLA_CACHE_E4M3) {
    if (c.d == 128) run(attend_kernel<SLA_CACHE_E4M3, 128>, weight_kernel<SLA_CACHE_E4M3, 128>);
    else run(attend_kernel<SLA_CACHE_E4M3, 64>, weight_kernel<SLA_CACHE_E4M3, 64>);
  } else {
    if (c.d == 128) run(attend_kernel<SLA_CACHE_INT8, 128>, weight_kernel<SLA_CACHE_INT8, 128>);
    else run(attend_kernel<SLA_CACHE_INT8, 64>, weight_kernel<SLA_CACHE_INT8, 64>);
  }
  return cudaGetLastError() == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

}  // extern "C"
