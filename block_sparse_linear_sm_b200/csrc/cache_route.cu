// sla_cache_route: the top-n mode's selection for one step over the paged cache.
//
// For every head h of a KV group: qbar = mean of the step's valid query rows, s_j = qbar .
// k_mean_j * scale over the past (full) blocks j, P = softmax(s); the group's sum of P ranks
// the blocks. All of it in fp64, as the whole-sequence router, so that only blocks whose
// sums agree to 1e-15 could change places.
#include "cache.cuh"

namespace sla {
namespace {

constexpr int kThreads = 256;

__device__ double block_reduce(double x, bool maximum, double* slots) {
  for (int o = 16; o > 0; o >>= 1) {
    const double y = __shfl_xor_sync(0xffffffffu, x, o);
    x = maximum ? fmax(x, y) : x + y;
  }
  __syncthreads();  // the previous use of slots is over
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = x;
  __syncthreads();
  x = slots[0];
  for (int i = 1; i < kThreads / 32; ++i) x = maximum ? fmax(x, slots[i]) : x + slots[i];
  return x;
}

// One CTA a (sequence, KV head). Dynamic shared memory: sums [n] and scores [n] of up to
// max_blocks past blocks, fp64.
__global__ void __launch_bounds__(kThreads) route_kernel(const CacheView c, const __nv_bfloat16* __restrict__ q, int T,
                                                         const int32_t* __restrict__ lens,
                                                         const int32_t* __restrict__ n_new, int top_n, int32_t* sel) {
  extern __shared__ double dyn[];
  __shared__ double qbar[128];
  __shared__ double slots[kThreads / 32];
  __shared__ int s_best;
  const int b = blockIdx.x / c.H_kv, hk = blockIdx.x % c.H_kv, tid = threadIdx.x, d = c.d;
  bool bad = false;
  const int L = checked_len(lens, b, c.cap, &bad), nq = checked_new(n_new, b, T, &bad);
  if (bad && tid == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
  const int n = nq > 0 ? max(0, L - nq) / kBlock : 0;
  int32_t* out = sel + (size_t)blockIdx.x * top_n;
  double *sum = dyn, *score = dyn + c.max_blocks;
  for (int j = tid; j < n; j += kThreads) sum[j] = 0.0;
  for (int g = 0; g < c.group; ++g) {
    const __nv_bfloat16* rows = q + ((size_t)(b * c.H + hk * c.group + g) * T) * d;
    __syncthreads();
    if (tid < d) {
      double a = 0.0;
      for (int t = 0; t < nq; ++t) a += (double)__bfloat162float(rows[(size_t)t * d + tid]);
      qbar[tid] = nq > 0 ? a / nq : 0.0;
    }
    __syncthreads();
    double top = -INFINITY;
    for (int j = tid; j < n; j += kThreads) {
      const int page = checked_page(c, b, j);
      double s = -INFINITY;
      if (page >= 0) {
        const float4* m = reinterpret_cast<const float4*>(c.k_mean + ((size_t)page * c.H_kv + hk) * d);
        s = 0.0;
        for (int e = 0; e < d / 4; ++e) {
          const float4 x = m[e];
          s += qbar[4 * e] * x.x + qbar[4 * e + 1] * x.y + qbar[4 * e + 2] * x.z + qbar[4 * e + 3] * x.w;
        }
        s *= (double)c.scale;
      }
      score[j] = s;
      top = fmax(top, s);
    }
    top = block_reduce(top, true, slots);
    double part = 0.0;
    for (int j = tid; j < n; j += kThreads) {
      score[j] = score[j] == -INFINITY ? 0.0 : exp(score[j] - top);
      part += score[j];
    }
    part = block_reduce(part, false, slots);
    for (int j = tid; j < n; j += kThreads) sum[j] += part > 0.0 ? score[j] / part : 0.0;
  }
  // pages out of range are never picked
  for (int j = tid; j < n; j += kThreads) {
    const int p = c.table[(size_t)b * c.max_blocks + j];
    if (p < 0 || p >= c.n_pages) sum[j] = -1.0;
  }
  // top_n times the largest left (equal sums: the lower block), marked by -2
  int found = 0;
  for (; found < top_n; ++found) {
    double best = -1.0;
    int at = 1 << 30;
    __syncthreads();
    for (int j = tid; j < n; j += kThreads)
      if (sum[j] > best) {
        best = sum[j];
        at = j;
      }
    const double top = block_reduce(best, true, slots);
    if (top <= -1.0) break;
    if (tid == 0) s_best = 1 << 30;
    __syncthreads();
    if (best == top) atomicMin(&s_best, at);
    __syncthreads();
    if (tid == 0) sum[s_best] = -2.0;
  }
  __syncthreads();
  if (tid == 0) {
    int i = 0;
    for (int j = 0; j < n; ++j)
      if (sum[j] == -2.0) out[i++] = j;
    for (; i < top_n; ++i) out[i] = -1;
  }
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" sla_status sla_cache_route(const void* q, const sla_cache_config* cfg, const sla_cache* cache, int32_t T,
                                      const int32_t* lens, const int32_t* n_new, int32_t top_n, int32_t* sel,
                                      void* stream) {
  CacheView c;
  const sla_status st = check_cache(cfg, cache, &c);
  if (st != SLA_OK) return st;
  if (!q || !lens || !sel || !c.k_mean || T < 1 || top_n < 1) return SLA_ERR_INVALID_ARG;
  if (((uintptr_t)q % 16) || ((uintptr_t)lens % 4) || ((uintptr_t)n_new % 4) || ((uintptr_t)sel % 4))
    return SLA_ERR_INVALID_ARG;
  if (T > kCacheMaxT || top_n > kCacheMaxSel) return SLA_ERR_UNSUPPORTED;
  const int bytes = 2 * c.max_blocks * (int)sizeof(double);
  if (cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           2 * kMaxBlocks * (int)sizeof(double)) != cudaSuccess)
    return SLA_ERR_CUDA;
  route_kernel<<<c.B * c.H_kv, kThreads, bytes, (cudaStream_t)stream>>>(c, (const __nv_bfloat16*)q, T, lens, n_new,
                                                                        top_n, sel);
  return cudaGetLastError() == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}
