// sla_cache_route: the top-n mode's selection for one step over the paged cache.
//
// For every head h of a KV group: qbar = mean of the step's valid query rows, s_j = qbar .
// k_mean_j * scale over the past (full) blocks j, P = softmax(s); the group's sum of P ranks
// the blocks. All of it in fp64, as the whole-sequence router, so that only blocks whose
// sums agree to 1e-15 could change places.
//
// One cluster of eight CTAs a (sequence, KV head), each with an eighth of the past blocks.
// The scores of 16 heads are products on the FP64 tensor path (mma m8n8k4): a warp takes
// eight blocks, whose means it reads once, for both groups of eight heads, the d order
// permuted so that a lane's loads are 16 bytes of one mean. The softmax's maximum and sum go
// through distributed shared memory; every CTA adds them in the same order, and a block's
// probability is exp(s - max) / sum with the cluster's max and sum, so equal means give equal
// sums wherever they are. A CTA then offers its own top_n, and a block is picked when fewer
// than top_n of all offered ones are ahead of it.
#include "cache.cuh"

namespace sla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kHeads = 16;                        // heads a pass

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ double peer_double(const double* p, uint32_t rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ int peer_int(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(d[0]), "+d"(d[1])
      : "d"(a), "d"(b));
}

// Past blocks of one CTA: a multiple of the eight that a warp takes.
__host__ __device__ inline int route_run(int n) { return ((n + kCluster - 1) / kCluster + 7) / 8 * 8; }

template <int D>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    route_kernel(const CacheView c, const __nv_bfloat16* __restrict__ q, int T, const int32_t* __restrict__ lens,
                 const int32_t* __restrict__ n_new, int top_n, int32_t* sel) {
  constexpr int S = D / 4;  // k steps; lane k = lane % 4 holds d = S k .. S k + S - 1
  extern __shared__ double dyn[];  // scores [16][run + 1], then sums [run]
  __shared__ double qbar[2][S][32];
  __shared__ double s_top[kHeads], s_sum[kHeads];
  __shared__ double cand_p[kCacheMaxSel];
  __shared__ int cand_j[kCacheMaxSel], s_cand, s_won;
  __shared__ double all_p[kCluster * kCacheMaxSel];
  __shared__ int all_j[kCluster * kCacheMaxSel];
  __shared__ uint8_t won[kCacheMaxSel];
  const int bh = blockIdx.x / kCluster, b = bh / c.H_kv, hk = bh % c.H_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  bool bad = false;
  const int L = checked_len(lens, b, c.cap, &bad), nq = checked_new(n_new, b, T, &bad);
  if (bad && tid == 0 && hk == 0 && rank == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
  const int n = nq > 0 ? max(0, L - nq) / kBlock : 0;
  int32_t* out = sel + (size_t)bh * top_n;
  if (n == 0) {  // the same for the whole cluster
    if (rank == 0 && tid < top_n) out[tid] = -1;
    return;
  }
  const int run = route_run(n), j0 = min(n, (int)rank * run), mine = min(n, j0 + run) - j0;
  const int pitch = run + 1;
  double *score = dyn, *sum = dyn + kHeads * pitch;
  for (int j = tid; j < mine; j += kThreads) sum[j] = 0.0;

  for (int h0 = 0; h0 < c.group; h0 += kHeads) {
    const int heads = min(kHeads, c.group - h0);
    // qbar of head h, element d, where the tensor step wants it: [h / 8][d % S][4 (h % 8) + d / S]
    for (int i = tid; i < kHeads * D; i += kThreads) {
      const int h = i / D, d = i % D;
      double a = 0.0;
      if (h < heads) {
        const __nv_bfloat16* rows = q + ((size_t)(b * c.H + hk * c.group + h0 + h) * T) * D + d;
        for (int t = 0; t < nq; ++t) a += (double)__bfloat162float(rows[(size_t)t * D]);
        a /= nq;
      }
      qbar[h >> 3][d % S][4 * (h & 7) + d / S] = a;
    }
    __syncthreads();
    for (int u = warp * 8; u < mine; u += kWarps * 8) {
      const int j = u + (lane >> 2);
      const int page = j < mine ? checked_page(c, b, j0 + j) : -1;
      const float4* m =
          reinterpret_cast<const float4*>(c.k_mean + ((size_t)max(page, 0) * c.H_kv + hk) * D) + (lane & 3) * (S / 4);
      double acc[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
#pragma unroll
      for (int s4 = 0; s4 < S / 4; ++s4) {
        const float4 x = page >= 0 ? m[s4] : make_float4(0.f, 0.f, 0.f, 0.f);
        const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_f64(acc[0], qbar[0][4 * s4 + i][lane], (double)e[i]);
          if (heads > 8) mma_f64(acc[1], qbar[1][4 * s4 + i][lane], (double)e[i]);
        }
      }
      // acc[i][e]: head 8 i + lane / 4, block u + 2 (lane % 4) + e
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = 2 * (lane & 3) + e;
        const bool there = __shfl_sync(0xffffffffu, page, 4 * at) >= 0;
        if (u + at < mine) {
          const double z = there ? 0.0 : -INFINITY;
          score[(lane >> 2) * pitch + u + at] = there ? acc[0][e] * (double)c.scale : z;
          if (heads > 8) score[(8 + (lane >> 2)) * pitch + u + at] = there ? acc[1][e] * (double)c.scale : z;
        }
      }
    }
    __syncthreads();
    // a warp two heads: maximum, then sum of exp, over the cluster's blocks
    for (int h = warp; h < heads; h += kWarps) {
      double top = -INFINITY;
      for (int j = lane; j < mine; j += 32) top = fmax(top, score[h * pitch + j]);
      for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) s_top[h] = top;
    }
    cluster_sync();
    for (int h = warp; h < heads; h += kWarps) {
      double top = lane < kCluster ? peer_double(&s_top[h], lane) : -INFINITY;
      for (int o = 4; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = __shfl_sync(0xffffffffu, top, 0);
      double part = 0.0;
      for (int j = lane; j < mine; j += 32) {
        const double s = score[h * pitch + j], e = s == -INFINITY ? 0.0 : exp(s - top);
        score[h * pitch + j] = e;
        part += e;
      }
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == 0) s_sum[h] = part;
    }
    cluster_sync();
    // every CTA adds the eight sums in the same order
    double* total = all_p;
    if (tid < heads) {
      double t = 0.0;
      for (uint32_t r = 0; r < kCluster; ++r) t += peer_double(&s_sum[tid], r);
      total[tid] = t;
    }
    __syncthreads();
    for (int j = tid; j < mine; j += kThreads) {
      double x = sum[j];
      for (int h = 0; h < heads; ++h) x += total[h] > 0.0 ? score[h * pitch + j] / total[h] : 0.0;
      sum[j] = x;
    }
    cluster_sync();  // s_top and s_sum are read; qbar, score and total are free
  }
  // pages out of range are never picked
  for (int j = tid; j < mine; j += kThreads) {
    const int p = c.table[(size_t)b * c.max_blocks + j0 + j];
    if (p < 0 || p >= c.n_pages) sum[j] = -1.0;
  }
  if (tid == 0) s_cand = s_won = 0;
  __syncthreads();
  // this CTA's best, in ascending block order
  for (int u = 0; u < mine; u += kThreads) {
    const int j = u + tid;
    int ahead = top_n;
    if (j < mine && sum[j] >= 0.0) {
      const double x = sum[j];
      ahead = 0;
      for (int i = 0; i < mine; ++i) ahead += sum[i] > x || (sum[i] == x && i < j);
    }
    const bool in = ahead < top_n;
    const uint32_t ins = __ballot_sync(0xffffffffu, in);
    // warps in turn, so that the offered blocks stay in order
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        const int at = s_cand + __popc(ins & ((1u << lane) - 1u));
        if (in) {
          cand_p[at] = sum[j];
          cand_j[at] = j0 + j;
        }
        __syncwarp();
        if (lane == 0) s_cand += __popc(ins);
      }
      __syncthreads();
    }
  }
  cluster_sync();
  for (int i = tid; i < kCluster * top_n; i += kThreads) {
    const uint32_t r = i / top_n;
    const int at = i % top_n;
    const bool there = at < peer_int(&s_cand, r);
    all_p[i] = there ? peer_double(&cand_p[at], r) : -1.0;
    all_j[i] = there ? peer_int(&cand_j[at], r) : kMaxBlocks;
  }
  __syncthreads();
  const int offered = s_cand;
  for (int i = tid; i < offered; i += kThreads) {
    int ahead = 0;
    for (int e = 0; e < kCluster * top_n; ++e)
      ahead += all_p[e] > cand_p[i] || (all_p[e] == cand_p[i] && all_j[e] < cand_j[i]);
    won[i] = ahead < top_n;
    if (won[i]) atomicAdd(&s_won, 1);
  }
  __syncthreads();
  cluster_sync();
  int before = 0, count = 0;
  for (uint32_t r = 0; r < kCluster; ++r) {
    const int x = peer_int(&s_won, r);
    before += r < rank ? x : 0;
    count += x;
  }
  for (int i = tid; i < offered; i += kThreads) {
    if (!won[i]) continue;
    int at = before;
    for (int e = 0; e < i; ++e) at += won[e];
    out[at] = cand_j[i];
  }
  if (rank == 0)
    for (int i = count + tid; i < top_n; i += kThreads) out[i] = -1;
  cluster_sync();  // no CTA leaves while another reads its counts
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
  auto bytes = [](int blocks) { return (kHeads * (route_run(blocks) + 1) + route_run(blocks)) * (int)sizeof(double); };
  auto run = [&](auto kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxBlocks)) != cudaSuccess)
      return SLA_ERR_CUDA;
    kernel<<<c.B * c.H_kv * kCluster, kThreads, bytes(c.max_blocks), (cudaStream_t)stream>>>(
        c, (const __nv_bfloat16*)q, T, lens, n_new, top_n, sel);
    return cudaGetLastError() == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
  };
  return c.d == 128 ? run(route_kernel<128>) : run(route_kernel<64>);
}
