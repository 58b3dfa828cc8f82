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
// permuted so that a lane's loads are 16 bytes of one mean. Every CTA sends its maximum, then
// its sum, of a head to all others' shared memory; a block's probability is exp(s - max) *
// (1 / sum) with the cluster's max and sum, added in the same order everywhere, so equal
// means give equal sums wherever they are. A CTA sends its own top_n to the first one, which
// picks the blocks that fewer than top_n of all those are ahead of.
// Bound by its chain of dependent steps (lengths, table, means, three cluster barriers), not by
// bytes, and in large batches not by a pipe either: with 16 sequences of up to 65536 tokens
// the fp64 pipe is 4 % busy, the tensor pipe 14 %, 30 % of the issue slots are taken, and warps
// wait at barriers, for loads and for shared memory (profiles/cache_calls.md). Remote stores
// before a barrier instead of remote loads behind it, one exponential a score and integer
// comparisons are what shortened it. 5000 tokens, 16 heads a KV head: 11 us; 16 sequences of up
// to 65536: 33 us.
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void send(double* p, uint32_t rank, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(peer_addr(p, rank)), "d"(v) : "memory");
}
__device__ __forceinline__ void send(long long* p, uint32_t rank, long long v) {
  asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(peer_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void send(int* p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(d[0]), "+d"(d[1])
      : "d"(a), "d"(b));
}

// Past blocks of one CTA: a multiple of the eight that a warp takes.
__host__ __device__ inline int route_run(int n) { return ((n + kCluster - 1) / kCluster + 7) / 8 * 8; }

template <int D>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4)
    route_kernel(const CacheView c, const __nv_bfloat16* __restrict__ q, int T, const int32_t* __restrict__ lens,
                 const int32_t* __restrict__ n_new, int top_n, int32_t* sel) {
  constexpr int S = D / 4;  // k steps; lane k = lane % 4 holds d = S k .. S k + S - 1
  extern __shared__ double dyn[];  // scores [16][run + 1], then sums [run] (-1: no such page)
  __shared__ double qbar[2][S][32];
  __shared__ double max_of[2][kCluster][kHeads], sum_of[2][kCluster][kHeads];  // by turn and sender
  __shared__ double inv[kHeads];
  __shared__ long long cand_p[kCluster][kCacheMaxSel];  // the first CTA's: by sender
  __shared__ int cand_j[kCluster][kCacheMaxSel], cands[kCluster];
  __shared__ int s_cand, picked[kMaxBlocks / 32];
  const int bh = blockIdx.x / kCluster, b = bh / c.H_kv, hk = bh % c.H_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  wait_for_previous();
  let_next_start();
  bool bad = false;
  const int L = checked_len(lens, b, c.cap, &bad), nq = checked_new(n_new, b, T, &bad);
  if (bad && tid == 0 && hk == 0 && rank == 0) report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCacheLen);
  const int n = nq > 0 ? max(0, L - nq) / kBlock : 0;
  int32_t* out = sel + (size_t)bh * top_n;
  if (n == 0) {  // the same for the whole cluster
    if (rank == 0 && tid < top_n) out[tid] = -1;
    return;
  }
  cluster_arrive();  // a CTA's shared memory may be written from when it has started: waited for below
  const int run = route_run(n), j0 = min(n, (int)rank * run), mine = min(n, j0 + run) - j0;
  const int pitch = run + 1;
  double *score = dyn, *sum = dyn + kHeads * pitch;
  if (tid == 0) s_cand = 0;
  if (rank == 0 && tid < kMaxBlocks / 32) picked[tid] = 0;

  const double inv_n = 1.0 / nq;
  int turn = 0;
  for (int h0 = 0; h0 < c.group; h0 += kHeads, turn ^= 1) {
    const int heads = min(kHeads, c.group - h0);
    // a warp's first eight blocks: their means are on the way while qbar is made
    float4 mean[S / 4];
    int page = -1;
    auto load_means = [&](int u) {
      const int j = u + (lane >> 2);
      page = j < mine ? checked_page(c, b, j0 + j) : -1;
      const float4* m =
          reinterpret_cast<const float4*>(c.k_mean + ((size_t)max(page, 0) * c.H_kv + hk) * D) + (lane & 3) * (S / 4);
#pragma unroll
      for (int s4 = 0; s4 < S / 4; ++s4) mean[s4] = page >= 0 ? m[s4] : make_float4(0.f, 0.f, 0.f, 0.f);
      if (h0 == 0 && (lane & 3) == 0 && j < mine) sum[j] = page >= 0 ? 0.0 : -1.0;
    };
    load_means(warp * 8);
    // qbar of head h, element d, where the tensor step wants it: [h / 8][d % S][4 (h % 8) + d / S]
    for (int i = tid; i < kHeads * (D / 8); i += kThreads) {
      const int h = i / (D / 8), d = i % (D / 8) * 8;
      double x[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
      if (h < heads) {
        const __nv_bfloat16* rows = q + ((size_t)(b * c.H + hk * c.group + h0 + h) * T) * D + d;
#pragma unroll 4
        for (int t = 0; t < nq; ++t) {
          const uint4 w = *reinterpret_cast<const uint4*>(rows + (size_t)t * D);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16(ws[e]);
            x[2 * e] += (double)f.x;
            x[2 * e + 1] += (double)f.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= inv_n;
          // every score of the head is to be NaN then, not one infinity beside means of one sign
          if (isinf(x[e])) x[e] = __longlong_as_double(0x7ff8000000000000ll);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) qbar[h >> 3][(d + e) % S][4 * (h & 7) + (d + e) / S] = x[e];
    }
    __syncthreads();
    for (int u = warp * 8; u < mine; u += kWarps * 8) {
      if (u >= kWarps * 8) load_means(u);
      double acc[2][2][2] = {};  // group of eight heads, even and odd steps apart
#pragma unroll
      for (int s4 = 0; s4 < S / 4; ++s4) {
        const float e[4] = {mean[s4].x, mean[s4].y, mean[s4].z, mean[s4].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_f64(acc[0][i & 1], qbar[0][4 * s4 + i][lane], (double)e[i]);
          if (heads > 8) mma_f64(acc[1][i & 1], qbar[1][4 * s4 + i][lane], (double)e[i]);
        }
      }
      // element e: head 8 i + lane / 4, block u + 2 (lane % 4) + e
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = 2 * (lane & 3) + e;
        const bool there = __shfl_sync(0xffffffffu, page, 4 * at) >= 0;
        if (u + at < mine) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (8 * i < heads)
              score[(8 * i + (lane >> 2)) * pitch + u + at] =
                  there ? (acc[i][0][e] + acc[i][1][e]) * c.scale64 : -INFINITY;
        }
      }
    }
    __syncthreads();
    if (h0 == 0) cluster_wait();
    // a warp two heads: this CTA's maximum, to every CTA
    for (int h = warp; h < heads; h += kWarps) {
      double t = -INFINITY;
      for (int j = lane; j < mine; j += 32) t = fmax(t, score[h * pitch + j]);
      for (int o = 16; o > 0; o >>= 1) t = fmax(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (lane < kCluster) send(&max_of[turn][rank][h], lane, t);
    }
    cluster_sync();
    // the exponentials and their sum
    for (int h = warp; h < heads; h += kWarps) {
      double t = lane < kCluster ? max_of[turn][lane][h] : -INFINITY, part = 0.0;
      for (int o = 4; o > 0; o >>= 1) t = fmax(t, __shfl_xor_sync(0xffffffffu, t, o));
      t = __shfl_sync(0xffffffffu, t, 0);
      for (int j = lane; j < mine; j += 32) {
        const double s = score[h * pitch + j], e = s == -INFINITY ? 0.0 : exp(s - t);
        score[h * pitch + j] = e;
        part += e;
      }
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane < kCluster) send(&sum_of[turn][rank][h], lane, part);
    }
    cluster_sync();
    if (tid < heads) {
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) s += sum_of[turn][r][tid];
      inv[tid] = s > 0.0 ? 1.0 / s : s;  // 0: no page at all; NaN stays
    }
    __syncthreads();
    for (int j = tid; j < mine; j += kThreads) {
      double x = sum[j];
      if (x < 0.0) continue;
      for (int h = 0; h < heads; ++h) x += score[h * pitch + j] * inv[h];
      sum[j] = x;
    }
    __syncthreads();
  }
  // This CTA's best go to the first one. Sums that are not negative order like their bits: the
  // many comparisons are integer ones.
  const long long* key = reinterpret_cast<const long long*>(sum);
  for (int j = tid; j < mine; j += kThreads) {
    const long long x = key[j];
    if (!(sum[j] >= 0.0)) continue;  // no page, or NaN
    int ahead = 0;
    if (mine > top_n) {
#pragma unroll 8
      for (int i = 0; i < mine; ++i) ahead += (key[i] > x) | ((key[i] == x) & (i < j));
    }
    if (ahead < top_n) {
      const int at = atomicAdd(&s_cand, 1);
      send(&cand_p[rank][at], 0, x);
      send(&cand_j[rank][at], 0, j0 + j);
    }
  }
  __syncthreads();
  if (tid == 0) send(&cands[rank], 0, s_cand);
  cluster_sync();
  if (rank != 0) return;
  for (int i = tid; i < kCluster * top_n; i += kThreads) {
    const int r = i / top_n, at = i - r * top_n;
    if (at >= cands[r]) continue;
    const long long x = cand_p[r][at];
    const int j = cand_j[r][at];
    int ahead = 0;
    for (int s = 0; s < kCluster; ++s) {
      const int m = cands[s];
#pragma unroll 8
      for (int e = 0; e < m; ++e) ahead += (cand_p[s][e] > x) | ((cand_p[s][e] == x) & (cand_j[s][e] < j));
    }
    if (ahead < top_n) atomicOr(&picked[j >> 5], (int)(1u << (j & 31)));
  }
  __syncthreads();
  if (warp == 0) {  // in ascending order: a lane four words
    constexpr int W = kMaxBlocks / 32 / 32;
    int words[W], count = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      words[i] = picked[lane * W + i];
      count += __popc(words[i]);
    }
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int at = upto - count;
#pragma unroll
    for (int i = 0; i < W; ++i)
      for (uint32_t w = (uint32_t)words[i]; w != 0; w &= w - 1) out[at++] = (lane * W + i) * 32 + __ffs(w) - 1;
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    for (int i = all + lane; i < top_n; i += 32) out[i] = -1;
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
  auto bytes = [](int blocks) { return (kHeads * (route_run(blocks) + 1) + route_run(blocks)) * (int)sizeof(double); };
  auto run = [&](auto kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxBlocks)) != cudaSuccess)
      return SLA_ERR_CUDA;
    const cudaError_t e = launch_overlapped(kernel, dim3(c.B * c.H_kv * kCluster), kThreads, bytes(c.max_blocks),
                                            (cudaStream_t)stream, c, (const __nv_bfloat16*)q, (int)T, lens, n_new,
                                            (int)top_n, sel);
    return e == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
  };
  return c.d == 128 ? run(route_kernel<128>) : run(route_kernel<64>);
}
