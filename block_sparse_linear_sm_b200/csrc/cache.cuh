// The 8-bit paged cache: what its kernels share (the view of the buffers, the two code
// formats, the power-of-two scales, checked lengths and page numbers).
#pragma once
#include <cuda_fp16.h>

#include <utility>

#include "common.cuh"

namespace sla {

constexpr int kCacheMaxB = 1024;       // sequences: the attention kernel scans their lengths in shared memory
constexpr int kCacheMaxT = 64;         // query rows of a step and head
constexpr int kCacheMaxRows = 1024;    // query rows of a step and KV head
constexpr int kCacheMaxSel = 64;       // selected blocks: two list entries a lane
constexpr float kCacheMaxAbs = 1.329227995784915873e36f;  // 2^120: larger magnitudes are cut to it

// Buffers and sizes of one call (include/sla.h: sla_cache, sla_cache_config).
struct CacheView {
  uint8_t *k, *v;
  float *k_scale, *v_scale, *k_mean, *weight;
  const int32_t* table;
  int* status;
  int B, H, H_kv, group, d, n_pages, max_blocks, cap, kind;
  float scale;
  double scale64;  // the router's: 1 / sqrt(128) rounded to fp32 is off by 1.7e-8 of it
};

// Every kernel of the cache is launched so that it may start while the one before it in the
// stream still runs (programmatic dependent launch): it sets itself up, waits for that one to
// be complete before it touches global memory (but see scan_lines), and lets the next one start
// likewise.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

sla_status check_cache(const sla_cache_config* c, const sla_cache* m, CacheView* view);

// ---------------------------------------------------------------------------
// scales: exponent of the least power of two s >= 2^-110 with a <= top * s, top = 448
// (1.75 * 2^8, e4m3) or 127 (1.984375 * 2^6, int8); a is finite, 0 <= a <= 2^120
// ---------------------------------------------------------------------------
template <int KIND>
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127;  // a = 1.f * 2^e (a subnormal one ends at the lower limit)
  const uint32_t f = bits & 0x7fffffu;
  const int x = KIND == SLA_CACHE_E4M3 ? e - 8 + (f > 0x600000u) : e - 6 + (f > 0x7e0000u);
  return max(-110, min(120, x));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ---------------------------------------------------------------------------
// codes
// ---------------------------------------------------------------------------
// four codes of x0 .. x3 (already divided by the scale), x0 in the lowest byte
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3) {
  if (KIND == SLA_CACHE_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  // |x| <= 128: adding 1.5 * 2^23 rounds to an integer (ties to even) in the low mantissa bits
  const float big = 12582912.f;
  const uint32_t a = __float_as_uint(x0 + big), b = __float_as_uint(x1 + big);
  const uint32_t c = __float_as_uint(x2 + big), e = __float_as_uint(x3 + big);
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, e, 0x0040), 0x5410);
}

// four codes as fp16 pairs (lo: bytes 0 and 1), exactly: |e4m3| <= 448 and its subnormals are
// fp16 normals or subnormals; |int8| <= 128
template <int KIND>
__device__ __forceinline__ void decode4_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  if (KIND == SLA_CACHE_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    return;
  }
  // byte ^ 0x80 = code + 128 in the mantissa of 1024 + (code + 128); minus 1152
  const uint32_t u = c ^ 0x80808080u, a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <int KIND>
__device__ __forceinline__ void decode4(uint32_t c, float* x) {
  uint32_t a, b;
  decode4_f16<KIND>(c, a, b);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&b));
  x[0] = f.x;
  x[1] = f.y;
  x[2] = g.x;
  x[3] = g.y;
}

// largest magnitude of 16 codes, by pairs of 16-bit lanes (e4m3 magnitudes order like integers)
template <int KIND>
__device__ __forceinline__ float max_magnitude16(const uint4& c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t hi = 0, lo = 0x00ff00ffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = KIND == SLA_CACHE_E4M3 ? w[i] & 0x7f7f7f7fu : w[i] ^ 0x80808080u;
    const uint32_t a = u & 0x00ff00ffu, b = (u >> 8) & 0x00ff00ffu;
    hi = __vmaxu2(hi, __vmaxu2(a, b));
    if (KIND == SLA_CACHE_INT8) lo = __vminu2(lo, __vminu2(a, b));
  }
  const int top = (int)max(hi & 0xffffu, hi >> 16);
  if (KIND == SLA_CACHE_INT8) {
    const int low = (int)min(lo & 0xffffu, lo >> 16);
    return (float)max(top - 128, 128 - low);
  }
  float x[4];
  decode4<KIND>((uint32_t)top, x);
  return x[0];
}

// ---------------------------------------------------------------------------
// checked device-side arguments
// ---------------------------------------------------------------------------
// n, or 0 where it is not in 0 .. most (*bad set)
__device__ __forceinline__ int in_range(int n, int most, bool* bad) {
  if (n >= 0 && n <= most) return n;
  *bad = true;
  return 0;
}
// cached tokens of sequence b
__device__ __forceinline__ int checked_len(const int32_t* lens, int b, int cap, bool* bad) {
  return in_range(lens[b], cap, bad);
}
// valid query rows of sequence b
__device__ __forceinline__ int checked_new(const int32_t* n_new, int b, int T, bool* bad) {
  return n_new == nullptr ? T : in_range(n_new[b], T, bad);
}
// page of block j of sequence b, -1 (and reported) where the table's number is out of range
__device__ __forceinline__ int checked_page(const CacheView& c, int b, int j) {
  const int p = c.table[(size_t)b * c.max_blocks + j];
  if (p >= 0 && p < c.n_pages) return p;
  report(c.status, SLA_ERR_DEVICE_CHECK, kDetailCachePage);
  return -1;
}

}  // namespace sla
