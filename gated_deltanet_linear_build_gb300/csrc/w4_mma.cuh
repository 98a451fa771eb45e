// Shared by the units that multiply by 4-bit weights on the tensor cores.
#pragma once

#include "w4.cuh"

namespace gdn {
namespace w4 {

// Bounded waits of a whole warp: all lanes go on, or none does. One lane polls (32 that
// poll the same word take 170 cycles though it is ready); where a warp waits for two
// barriers, two lanes do.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned sleep_ns = 0) {
  const bool polls = (threadIdx.x & 31) == 0;
  if (__all_sync(0xffffffffu, !polls || tc::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, !polls || mbar_wait_abortable(bar, parity, abort, sleep_ns));
}
// Two barriers, by two lanes.
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  uint64_t* bar = lane == 0 ? a : b;
  const uint32_t parity = lane == 0 ? pa : pb;
  if (__all_sync(0xffffffffu, lane > 1 || tc::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, lane > 1 || mbar_wait_abortable(bar, parity, abort));
}
// The same in two halves: `ask` polls once, early, and `granted` waits where that was
// too early. (Beside the warps that widen codes a poll takes some 200 cycles to come
// back, be it ready or not.)
struct Asked {
  uint64_t* bar;
  uint32_t parity, ok;
};
__device__ __forceinline__ Asked ask(uint64_t* bar, uint32_t parity) {
  Asked q = {bar, parity, 1};
  if ((threadIdx.x & 31) == 0) q.ok = tc::mbar_try_wait(bar, parity);
  return q;
}
__device__ __forceinline__ bool granted(const Asked& q, volatile int* abort) {
  if (__all_sync(0xffffffffu, q.ok)) return true;
  return __all_sync(0xffffffffu, q.ok || mbar_wait_abortable(q.bar, q.parity, abort));
}
// K-major operand of 128-byte swizzled rows, 8-row groups 1,024 bytes apart.
__device__ __forceinline__ uint64_t x_desc(uint32_t addr) { return tc::smem_desc(addr, 16, 1024) | (2ull << 61); }
// kind::f16: f16 A and B, float32 D.
__device__ __forceinline__ uint32_t idesc_f16(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

// 32 codes of a row, in two groups with their scales (f16 pairs), as f16.
__device__ __forceinline__ void widen32(const uint4& c, uint32_t s0, uint32_t s1, uint32_t* out) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i % 4 == 0) codes8(w[i >> 2], out + i);
    const uint32_t sc = i < 8 ? s0 : s1;
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(out + i), *reinterpret_cast<const __half2*>(&sc));
    out[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Behind it nothing has to be seen (a release would wait for y's stores): no CTA ends
// before those that send to its shared memory are through.
__device__ __forceinline__ void cluster_end() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// A buffer of f16 is filled: the 128 threads that do arrive, the warp of the MMAs waits.
__device__ __forceinline__ void filled_arrive(int buffer) {
  asm volatile("bar.arrive %0, 160;" :: "r"(2 + buffer) : "memory");
}
__device__ __forceinline__ void filled_sync(int buffer) {
  asm volatile("bar.sync %0, 160;" :: "r"(2 + buffer) : "memory");
}

// A row's codes of a tile, and their scales.
struct Codes {
  uint4 a, b;
  uint32_t scales;
};
__device__ __forceinline__ Codes load_codes(const unsigned char* tile, int r) {
  Codes c;
  c.a = *reinterpret_cast<const uint4*>(tile + r * 16);
  c.b = *reinterpret_cast<const uint4*>(tile + kRows * 16 + r * 16);
  c.scales = *reinterpret_cast<const uint32_t*>(tile + kCodeBytes + r * 4);
  return c;
}
// As f16 to 32 columns of tensor memory (without the wait).
__device__ __forceinline__ void widen_codes(const Codes& c, uint32_t taddr) {
  const uint32_t s01 = half2_of_e4m3(c.scales), s23 = half2_of_e4m3(c.scales >> 16);
  uint32_t h[32];
  widen32(c.a, __byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232), h);
  widen32(c.b, __byte_perm(s23, 0, 0x1010), __byte_perm(s23, 0, 0x3232), h + 16);
  tc::tmem_st32_async(taddr, h);
}

// y = acc * 2^e in two steps, each within float32's range.
__device__ __forceinline__ float scaled(float acc, int e) {
  const int h = e >> 1;
  return acc * pow2(h) * pow2(e - h);
}
__device__ __forceinline__ void store(void* y, int f32, int64_t at, float v) {
  if (f32) static_cast<float*>(y)[at] = v;
  else static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

// Exponent of a power of two.
__device__ __forceinline__ int exponent(float power) { return (__float_as_int(power) >> 23) - 127; }
// Largest finite magnitude of 8 BF16 values, as bits.
__device__ __forceinline__ uint32_t finite_top8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return top;
}
// The exponent e under which a row with that largest magnitude becomes f16: x * 2^-e
// has its largest in [2^14, 2^15).
__device__ __forceinline__ int x_exponent(uint32_t top) { return top ? max(-120, (int)(top >> 7) - 127 - 14) : 0; }
__device__ __forceinline__ uint4 to_half8(const uint4& v, float down) {
  float f[8];
  unpack8(v, f);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 two = __floats2half2_rn(f[2 * i] * down, f[2 * i + 1] * down);
    h[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

}  // namespace w4

// A launch of clusters of `cluster` CTAs, else as launch_pdl's.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), int clusters, int cluster, int threads, size_t smem,
                                   cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
// Clusters of that size that the device holds at a time (0: unknown).
template <typename Kernel>
inline int clusters_of(Kernel kernel, int cluster, int threads, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms() / cluster * cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
  cudaGetLastError();
  return 0;
}

// What the general kernel takes for up to 64 tokens, in the time of a tile of 64 k there
// (some 0.13 us).
double w4_general_cost(int32_t T, int32_t N, int32_t K);

// The product for few tokens (w4_few.cu). False: not for these sizes.
bool launch_w4_few(const void* x, int64_t x_stride, const void* packed, void* y, int64_t y_stride,
                   int32_t y_type, int32_t T, int32_t N, int32_t K, cudaStream_t st, gdn_status_t* rc);

}  // namespace gdn
