// Weights to 4 bits and back (w4.cuh has the layout).
//
// For a row with largest magnitude a, a group with largest magnitude g, all of finite
// values:
//   power = 2^e, e the smallest in [-100, 110] with a <= 6 * 448 * 2^e,
//   scale = e4m3(g / power / 6), nearest even, at most 448 and, where g > 0, at least 2^-9,
//   code  = nearest of w / power / scale, ties to the even code, at most 6.
// w has 8 significant bits and a scale 4, so a quotient either is a border between codes
// or is off it by 2^-12 of itself: an approximate quotient, rounded to 16 bits before it
// is compared, decides as the exact one does.
#include <algorithm>

#include <cuda_fp8.h>

#include "w4.cuh"

namespace gdn {
namespace {
using namespace w4;

constexpr int kPackRows = 8;            // of a CTA
constexpr int kWarps = 8;               // (a row each at first)
constexpr int kThreads = kWarps * 32;

// Largest magnitude of 8 BF16 values, as their bits (infinities and NaN above all).
__device__ __forceinline__ uint32_t top8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) t = max(t, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  return t;
}
constexpr uint32_t kInf = 0x7f80u;

// Smallest e with top <= 2688 * 2^e, 2688 = 0.65625 * 2^12.
__device__ __forceinline__ int power_exp(float top) {
  if (!(top > 0.f)) return kMinExp;
  int ex;
  const float m = frexpf(top, &ex);
  return min(kMaxExp, max(kMinExp, ex - 12 + (m > 0.65625f ? 1 : 0)));
}

// Two values as codes, the first in the low half.
__device__ __forceinline__ uint32_t to_codes2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.u32.u8 %0, a;\n\t}"
      : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// To 16 significant bits.
__device__ __forceinline__ float round16(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80u) & ~0xffu);
}

// A group of 16: its codes to c, its scale.
__device__ __forceinline__ uint32_t pack_group(const uint4& a, const uint4& b, float down, uint32_t* c) {
  const uint32_t t = max(top8(a), top8(b));
  c[0] = c[1] = 0;
  if (t >= kInf) return 0x7f;            // an infinity or NaN: the group is NaN
  if (t == 0) return 0;
  const float q = __fdiv_rn(__uint_as_float(t << 16) * down, 6.f);
  const uint32_t scale = max(1u, (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3));
  const float sc = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale, __NV_E4M3)));
  const float inv = __frcp_rn(sc);
  float x[16];
  unpack8(a, x);
  unpack8(b, x + 8);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i >> 2] |= to_codes2(round16(x[2 * i] * down * inv), round16(x[2 * i + 1] * down * inv)) << (8 * (i & 3));
  return scale;
}

// A lane's place in 8 rows x 128 k: 32 k of a row, of which it has the tile's 16 bytes of
// codes; 8 lanes write 128 bytes in one piece.
struct Place {
  int r, k;                              // row of 8, first k of 128
  __device__ __forceinline__ explicit Place(int lane) : r(lane & 7), k((lane >> 3) * 32) {}
};

__global__ void __launch_bounds__(kThreads) w4_pack_kernel(const __nv_bfloat16* w, int64_t stride, int N, int K,
                                                           unsigned char* packed) {
  __shared__ uint32_t s_top[kPackRows];
  pdl_wait();
  pdl_trigger();
  const Shape s(N, K);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * kPackRows;                       // < rt * 128
  // The rows' largest, a warp each.
  uint32_t top = 0;
  if (row0 + warp < N) {
    const __nv_bfloat16* src = w + (int64_t)(row0 + warp) * stride;
    // (A group is two lanes', which both see its other half: one that holds an infinity is
    // left out.)
    auto seen = [&](uint4 v) {
      const uint32_t t = top8(v), group = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
      if (group < kInf) top = max(top, group);
    };
    int k = 0;
    for (; k + 1024 <= K; k += 1024) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ldg16(src + k + j * 256 + lane * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) seen(v[j]);
    }
    for (; k < K; k += 256) seen(k + lane * 8 < K ? load8(src, k + lane * 8, K) : make_uint4(0, 0, 0, 0));
    top = __reduce_max_sync(0xffffffffu, top);
  }
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  if (threadIdx.x < kPackRows)
    reinterpret_cast<float*>(packed + s.powers())[row0 + threadIdx.x] =
        pow2(power_exp(__uint_as_float(s_top[threadIdx.x] << 16)));
  const Place at(lane);
  const int row = row0 + at.r, r = row % kRows;
  const bool real = row < N;
  const __nv_bfloat16* src = w + (int64_t)row * stride;
  const float down = pow2(-power_exp(__uint_as_float(s_top[at.r] << 16)));
  unsigned char* const tiles = packed + (size_t)(row / kRows) * s.kb * kTileBytes;
#pragma unroll 1
  for (int k0 = warp * 128; k0 < s.kb * kK; k0 += kWarps * 128) {
    const int k = k0 + at.k;
    uint4 v[4];
    if (real && k + 32 <= K) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ldg16(src + k + j * 8);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = real && k + j * 8 < K ? load8(src, k + j * 8, K) : make_uint4(0, 0, 0, 0);
    }
    uint32_t c[4];
    const uint32_t lo = pack_group(v[0], v[1], down, c), hi = pack_group(v[2], v[3], down, c + 2);
    // The row's four scales of the tile: two lanes'.
    const uint32_t mine = lo | hi << 8, other = __shfl_xor_sync(0xffffffffu, mine, 8);
    if (k >= s.kb * kK) continue;        // (the last tile has no second beside it)
    unsigned char* const tile = tiles + (size_t)(k / kK) * kTileBytes;
    const int half = k % kK / 32;
    *reinterpret_cast<uint4*>(tile + half * (kRows * 16) + r * 16) = make_uint4(c[0], c[1], c[2], c[3]);
    if (half == 0) *reinterpret_cast<uint32_t*>(tile + kCodeBytes + r * 4) = mine | other << 16;
  }
}

__global__ void __launch_bounds__(kThreads) w4_unpack_kernel(const unsigned char* packed, int N, int K,
                                                             __nv_bfloat16* w, int64_t stride) {
  pdl_wait();
  pdl_trigger();
  const Shape s(N, K);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // A warp: 8 rows x 128 k, two rows at a time, of which a lane writes 16 bytes.
  const int row0 = blockIdx.x * kPackRows, side = lane >> 4, of = (lane & 15) * 8;
  const unsigned char* const tiles = packed + (size_t)(row0 / kRows) * s.kb * kTileBytes;
  const float* const powers = reinterpret_cast<const float*>(packed + s.powers());
#pragma unroll 1
  for (int k = warp * 128 + of; k < K; k += kWarps * 128) {
    const unsigned char* const tile = tiles + (size_t)(k / kK) * kTileBytes;
    const int half = k % kK / 32, g = k % kK / kGroup;
    uint32_t code[4], sc[4];
    float power[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {        // (the tile has rows behind the last)
      const int row = row0 + 2 * j + side, r = row % kRows;
      code[j] = __ldg(reinterpret_cast<const uint32_t*>(tile + half * (kRows * 16) + r * 16 + k % 32 / 2));
      sc[j] = __ldg(tile + kCodeBytes + r * 4 + g);
      power[j] = __ldg(powers + row);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + 2 * j + side;
      if (row >= N) break;
      const float scale = __half2float(__ushort_as_half((unsigned short)half2_of_e4m3(sc[j]))) * power[j];
      float x[8];
      uint32_t two[4];
      codes8(code[j], two);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(two + i));
        x[2 * i] = f.x * scale;
        x[2 * i + 1] = f.y * scale;
      }
      __nv_bfloat16* const dst = w + (int64_t)row * stride + k;
      if (k + 8 <= K)
        *reinterpret_cast<uint4*>(dst) = pack8(x);
      else
        for (int i = 0; i < 8 && k + i < K; ++i) dst[i] = __float2bfloat16_rn(x[i]);
    }
  }
}

}  // namespace

gdn_status_t launch_w4_pack(const void* w, int64_t stride, int32_t N, int32_t K, void* packed, cudaStream_t st) {
  const Shape s(N, K);
  return check_launch(launch_pdl(w4_pack_kernel, dim3((unsigned)(s.rt * (kRows / kPackRows))), dim3(kThreads), 0, st,
                                 static_cast<const __nv_bfloat16*>(w), stride, N, K,
                                 static_cast<unsigned char*>(packed)));
}

gdn_status_t launch_w4_unpack(const void* packed, int32_t N, int32_t K, void* w, int64_t stride, cudaStream_t st) {
  return check_launch(launch_pdl(w4_unpack_kernel, dim3((unsigned)((N + kPackRows - 1) / kPackRows)),
                                 dim3(kThreads), 0, st, static_cast<const unsigned char*>(packed), N, K,
                                 static_cast<__nv_bfloat16*>(w), stride));
}

}  // namespace gdn
