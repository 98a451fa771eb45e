// Weights held in 4 bits: their layout, shared by the units that write and read it.
//
// w[n, k] = code * scale[n, k / 16] * power[n]: code one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
// (1 sign, 2 exponent, 1 fraction bit), scale e4m3 (not negative), power a power of two.
// code * scale has 6 significant bits and lies between 2^-10 and 2688 where it is not 0:
// exact as BF16 and as f16, so that a product's operands are what the weights stand for.
//
// Layout: tiles of 128 rows x 64 k (N and K are filled up with zeros), row-major by
// tiles, each one contiguous run of 4,608 bytes
//   codes   [2][128] x 16 bytes: 32 codes of a row, the even k in the low half of a byte;
//   scales  [128] x 4 bytes: the row's 4 groups,
// then the powers, float [rows]. A thread of the product owns a row: its 16-byte reads
// of neighbouring rows are neighbours, and a tile is one bulk copy.
#pragma once

#include <cuda_fp16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace w4 {

constexpr int kRows = 128, kK = 64, kGroup = 16;
constexpr int kCodeBytes = kRows * kK / 2;
constexpr int kTileBytes = kCodeBytes + kRows * kK / kGroup;
constexpr int kMinExp = -100, kMaxExp = 110;     // of a power

struct Shape {
  int rt, kb;                                    // tiles along N and K
  __host__ __device__ Shape(int N, int K) : rt((N + kRows - 1) / kRows), kb((K + kK - 1) / kK) {}
  __host__ __device__ size_t powers() const { return (size_t)rt * kb * kTileBytes; }
  __host__ __device__ size_t bytes() const { return powers() + (size_t)rt * kRows * 4; }
};

// 8 codes as pairs of f16, each byte's low half first. (The bytes by a move into four
// registers of 8 bits: shifts and masks take as long as the conversions again, 24
// cycles a warp instead of 12.)
__device__ __forceinline__ void codes8(uint32_t w, uint32_t* out) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// 8 values of a row from k on, zeros behind its end.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int k, int K) {
  if (k + 8 <= K) return ldg16(row + k);
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 8 && k + i < K; ++i)
    w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(row) + k + i) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace w4
}  // namespace gdn
