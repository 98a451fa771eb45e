// Rotary positions, alone and fused with the append of k and v to an 8-bit
// paged cache.
//
// Pair i of a head at position p turns by the angle 2 pi frac(p phase_i), with
// phase_i = f_i / (2 pi) turns per token held as a 64-bit fixed-point fraction.
// The product wraps modulo 2^64, which IS the reduction to one turn: exact for
// every 32-bit position, where a float32 product p f_i is off by 0.06 rad at a
// million tokens. Its top 32 bits are the angle. BF16 results take the hardware's
// sine and cosine of it as a signed fraction of a turn, which are within 2^-21 on
// [-pi, pi]. 8-bit codes, where that moved one in some ten thousand to its
// neighbour, take the quadrant and the Taylor series on [-pi/4, pi/4] (to x^9 and
// x^10: below 2^-29), right to float32's last bits: 16,384 tokens of 8 heads of
// 128 appended take 65.1 us instead of 63.2. (In rotary alone, 32 + 8 heads:
// 53.6 instead of 52.0.)
//
// Measured: rotation of 16,384 tokens, 32 + 8 heads of 128, 336 MB: 52.0 us, 6.46
// TB/s, 95% of the copy rate; with the append of 8 heads of K and V, 370 MB: 65.1
// us, 84%.
//
// Both kernels are one pass over memory. A thread owns two 8-element vectors
// of a head (the two halves of its 8 pairs) and keeps its 8 sines and cosines
// in registers over kHeads heads, all of whose loads are issued first.
#include <algorithm>

#include <cuda_fp8.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kRotThreads = 256;
constexpr int kHeads = 4;               // heads per thread

struct RotArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;   // elements per token
  const int32_t* positions;
  const uint64_t* phases;
  int T, Hq, Hk, log_j, rot;            // d = 16 << log_j
  float scale;
  int interleaved, inverse;
};

// Element offsets of vector pair j of a head: the pairs of a rotated unit in
// the half layout lie rot / 2 apart; otherwise 16 elements are contiguous.
__device__ __forceinline__ void unit_offsets(int j, int rot, int interleaved, int& oa, int& ob) {
  const bool split = !interleaved && j * 16 < rot;
  oa = split ? j * 8 : j * 16;
  ob = split ? rot / 2 + j * 8 : j * 16 + 8;
}

__device__ __forceinline__ void load_phases(const uint64_t* phases, int j, uint64_t (&ph)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2*>(phases + j * 8) + i);
    ph[2 * i] = v.x;
    ph[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint32_t turn_of(uint64_t phase, int pos) {
  return (uint32_t)(((uint64_t)(int64_t)pos * phase) >> 32);
}

// Cosines and sines by the hardware (BF16 results).
__device__ __forceinline__ void angles(const uint64_t (&ph)[8], int pos, float scale, int inverse,
                                       float (&co)[8], float (&si)[8]) {
  constexpr float kTurn = 1.4629180792671596e-09f;     // 2 pi / 2^32
  const float ss = inverse ? -scale : scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s, c;
    __sincosf((float)(int32_t)turn_of(ph[i], pos) * kTurn, &s, &c);
    co[i] = c * scale;
    si[i] = s * ss;
  }
}

// The same of the first N phases (N even) to float32's last bits, two angles at a
// time for the packed instructions.
template <int N>
__device__ __forceinline__ void exact_angles(const uint64_t (&ph)[8], int pos, float scale, float (&co)[N],
                                             float (&si)[N]) {
  constexpr float kTurn = 1.4629180792671596e-09f;     // 2 pi / 2^32
  auto both = [](float v) { return make_float2(v, v); };
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    uint32_t quadrant[2];
    float r[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t turn = turn_of(ph[i + e], pos);
      quadrant[e] = (turn + 0x20000000u) >> 30;
      r[e] = (float)(int32_t)(turn - (quadrant[e] << 30));
    }
    const float2 x = mul2(make_float2(r[0], r[1]), both(kTurn)), x2 = mul2(x, x);
    float2 a = fma2(x2, both(1.f / 362880.f), both(-1.f / 5040.f));
    float2 b = fma2(x2, both(-1.f / 3628800.f), both(1.f / 40320.f));
    a = fma2(x2, a, both(1.f / 120.f));
    b = fma2(x2, b, both(-1.f / 720.f));
    a = fma2(x2, a, both(-1.f / 6.f));
    b = fma2(x2, b, both(1.f / 24.f));
    a = fma2(mul2(x, x2), a, x);
    b = fma2(x2, b, both(-0.5f));
    b = fma2(x2, b, both(1.f));
    const float sn[2] = {a.x, a.y}, cs[2] = {b.x, b.y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t q = quadrant[e];
      si[i + e] = __uint_as_float(__float_as_uint(q & 1 ? cs[e] : sn[e]) ^ ((q & 2) << 30)) * scale;
      co[i + e] = __uint_as_float(__float_as_uint(q & 1 ? sn[e] : cs[e]) ^ (((q + 1) & 2) << 30)) * scale;
    }
  }
}

// The angles of a row's rot / 2 = N J pairs, N a lane of its J, brought to the lanes
// that turn: lane j < rot / 16 gets those of pairs 8 j to 8 j + 7. All lanes take part.
template <int N>
__device__ __forceinline__ void shared_angles(const uint64_t (&ph)[8], int pos, float scale, int j, int J,
                                              float (&co)[8], float (&si)[8]) {
  float c[N], s[N];
  exact_angles<N>(ph, pos, scale, c, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int from = (8 * j + i) / N & (J - 1);
    co[i] = __shfl_sync(0xffffffffu, c[i % N], from, J);
    si[i] = __shfl_sync(0xffffffffu, s[i % N], from, J);
  }
}

// x[0..8) and x[8..16) are the unit's two vectors.
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&co)[8],
                                         const float (&si)[8], int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * co[i] - b * si[i];
      x[2 * i + 1] = a * si[i] + b * co[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[i + 8];
      x[i] = a * co[i] - b * si[i];
      x[i + 8] = a * si[i] + b * co[i];
    }
  }
}

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  unpack8(a, x);
  unpack8(b, x + 8);
}

// Unit `u` of the rotation of q (heads [0, Hq)) and k (heads [Hq, Hq + Hk)):
// vector pair j of the kHeads heads of one group of one token.
__device__ __forceinline__ void rotate_unit(const RotArgs& p, int64_t u) {
  const int J = 1 << p.log_j;
  const int H = p.Hq + p.Hk, groups = (H + kHeads - 1) / kHeads;
  const int j = (int)(u & (J - 1));
  const int64_t rest = u >> p.log_j;
  const int64_t tok = rest / groups;
  if (tok >= p.T) return;
  const int h0 = (int)(rest - tok * groups) * kHeads;
  int oa, ob;
  unit_offsets(j, p.rot, p.interleaved, oa, ob);
  const bool turn = j * 16 < p.rot;
  const int d = 16 << p.log_j;
  uint4 a[kHeads], b[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h < H) {
      const __nv_bfloat16* src = h < p.Hq ? p.q + tok * p.q_stride + h * d
                                          : p.k + tok * p.k_stride + (h - p.Hq) * d;
      // Plain loads: the output may be the input itself.
      a[i] = *reinterpret_cast<const uint4*>(src + oa);
      b[i] = *reinterpret_cast<const uint4*>(src + ob);
    }
  }
  float co[8], si[8];
  if (turn) {
    uint64_t ph[8];
    load_phases(p.phases, j, ph);
    angles(ph, __ldg(p.positions + tok), p.scale, p.inverse, co, si);
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h < H) {
      __nv_bfloat16* dst = h < p.Hq ? p.q_out + tok * p.q_out_stride + h * d
                                    : p.k_out + tok * p.k_out_stride + (h - p.Hq) * d;
      if (turn) {
        float x[16];
        unpack16(a[i], b[i], x);
        rotate16(x, co, si, p.interleaved);
        a[i] = pack8(x);
        b[i] = pack8(x + 8);
      }
      *reinterpret_cast<uint4*>(dst + oa) = a[i];
      *reinterpret_cast<uint4*>(dst + ob) = b[i];
    }
  }
}

__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs p) {
  pdl_wait();
  pdl_trigger();
  rotate_unit(p, (int64_t)blockIdx.x * kRotThreads + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Append to the cache.
//
// One CTA per (page piece, heads, K or V): 32 KB of them (64 KB where one head of
// a block is that much) are held in registers between the reduction that gives
// the scales and the rounding, so k and v are read once, and enough bytes are
// in flight per SM; a token's sines serve all heads of the unit. The scale is the smallest power of
// two that brings the largest finite magnitude of the piece within 448 (for a
// rotated k with the headroom of the rotation, so that it follows from the
// inputs' exponents alone and no rounding can move it). Powers of two cost an
// 8-bit float nothing: only its exponent field moves. A block that already
// holds tokens keeps the larger of the two scales, and where it grew its older
// codes are rounded once more to the coarser grid of subnormals.
// ---------------------------------------------------------------------------
struct AppendArgs {
  RotArgs r;                            // q only: Hk = 0 in the rotation
  const __nv_bfloat16 *k, *v;
  int64_t k_stride, v_stride;
  const gdn_page_piece_t* pieces;
  const int32_t* num_pieces;
  int piece_cap, Hk, hg, head_groups, log_b, num_blocks, k_grow;
  uint8_t *kc, *vc;
  float *ks, *vs;
  int kv_ctas;
};

constexpr int kMinExp = -100;           // smallest exponent of a scale

// Smallest e with top <= 448 * 2^e, 448 = 0.875 * 2^9.
__device__ __forceinline__ int scale_exp(float top, int grow) {
  if (!(top > 0.f)) return kMinExp;
  int ex;
  const float m = frexpf(top, &ex);
  return max(kMinExp, ex - 9 + (m > 0.875f ? 1 : 0) + grow);
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint2 to_codes8(const float* x, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(__half(h));
}

// Largest magnitude of 16 BF16 values, as float bits (NaN and infinities above
// all); with `finite` they do not count.
__device__ __forceinline__ uint32_t max_bits(const uint4& a, const uint4& b, uint32_t top, bool finite) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t lo = (w[i] << 16) & 0x7fff0000u, hi = w[i] & 0x7fff0000u;
    if (finite) {
      if (lo >= 0x7f800000u) lo = 0;
      if (hi >= 0x7f800000u) hi = 0;
    }
    top = max(top, max(lo, hi));
  }
  return top;
}

// One unit: a page piece, K or V, `hg` heads. Row r of the unit is token r % B of
// head r / B; a thread's rows are 256 / J apart (J threads a row).
constexpr int kMaxHeads = 64;           // of a unit: 4 passes of 256 threads, 16 tokens x 4 threads
template <int kPasses>
__device__ __forceinline__ void append_piece(const AppendArgs& p, int unit, uint32_t* s_top, float* s_old,
                                             float* s_scale) {
  const int is_v = unit & 1;
  const int rest = unit >> 1;
  const int grp = rest % p.head_groups, pi = rest / p.head_groups;
  const int head0 = grp * p.hg, heads = min(p.hg, p.Hk - head0);
  const int tid = threadIdx.x;
  if (pi >= __ldg(p.num_pieces)) return;
  const int4 pc = __ldg(reinterpret_cast<const int4*>(p.pieces) + pi);
  const int block = pc.x, first = pc.y, len = pc.z, off = pc.w;
  const int B = 1 << p.log_b;
  // (Differences: the sums of arbitrary numbers may pass 32 bits.)
  if (block < 0 || block >= p.num_blocks || off < 0 || off >= B || len <= 0 || len > B - off || first < 0 ||
      first > p.r.T - len)
    return;
  const int J = 1 << p.r.log_j, d = 16 << p.r.log_j;
  const int j = tid & (J - 1), row0 = tid >> p.r.log_j;
  const int rows = kRotThreads >> p.r.log_j;
  const int rot = is_v ? 0 : p.r.rot;
  int oa, ob;
  unit_offsets(j, rot, p.r.interleaved, oa, ob);
  const __nv_bfloat16* src = (is_v ? p.v + (int64_t)first * p.v_stride
                                   : p.k + (int64_t)first * p.k_stride) + head0 * d;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  float* scale_at = (is_v ? p.vs : p.ks) + (int64_t)block * p.Hk + head0;
  uint4 a[kPasses], b[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * rows, t = r & (B - 1), h = r >> p.log_b;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (t < len && h < heads) {
      const __nv_bfloat16* at = src + t * stride + h * d;
      a[i] = ldg16(at + oa);
      b[i] = ldg16(at + ob);
    }
  }
  if (tid < heads) {
    s_top[tid] = 0;
    s_old[tid] = off > 0 ? scale_at[tid] : 0.f;
  }
  __syncthreads();
  // A warp's rows of one pass lie in one head (at most 8 rows, 16 tokens).
  auto reduce = [&](bool finite) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, max_bits(a[i], b[i], 0u, finite));
      const int h = (row0 + i * rows) >> p.log_b;
      if ((tid & 31) == 0 && h < heads) atomicMax(s_top + h, top);
    }
    __syncthreads();
  };
  reduce(false);
  bool special = false;                  // an infinity or NaN: count the finite ones
  for (int h = 0; h < heads; ++h) special |= s_top[h] >= 0x7f800000u;
  if (special) {
    __syncthreads();
    if (tid < heads) s_top[tid] = 0;
    __syncthreads();
    reduce(true);
  }
  if (tid < heads) {
    const int e = scale_exp(__uint_as_float(s_top[tid]), is_v ? 0 : p.k_grow);
    const float scale = fmaxf(pow2i(min(e, 127)), s_old[tid]);
    s_scale[tid] = scale;
    scale_at[tid] = scale;
  }
  __syncthreads();
  uint8_t* page = (is_v ? p.vc : p.kc) + ((int64_t)block * p.Hk + head0) * ((int64_t)B * d);
  if (off > 0) {
    // The tokens that the block held, on a scale that grew.
    for (int h = 0; h < heads; ++h) {
      if (s_scale[h] == s_old[h]) continue;
      const float ratio = s_old[h] / s_scale[h];
      uint32_t* held = reinterpret_cast<uint32_t*>(page + (int64_t)h * B * d);
      for (int i = tid; i < off * d / 4; i += kRotThreads) {
        uint32_t w = held[i], o = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float x = e4m3_value((w >> (8 * c)) & 0xffu) * ratio;
          o |= (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3) << (8 * c);
        }
        held[i] = o;
      }
    }
  }
  const bool turn = j * 16 < rot;
  // Where half or a quarter of a head turns, the row's other lanes help with the
  // angles (2,048 tokens, 64 of 256: 10.1 -> 9.3 us).
  const int share = rot * 2 == d ? 4 : rot * 4 == d ? 2 : 0;
  uint64_t ph[8];
  float co[8], si[8];
  if (share) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < share) ph[i] = __ldg(p.r.phases + j * share + i);
  } else if (turn) {
    load_phases(p.r.phases, j, ph);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * rows, t = r & (B - 1), h = r >> p.log_b;
    const bool here = t < len && h < heads;
    const bool other = i == 0 || (rows & (B - 1)) != 0;  // token than the pass before
    if (share) {
      if (!__any_sync(0xffffffffu, here)) continue;
      if (other) {
        const int pos = t < len ? __ldg(p.r.positions + first + t) : 0;
        if (share == 2) shared_angles<2>(ph, pos, p.r.scale, j, J, co, si);
        else shared_angles<4>(ph, pos, p.r.scale, j, J, co, si);
      }
    }
    if (here) {
      float x[16];
      unpack16(a[i], b[i], x);
      if (turn) {
        if (!share && other) exact_angles<8>(ph, __ldg(p.r.positions + first + t), p.r.scale, co, si);
        rotate16(x, co, si, p.r.interleaved);
      }
      const float inv = 1.f / s_scale[h];
      uint8_t* dst = page + ((int64_t)h * B + off + t) * d;
      *reinterpret_cast<uint2*>(dst + oa) = to_codes8(x, inv);
      *reinterpret_cast<uint2*>(dst + ob) = to_codes8(x + 8, inv);
    }
  }
}

// CTAs [0, kv_ctas): one unit of the append each, the longer work first; the
// others: rotation of q.
template <int kPasses>
__global__ void __launch_bounds__(kRotThreads, kPasses <= 4 ? 3 : 2) rotary_append_kernel(const AppendArgs p) {
  __shared__ uint32_t s_top[kMaxHeads];
  __shared__ float s_old[kMaxHeads], s_scale[kMaxHeads];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < p.kv_ctas)
    append_piece<kPasses>(p, (int)blockIdx.x, s_top, s_old, s_scale);
  else
    rotate_unit(p.r, (int64_t)((int)blockIdx.x - p.kv_ctas) * kRotThreads + threadIdx.x);
}

int64_t rotary_units(int T, int H, int log_j) {
  return ((int64_t)T * ((H + kHeads - 1) / kHeads)) << log_j;
}

RotArgs rot_args(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                 const int32_t* positions, const int64_t* phases, void* q_out,
                 int64_t q_out_stride, void* k_out, int64_t k_out_stride, int T, int Hq, int Hk,
                 int d, int rot, float scale, int interleaved, int inverse) {
  RotArgs r;
  r.q = static_cast<const __nv_bfloat16*>(q);
  r.k = static_cast<const __nv_bfloat16*>(k);
  r.q_out = static_cast<__nv_bfloat16*>(q_out);
  r.k_out = static_cast<__nv_bfloat16*>(k_out);
  r.q_stride = q_stride;
  r.k_stride = k_stride;
  r.q_out_stride = q_out_stride;
  r.k_out_stride = k_out_stride;
  r.positions = positions;
  r.phases = reinterpret_cast<const uint64_t*>(phases);
  r.T = T;
  r.Hq = Hq;
  r.Hk = Hk;
  r.log_j = __builtin_ctz((unsigned)d / 16u);
  r.rot = rot;
  r.scale = scale;
  r.interleaved = interleaved;
  r.inverse = inverse;
  return r;
}

}  // namespace

gdn_status_t launch_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const int32_t* positions, const int64_t* phases, void* q_out,
                           int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t T,
                           int32_t Hq, int32_t Hk, int32_t d, int32_t rot, float scale,
                           int32_t interleaved, int32_t inverse, cudaStream_t st) {
  const RotArgs r = rot_args(q, q_stride, k, k_stride, positions, phases, q_out, q_out_stride,
                             k_out, k_out_stride, T, Hq, Hk, d, rot, scale, interleaved, inverse);
  const int64_t ctas = (rotary_units(T, Hq + Hk, r.log_j) + kRotThreads - 1) / kRotThreads;
  if (ctas > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  return check_launch(launch_pdl(rotary_kernel, dim3((unsigned)ctas), dim3(kRotThreads), 0, st, r));
}

gdn_status_t launch_rotary_kv_append(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     const int32_t* positions, const int64_t* phases,
                                     const gdn_page_piece_t* pieces, const int32_t* num_pieces,
                                     int32_t piece_cap, void* q_out, int64_t q_out_stride,
                                     void* kc, void* vc, float* ks, float* vs, int32_t num_blocks,
                                     int32_t block_tokens, int32_t T, int32_t Hq, int32_t Hk,
                                     int32_t d, int32_t rot, float scale, int32_t interleaved,
                                     cudaStream_t st) {
  AppendArgs p;
  p.r = rot_args(q, q_stride, nullptr, 0, positions, phases, q_out, q_out_stride, nullptr, 0, T,
                 Hq, 0, d, rot, scale, interleaved, 0);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.pieces = pieces;
  p.num_pieces = num_pieces;
  p.piece_cap = piece_cap;
  p.Hk = Hk;
  p.log_b = __builtin_ctz((unsigned)block_tokens);
  p.num_blocks = num_blocks;
  // A rotation grows a coordinate by sqrt(2) at most, and `scale` multiplies it; the
  // values behind the rotated ones stay as they are, however small `scale` is.
  int grow = 0;
  if (rot > 0) {
    grow = 1;
    for (float s = 1.f; s < scale; s *= 2.f) ++grow;
    for (float s = 0.5f; s >= scale; s *= 0.5f) --grow;
    if (rot < d) grow = std::max(grow, 0);
  }
  p.k_grow = grow;
  p.kc = static_cast<uint8_t*>(kc);
  p.vc = static_cast<uint8_t*>(vc);
  p.ks = ks;
  p.vs = vs;
  const int64_t q_ctas = q ? (rotary_units(T, Hq, p.r.log_j) + kRotThreads - 1) / kRotThreads : 0;
  const int per_head = block_tokens * d / 16;                  // threads of one head's block
  p.hg = std::max(1, std::min(Hk, 4 * kRotThreads / per_head));
  p.head_groups = (Hk + p.hg - 1) / p.hg;
  const int64_t ctas = q_ctas + 2 * (int64_t)piece_cap * p.head_groups;
  if (ctas > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  if (ctas == 0) return GDN_OK;
  p.kv_ctas = 2 * piece_cap * p.head_groups;
  const int passes = (per_head * p.hg + kRotThreads - 1) / kRotThreads;
  auto kern = passes <= 1   ? rotary_append_kernel<1>
              : passes <= 2 ? rotary_append_kernel<2>
              : passes <= 4 ? rotary_append_kernel<4>
                            : rotary_append_kernel<8>;
  return check_launch(launch_pdl(kern, dim3((unsigned)ctas), dim3(kRotThreads), 0, st, p));
}

}  // namespace gdn
