// y = x W^T over weights in 4 bits (w4.cuh), for one token to thousands.
//
// W is the 128-row operand of the tensor core, tokens its columns, so that a single
// token and a full tile of them are one kernel:
//
//   D[n, t] += A[n, k] B[t, k],   A = code * scale (f16, exact), B = x (f16),
//   y[t, n] = D[n, t] * power[n] * 2^(exponent of x's row t).
//
// * The codes never become a tile in shared memory: a thread owns a row of W, turns 64
//   codes a step into f16 (a conversion and a product a pair) and stores them to tensor
//   memory, where the tensor core takes A from. Through shared memory the same f16 would
//   be written and read at 83 bytes a cycle each, beside the codes' own 47: more than
//   the 128 there are.
// * x becomes f16 in a kernel before, scaled by a power of two for each row (BF16's 8
//   bits fit f16's 11; the scale makes up for its range), and is left in the very layout
//   of the tensor core's shared-memory operand, so that a stage of it is one bulk copy.
// * All (row tile, token tile)s times their k steps form one line, cut into pieces, one a
//   CTA: of whole tiles where that leaves few SMs without work, else equal ones. A tile
//   that a cut divides is left as float32 parts, which the CTA that comes last to it adds
//   up in a fixed order (equal inputs give equal bits).
//
// Bound: up to some 300 tokens the weights' bytes, then the tensor cores.
//   tokens x N x K          us   floor
//     32 x 131,072 x 4,096   68     47   4.7 TB/s
//     48 x 12,288 x 4,096    15      4   one tile a CTA: its 64 steps of 0.13 us, and 8 us
//                                        around them (x's kernel, the first codes, results)
//    512 x 4,096 x 8,192     44     18
//  2,048 x 4,096 x 8,192    115     72   1.19 PFLOP/s: a tile of 64 k takes 512 cycles of the
//                                        tensor core, some 200 go by beside them; results
//                                        are not taken while the next tile runs (one
//                                        accumulator of 256 columns beside W's f16)
//  2,048 x 16,384 x 4,096   220    143
#include <algorithm>
#include <cmath>

#include "w4_mma.cuh"

namespace gdn {
namespace {
using namespace w4;

constexpr int kThreads = 512;
constexpr int kMaxTokens = 256;        // of a tile
constexpr int kWBytes = 92160;         // ring of codes
constexpr int kXBytes = 131072;        // ring of x
constexpr int kMaxXStages = 8;
constexpr int kMinTiles = 4;           // of a CTA that has parts of results alone

// A step is S tiles of 64 k of a row tile: one stage of codes, one buffer of f16 in
// tensor memory, one round of the warp that issues the MMAs. A round costs some 250
// cycles beside its MMAs (16 cycles each for up to 32 tokens, 32 for 64, 128 for 256), so
// that few tokens take longer steps. Where tokens are many a stage of x is one tile.
template <int S>
struct Cfg {
  static constexpr int w_stages = kWBytes / (S * kTileBytes);
  static constexpr int x_tiles = S == 4 ? 4 : 1;               // of a stage of x
  static constexpr int a_cols = S * 32;
  static constexpr int a_bufs = S == 4 ? 3 : 4;
  static constexpr int a_first = 512 - a_bufs * a_cols;        // columns before: accumulators
};

constexpr int kJoin = 48;              // units' time
struct Plan {
  int rt, kb, tt, nt, nr;              // tiles along N, K and T; tokens a tile, and rows of x
  int line, grid, cut;                 // CTAs that share the line; CTAs; a piece's end divides by cut
  int64_t units;                       // tiles of 128 x 64 x nt
  Plan(int T, int N, int K) {
    const Shape s(N, K);
    rt = s.rt;
    kb = s.kb;
    tt = (T + kMaxTokens - 1) / kMaxTokens;
    nt = ((T + tt - 1) / tt + 15) / 16 * 16;
    nr = tt == 1 ? (T + 7) / 8 * 8 : nt;
    units = (int64_t)rt * tt * kb;
    // A unit is 0.2 to 0.3 us. The CTA that joins a tile reads its parts at the pace of one
    // SM, some two units' time each, so that a piece is of 1.5 sqrt(kb) at least
    // (1,262 x 128 x 9,520: 70 -> 45 us, of 4: 70).
    const int64_t sms = num_sms(), tiles = (int64_t)rt * tt, least = std::max(kMinTiles, (int)std::sqrt(2.25 * kb));
    line = (int)std::max<int64_t>(1, std::min(sms, units / least));
    // Whole tiles leave SMs without work, but nothing to join, which takes as long as 22 (80
    // tokens) to 44 units (256), or 48 of the shorter ones of up to 64 tokens: 500 x 8,192 x
    // 4,096 45 us divided and 36 whole, 512 x 4,096 x 8,192 48 and 57.
    const int64_t rounds = (tiles + sms - 1) / sms;
    const bool whole = rounds * kb - (units + line - 1) / line <= (nt <= 64 ? kJoin : 12 + nt / 8);
    cut = whole ? kb : 1;
    grid = whole ? (int)((tiles + rounds - 1) / rounds) : line;
  }
};
// Offsets in the workspace. A workspace for T tokens serves fewer ones: its parts are
// as large as any number of tokens up to T takes them.
struct Layout {
  size_t x, exps, counters, partials, total;
  Layout(int T, int N, int K) {
    const Plan p(T, N, K);
    const size_t tokens = (size_t)T + 16 * (size_t)p.tt;
    x = 0;
    exps = x + tokens * p.kb * 128;
    counters = exps + (tokens * 4 + 255) / 256 * 256;
    partials = counters + ((size_t)p.rt * p.tt * 4 + 255) / 256 * 256;
    total = partials + (size_t)p.line * 2 * kRows * 4 * std::min(kMaxTokens, (T + 15) / 16 * 16);
  }
};

struct Args {
  const unsigned char* packed;
  const float* powers;
  const unsigned char* x;
  const int* exps;
  int* counters;
  float* partials;
  void* y;
  int64_t y_stride, units;
  int T, N, kb, tt, nt, nr, x_stages, f32, cut;
};

// ---------------------------------------------------------------------------
// x as f16, in tiles of nr tokens x 64 k: 128-byte rows, their 16-byte chunks swizzled.
// ---------------------------------------------------------------------------
// A thread keeps its values between the row's largest and their rounding: one round of
// loads. (Rows of more than 8,192 values are read again; twice as many kept: 2,048 x 4,096 x
// 8,192 116 -> 119 us, 2,048 x 4,096 x 16,384 216 -> 214.)
constexpr int kXThreads = 512, kXKept = 2;
__global__ void __launch_bounds__(kXThreads) w4_x_kernel(const __nv_bfloat16* x, int64_t stride, int K, int nr, int kb,
                                                         unsigned char* out, int* exps, int* counters, int tiles) {
  __shared__ uint32_t s_top[kXThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x;
  for (int64_t i = (int64_t)t * kXThreads + tid; i < tiles; i += (int64_t)gridDim.x * kXThreads) counters[i] = 0;
  const __nv_bfloat16* row = x + (int64_t)t * stride;
  uint4 kept[kXKept];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kXKept; ++i) kept[i] = load8(row, (i * kXThreads + tid) * 8, K);
#pragma unroll
  for (int i = 0; i < kXKept; ++i) top = max(top, finite_top8(kept[i]));
  for (int k = (kXKept * kXThreads + tid) * 8; k < K; k += kXThreads * 8) top = max(top, finite_top8(load8(row, k, K)));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kXThreads / 32; ++i) top = max(top, s_top[i]);
  const int e = x_exponent(top);
  const float down = pow2(-e);
  if (tid == 0) exps[t] = e;
  const int j = t / nr, r = t % nr;
  unsigned char* at = out + ((size_t)j * kb * nr + r) * 128;
  auto put8 = [&](int k, const uint4& v) {
    const int c = k % kK / 8;
    *reinterpret_cast<uint4*>(at + (size_t)(k / kK) * nr * 128 + ((c ^ (r & 7)) << 4)) = to_half8(v, down);
  };
#pragma unroll
  for (int i = 0; i < kXKept; ++i)
    if ((i * kXThreads + tid) * 8 < kb * kK) put8((i * kXThreads + tid) * 8, kept[i]);
  for (int k = (kXKept * kXThreads + tid) * 8; k < kb * kK; k += kXThreads * 8)
    put8(k, load8(row, k, K));
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------
struct Smem {
  static constexpr int o_x = 0;
  static constexpr int o_w = kXBytes;
  static constexpr int o_bar = o_w + kWBytes;
  static constexpr int max_w = kWBytes / (2 * kTileBytes), max_a = 4;
  static constexpr int n_bar = 2 * max_w + 2 * kMaxXStages + 2 * max_a + 4 + 4;     // (one is spare)
  static constexpr int o_misc = o_bar + n_bar * 8;       // tmem base, abort, last [2]
  static constexpr int o_exps = o_misc + 16;             // of a tile's tokens, for each result warp
  static constexpr int total = o_exps + 4 * kMaxTokens * 4;
};
static_assert(Smem::total <= 232448 && Smem::o_exps % 16 == 0, "shared memory of one CTA");

// A CTA's way along its piece of the line, in steps.
template <int S>
struct Walk {
  int b, left, kb;                     // tile in the row, tiles to go
  __device__ Walk(int64_t u0, int count, int kb) : b((int)(u0 % kb)), left(count), kb(kb) {}
  __device__ int tiles() const { return min(S, min(kb - b, left)); }
  // True where a row of tiles ends.
  __device__ bool pass(int m) {
    left -= m;
    b += m;
    if (b < kb) return false;
    b = 0;
    return true;
  }
};

// The CTA whose piece tile u of the line is in.
__device__ __forceinline__ int owner(const Args& p, int64_t u) {
  const int grid = gridDim.x;
  int k = (int)min((int64_t)grid - 1, u * grid / p.units);
  while (p.units * k / grid > u) --k;
  while (p.units * (k + 1) / grid <= u) ++k;
  return k;
}

// Adds up the parts of a tile, in the order of their CTAs. A warp takes every 16th
// column, a lane 4 rows of it; the loads of kCols columns and two parts are in flight.
__device__ __forceinline__ void join(const Args& p, int64_t tile) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = owner(p, tile * p.kb), c1 = owner(p, tile * p.kb + p.kb - 1);
  const int i = (int)(tile / p.tt), j = (int)(tile % p.tt);
  const int t0 = j * p.nt, cols = min(p.nt, p.T - t0), n = i * kRows + lane * 4;
  // The first CTA's part is its last tile's, unless its piece begins here.
  const int slot0 = p.units * c0 / gridDim.x < tile * p.kb ? 1 : 0;
  int e[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) e[q] = exponent(p.powers[n + q]);
  constexpr int kCols = 4, kStep = kThreads / 32;
  __threadfence();
  for (int t = warp; t < cols; t += kCols * kStep) {
    float4 v[kCols] = {};
#pragma unroll 4
    for (int k = c0; k <= c1; ++k) {
      const float* at = p.partials + (((size_t)k * 2 + (k == c0 ? slot0 : 0)) * p.nt + t) * kRows + lane * 4;
      float4 a[kCols];
#pragma unroll
      for (int m = 0; m < kCols; ++m)
        a[m] = t + m * kStep < cols ? __ldcg(reinterpret_cast<const float4*>(at + (size_t)m * kStep * kRows))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
        v[m].x += a[m].x;
        v[m].y += a[m].y;
        v[m].z += a[m].z;
        v[m].w += a[m].w;
      }
    }
#pragma unroll
    for (int m = 0; m < kCols; ++m) {
      const int tm = t + m * kStep;
      if (tm >= cols) break;
      const int64_t y = (int64_t)(t0 + tm) * p.y_stride + n;
      const int ex = __ldcg(p.exps + t0 + tm);
      const float a[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < p.N) store(p.y, p.f32, y + q, scaled(a[q], ex + e[q]));
    }
  }
}

template <int S>
__global__ void __launch_bounds__(kThreads, 1) w4_linear_kernel(const Args p) {
  using C = Cfg<S>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* w_full = reinterpret_cast<uint64_t*>(smem + Smem::o_bar);
  uint64_t* w_empty = w_full + C::w_stages;
  uint64_t* x_full = w_empty + C::w_stages;
  uint64_t* x_empty = x_full + kMaxXStages;
  uint64_t* a_full = x_empty + kMaxXStages;
  uint64_t* a_empty = a_full + C::a_bufs;
  uint64_t* d_full = a_empty + C::a_bufs;  // [2]
  uint64_t* d_empty = d_full + 2;        // [2]
  uint64_t* parted = d_empty + 2;        // [2]: the result warps have stored a part, one for each part
  uint64_t* drained = parted + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Smem::o_misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Smem::o_misc + 4);
  volatile int* s_last = reinterpret_cast<volatile int*>(smem + Smem::o_misc + 8);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nd = 2 * p.nt <= C::a_first ? 2 : 1;    // accumulators
  const int grid = gridDim.x, c = blockIdx.x;
  const int64_t pieces = p.units / p.cut, u0 = pieces * c / grid * p.cut, u1 = pieces * (c + 1) / grid * p.cut;
  const int count = (int)(u1 - u0);

  if (tid == 0) {
    for (int i = 0; i < C::w_stages; ++i) {
      tc::mbar_init(w_full + i, 1);
      tc::mbar_init(w_empty + i, 4);
    }
    for (int i = 0; i < kMaxXStages; ++i) {
      tc::mbar_init(x_full + i, 1);
      tc::mbar_init(x_empty + i, 1);
    }
    for (int i = 0; i < C::a_bufs; ++i) {
      tc::mbar_init(a_full + i, 4);
      tc::mbar_init(a_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(d_full + i, 1);
      tc::mbar_init(d_empty + i, 4);
      tc::mbar_init(parted + i, 4);
    }
    tc::mbar_init(drained, 1);
    *s_abort = s_last[0] = s_last[1] = 0;
  }
  if (warp == 1) {
    tc::tmem_alloc(s_tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // All 512 columns begin at address 0. (A constant, so that the MMAs' operands stay in
  // uniform registers.)
  constexpr uint32_t tmem = 0;
  const uint32_t a_base = tmem + C::a_first;
  Walk<S> at(u0, count, p.kb);

  if (warp == 0) {
    // ======================= codes =================================================
    if (lane == 0) {
      // Token tiles share a row tile's codes. (Counted along: a division of 64 bits takes
      // longer than a tile.)
      int issued = 0, s = 0, j = (int)(u0 / p.kb % p.tt);
      uint32_t phase = 1;
      const unsigned char* row = p.packed + (size_t)(u0 / p.kb / p.tt) * p.kb * kTileBytes;
      auto post = [&]() {
        const int m = at.tiles();
        tc::mbar_arrive_expect_tx(w_full + s, m * kTileBytes);
        tc::bulk_g2s(smem + Smem::o_w + s * (S * kTileBytes), row + (size_t)at.b * kTileBytes, m * kTileBytes,
                     w_full + s);
        ++issued;
        if (++s == C::w_stages) {
          s = 0;
          phase ^= 1;
        }
        if (at.pass(m) && ++j == p.tt) {
          j = 0;
          row += (size_t)p.kb * kTileBytes;
        }
      };
      // (This role, the conversion and the MMAs do not wait for the kernel before: it does
      // not write the weights, and has waited for those that may have.)
      while (at.left > 0 && issued < C::w_stages) post();
      while (at.left > 0) {
        if (!mbar_wait_abortable(w_empty + s, phase, s_abort, 64)) break;
        post();
      }
      if (*s_abort)                      // copies in flight land before the CTA ends
        for (int i = max(0, issued - C::w_stages); i < issued; ++i)
          tc::mbar_wait(w_full + i % C::w_stages, (i / C::w_stages) & 1);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ======================= x =====================================================
    pdl_wait();
    pdl_trigger();
    if (lane == 0) {
      const int tile = p.nr * 128, stage = C::x_tiles * tile;
      int issued = 0, s = 0, j = (int)(u0 / p.kb % p.tt);
      uint32_t phase = 1;
      while (at.left > 0) {
        if (!mbar_wait_abortable(x_empty + s, phase, s_abort, 64)) break;
        const int m = min(C::x_tiles, at.tiles());
        // (The last tile's rows behind the last token are left as they are: columns of the
        // result that nobody reads. So are those between nr and nt.)
        const int bytes = m > 1 || p.tt == 1 ? m * tile : min(p.nr, (p.T - j * p.nt + 7) & ~7) * 128;
        tc::mbar_arrive_expect_tx(x_full + s, bytes);
        tc::bulk_g2s(smem + Smem::o_x + s * stage, p.x + ((size_t)j * p.kb + at.b) * tile, bytes, x_full + s);
        ++issued;
        if (++s == p.x_stages) {
          s = 0;
          phase ^= 1;
        }
        if (at.pass(m) && ++j == p.tt) j = 0;
      }
      if (*s_abort)
        for (int i = max(0, issued - p.x_stages); i < issued; ++i)
          tc::mbar_wait(x_full + i % p.x_stages, (i / p.x_stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA ===================================================
    const bool one = tc::elect_one();
    const uint32_t id = idesc_f16(p.nt);
    const uint64_t xd = x_desc(tc::smem_u32(smem + Smem::o_x));
    const int x_tile = p.nr * 128 / 16, x_stage = C::x_tiles * x_tile;
    int xs = 0, ab = 0, db = 0;
    uint32_t xp = 0, ap = 0, dp = 1;
    bool first = true, ok = true;
    while (ok && at.left > 0) {
      const int m = at.tiles();
      const bool last = at.pass(m) || at.left == 0;
      if (first) ok = warp_wait(d_empty + db, dp, s_abort);
      const uint32_t d = tmem + (db ? p.nt : 0);
#pragma unroll
      for (int i = 0; i < S; i += C::x_tiles) {
        if (i >= m) break;
        ok = ok && (i == 0 ? warp_wait2(x_full + xs, xp, a_full + ab, ap, s_abort) : warp_wait(x_full + xs, xp, s_abort));
        tc::fence_after_sync();
        if (!ok) break;
        if (one) {
          const int n = C::x_tiles == 1 ? 1 : m;
          const uint32_t a = a_base + ab * C::a_cols + i * 32;
          const uint64_t b = xd + (uint32_t)(xs * x_stage);
#pragma unroll 1
          for (int k = 0; k < n; ++k)
#pragma unroll
            for (int e = 0; e < kK / 16; ++e)
              tc::mma_bf16_tmem_a(d, a + k * 32 + e * 8, b + (uint32_t)(k * x_tile) + e * 2, id, !first || i + k + e > 0);
          tc::mma_commit(x_empty + xs);
          if (i + C::x_tiles >= m) {
            tc::mma_commit(a_empty + ab);
            if (last) tc::mma_commit(d_full + db);
          }
        }
        if (++xs == p.x_stages) {
          xs = 0;
          xp ^= 1;
        }
      }
      first = last;
      if (++ab == C::a_bufs) {
        ab = 0;
        ap ^= 1;
      }
      if (last && ++db == nd) {
        db = 0;
        dp ^= 1;
      }
    }
    // Nothing is in flight when tensor memory is freed.
    if (one) tc::mma_commit(drained);
    if (!tc::mbar_wait(drained, 0)) record_device_status(GDN_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ======================= codes to f16 ==========================================
    // Two warpgroups take turns; a thread has the row of its lane in tensor memory.
    const int r = (warp & 3) * 32 + lane;
    const uint32_t turn = (warp - 4) >> 2;
    int s = 0, ab = 0;
    uint32_t wp = 0, ap = 1;
    for (uint32_t i = 0; at.left > 0; ++i) {
      const int m = at.tiles();
      at.pass(m);
      if ((i & 1) == turn) {
        if (!warp_wait(w_full + s, wp, s_abort, 20)) break;
        if (!warp_wait(a_empty + ab, ap, s_abort, 20)) break;
        tc::fence_after_sync();
        // (One tile's instructions, looped over: those of a whole step do not stay in the
        // instruction cache beside the other roles'.)
        const unsigned char* tile = smem + Smem::o_w + s * (S * kTileBytes);
        uint32_t to = tc::tmem_warp_addr(a_base, ab * C::a_cols);
        Codes next = load_codes(tile, r);
#pragma unroll 1
        for (int k = m; k > 0; --k) {
          const Codes now = next;
          tile += kTileBytes;
          if (k > 1) next = load_codes(tile, r);
          widen_codes(now, to);
          to += 32;
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(a_full + ab);
          tc::mbar_arrive(w_empty + s);
        }
      }
      if (++s == C::w_stages) {
        s = 0;
        wp ^= 1;
      }
      if (++ab == C::a_bufs) {
        ab = 0;
        ap ^= 1;
      }
    }
  } else if (warp >= 12) {
    // ======================= results ===============================================
    pdl_wait();
    pdl_trigger();
    const int r = (warp & 3) * 32 + lane;
    int* s_exps = reinterpret_cast<int*>(smem + Smem::o_exps) + (warp & 3) * kMaxTokens;
    int64_t u = u0;
    for (int seg = 0; u < u1; ++seg) {
      const int64_t tile = u / p.kb;
      const int from = (int)(u - tile * p.kb), to = (int)min((int64_t)p.kb, from + (u1 - u));
      u += to - from;
      const int i = (int)(tile / p.tt), j = (int)(tile % p.tt);
      const int n = i * kRows + r, t0 = j * p.nt, cols = min(p.nt, p.T - t0);
      const bool whole = to - from == p.kb;
      const int e_n = exponent(p.powers[n]);
      int far = 0;                       // the largest exponent's size
      if (whole)
        for (int t = lane; t < cols; t += 32) {
          s_exps[t] = __ldcg(p.exps + t0 + t);
          far = max(far, abs(s_exps[t]));
        }
      far = __reduce_max_sync(0xffffffffu, far);
      if (!warp_wait(d_full + seg % nd, (seg / nd) & 1, s_abort, 200)) break;
      tc::fence_after_sync();
      const uint32_t d = tc::tmem_warp_addr(tmem, (seg % nd) * p.nt);
      // A CTA has two parts at most: of its first tile, and of its last.
      const int slot = from == 0 && seg > 0 ? 1 : 0;
      float* part = p.partials + ((size_t)c * 2 + slot) * p.nt * kRows;
      // Where all of the warp's scales are float32's own, one product applies one.
      const bool near = __all_sync(0xffffffffu, abs(e_n) + far <= 126);
      for (int t = 0; t < cols; t += 16) {
        float v[16];
        tc::tmem_ld16(d + t, v);
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k) part[(t + k) * kRows + r] = v[k];
          continue;
        }
        const int4* const e4 = reinterpret_cast<const int4*>(s_exps + t);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const int4 q = e4[k / 4];
          const int e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int m = 0; m < 4; ++m)
            v[k + m] = near ? v[k + m] * __int_as_float((e_n + 127 + e[m]) << 23) : scaled(v[k + m], e_n + e[m]);
        }
        const int left = n < p.N ? cols - t : 0;
        const int64_t at0 = (t0 + t) * p.y_stride + n;
        if (p.f32) {
          float* to = static_cast<float*>(p.y) + at0;
#pragma unroll
          for (int k = 0; k < 16; ++k, to += p.y_stride)
            if (k < left) *to = v[k];
        } else {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.y) + at0;
#pragma unroll
          for (int k = 0; k < 16; ++k, to += p.y_stride)
            if (k < left) *to = __float2bfloat16_rn(v[k]);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(d_empty + seg % nd);
      if (whole) continue;
      // Counted once all four warps have stored theirs. (Each part has a barrier of its own:
      // with two accumulators a warp may be through with both before another has stored the
      // first.)
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(parted + slot);
      if (warp == 12) {
        if (!warp_wait(parted + slot, 0, s_abort)) break;
        if (lane == 0) {
          __threadfence();
          if (atomicAdd(p.counters + tile, 1) == owner(p, tile * p.kb + p.kb - 1) - owner(p, tile * p.kb))
            s_last[from == 0] = 1;
        }
      }
    }
  }
  // Every role is here, done or given up.
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
  // Divided tiles, by the CTA that came last to them: its first tile, its last one.
  if (*s_abort) return;
  if (s_last[0]) join(p, u0 / p.kb);
  if (s_last[1]) join(p, (u1 - 1) / p.kb);
}

template <int S>
gdn_status_t launch_product(Args& a, int grid, cudaStream_t st) {
  static DeviceOnce once;
  const cudaError_t set = allow_smem(once, w4_linear_kernel<S>, Smem::total);
  if (set != cudaSuccess) return check_launch(set);
  a.x_stages = std::min(kMaxXStages, kXBytes / (Cfg<S>::x_tiles * a.nr * 128));
  return check_launch(launch_pdl(w4_linear_kernel<S>, dim3((unsigned)grid), dim3(kThreads), Smem::total, st, a));
}

}  // namespace

size_t w4_linear_workspace_bytes(int32_t T, int32_t N, int32_t K) {
  if (T == 0) return 256;
  const Plan p(T, N, K);
  // Tiles, and a CTA's units, are counted in 32 bits.
  if ((int64_t)p.rt * p.tt > 0x7fffffff || p.units / p.grid > 0x3fffffff) return 0;
  return Layout(T, N, K).total;
}

double w4_general_cost(int32_t T, int32_t N, int32_t K) {
  const Plan p(T, N, K);
  // The kernel for x and what begins and ends this one, the units, each tile's results.
  const int64_t tiles = (int64_t)p.rt * p.tt, rounds = (tiles + p.grid - 1) / p.grid;
  return 45 + 0.25 * T + (double)p.units / p.grid + (p.cut > 1 || p.kb == 1 ? 0 : kJoin) + rounds * (9 + 0.1 * T);
}

gdn_status_t launch_w4_linear(const void* x, int64_t x_stride, const void* packed, void* y, int64_t y_stride,
                              int32_t y_type, int32_t T, int32_t N, int32_t K, void* workspace, cudaStream_t st) {
  gdn_status_t few;
  if (launch_w4_few(x, x_stride, packed, y, y_stride, y_type, T, N, K, st, &few)) return few;
  const Plan pl(T, N, K);
  const Layout l(T, N, K);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Args a;
  a.packed = static_cast<const unsigned char*>(packed);
  a.powers = reinterpret_cast<const float*>(a.packed + Shape(N, K).powers());
  a.x = ws + l.x;
  a.exps = reinterpret_cast<const int*>(ws + l.exps);
  a.counters = reinterpret_cast<int*>(ws + l.counters);
  a.partials = reinterpret_cast<float*>(ws + l.partials);
  a.y = y;
  a.y_stride = y_stride;
  a.units = pl.units;
  a.T = T;
  a.N = N;
  a.kb = pl.kb;
  a.cut = pl.cut;
  a.tt = pl.tt;
  a.nt = pl.nt;
  a.nr = pl.nr;
  a.f32 = y_type == GDN_TYPE_F32;
  const gdn_status_t rc = check_launch(launch_pdl(
      w4_x_kernel, dim3((unsigned)T), dim3(kXThreads), 0, st, static_cast<const __nv_bfloat16*>(x), x_stride, (int)K,
      pl.nr, pl.kb, ws + l.x, reinterpret_cast<int*>(ws + l.exps), a.counters, pl.rt * pl.tt));
  if (rc != GDN_OK) return rc;
  return pl.nt <= 64 ? launch_product<4>(a, pl.grid, st) : launch_product<2>(a, pl.grid, st);
}

GDN_DEFINE_STATUS_GATHER(gather_status_w4_linear)

}  // namespace gdn
