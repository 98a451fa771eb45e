// y = x W^T over weights in 4 bits (w4.cuh) for at most 64 tokens: the steps of a
// decode loop, where the weights' bytes are the work and the rest is latency.
//
// The product itself is w4_linear.cu's: 128 rows of W become f16 in tensor memory, x is
// the operand in shared memory. What differs is everything around it, so that one launch
// does without a workspace:
//
// * A cluster of P CTAs shares a row tile, each with a slice of K of its own: the slice
//   of x stays in its shared memory for all row tiles. It comes by TMA, in the layout of
//   the tensor core's operand, and becomes f16 in its place, scaled by a power of two for
//   each token of the slice, while the first codes are on their way to tensor memory.
// * The P partial results of a token go straight to the shared memory of one of the CTAs
//   (every CTA has some of the tokens), which adds them up in a fixed order.
//
// Bound: latency; up to some tens of MB of weights that of setting up and of the tail, then
// that of a step's chain (place free, codes there, read, widened, stored, told), with
// HBM two thirds busy and no unit of the SM full. us (floor), as N x K: 4,096 x 8,192 for 1 token 10.8 (2.8), 16 11.8, 32 13.1;
// 5,003 x 1,111 for 7 6.5 (0.5); 131,072 x 4,096 for 1 61 (45).
#include <algorithm>

#include "tensor_map.cuh"
#include "w4_mma.cuh"

namespace gdn {
namespace {
using namespace w4;

// Warps: 0 copies codes, 1 issues the MMAs, 2 copies x, those from 4 on widen codes, in two
// warpgroups or three, the next four take the results; 1 to 3 and the last five make f16
// of x before all else.
constexpr int few_threads(int turns) { return (4 + 4 * turns + 5) * 32; }
constexpr int kFewTokens = 64;
constexpr int kMaxParts = 8;           // CTAs of a cluster
constexpr int S = 4;                   // tiles of 64 k a step
constexpr int kWTiles = S, kMinWStages = 3, kMaxWStages = 10;   // ring of codes: tiles a stage, stages
constexpr int kABufs = 3, kACols = S * 32;
constexpr int kAFirst = 512 - kABufs * kACols;   // columns before: two accumulators
static_assert(kWTiles == S && 2 * kFewTokens <= kAFirst, "steps");

// Shared memory: x's slice, the parts of this CTA's tokens, the ring of codes in what is
// left (the more stages the better, for the first ones come before x).
struct Smem {
  static constexpr int o_exps = 0;                                   // [P][T]
  static constexpr int o_share = o_exps + kMaxParts * kFewTokens * 4;  // [P][share], and [share]
  static constexpr int o_top = o_share + (kMaxParts + 1) * kFewTokens * 4;
  static constexpr int o_exp = o_top + kFewTokens * 4;                // of this CTA's slice
  static constexpr int o_bar = o_exp + kFewTokens * 4;
  static constexpr int n_bar = 2 * kMaxWStages + kABufs + 4 + 4;
  static constexpr int o_misc = o_bar + n_bar * 8;                   // tmem base, abort
  static constexpr int o_x = 6144;
  static constexpr int total = 232448 - 1024;
};
static_assert(Smem::o_misc + 16 <= Smem::o_x, "shared memory");
constexpr int kWStageBytes = kWTiles * kTileBytes;

struct Args {
  const __nv_bfloat16* x;
  int64_t x_stride;
  const unsigned char* packed;
  const float* powers;
  void* y;
  int64_t y_stride;
  int T, N, K, rt, kb, nt, nr, share, f32, o_part, o_w, w_stages;
};

// Address of this CTA's shared memory word in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  return a;
}
// Stores whose bytes the barrier of the receiving CTA counts.
__device__ __forceinline__ void send(uint32_t at, int v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
               :: "r"(at), "r"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void send4(uint32_t at, const float* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
               :: "r"(at), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                  "r"(__float_as_uint(v[3])), "r"(bar) : "memory");
}
// Tile of 64 k (from column x) of all tokens.
__device__ __forceinline__ void tma_x(void* dst, const CUtensorMap* map, int x, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(tc::smem_u32(dst)), "l"(map), "r"(x), "r"(0), "r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// A warp's wait for a place once another wait has run out. (Out of line: in the loop it cost
// 4,096 x 8,192 for 1 token 0.4 us of 10.9, 131,072 x 4,096 0.5 of 65.5.)
__device__ __noinline__ void place_wait(uint64_t* bar, uint32_t parity) {
  if ((threadIdx.x & 31) == 0 && !tc::mbar_wait(bar, parity)) record_device_status(GDN_ERR_TIMEOUT);
  __syncwarp();
}
// 2^d, d <= 0, as what a part counts: below 2^-149 that, next to nothing and not nothing,
// so that an infinity stays one.
__device__ __forceinline__ float weight_of(int d) {
  return d >= -126 ? pow2(d) : __int_as_float(1 << (max(d, -149) + 149));
}
// A warp's bounded wait for arrivals of other CTAs.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    const long long t0 = clock64();
    for (uint32_t done = 0; !done;) {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.b32 %0, 1, 0, p;\n\t}\n"
          : "=r"(done) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
      if (done) break;
      if (*abort || clock64() - t0 > 4000000000LL) {
        if (!*abort) record_device_status(GDN_ERR_TIMEOUT);
        *abort = 1;
        ok = false;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// x's slice (kn tiles of nr tokens) to f16 in its place, by the 256 threads of the eight
// warps that have no other work yet: 8 lanes a row of 128 bytes, a thread one chunk of a
// token in every `step`th tile. As it is, where the token's largest value is from 2^-3 to
// 2^15 (what f16 rounds then, values below 2^-14, it rounds by 2^-22 of the largest at
// most); other tokens are made again from memory, scaled. (In one pass, by few
// instructions: the largest first and a product for each value took 5 instead of 2 us for
// 32 tokens of 2,048. Out of line and in short loops: unrolled in every role it was 10 us
// of instruction fetches.)
constexpr uint32_t kLeast = (127 - 3) << 7, kMost = (127 + 15) << 7;   // as BF16 bits
__device__ __noinline__ void convert_x(unsigned char* smem, const Args& p, int k0, int kn, int part, uint64_t* full,
                                       volatile int* abort) {
  const int nr = p.nr, slot = part >> 3, c = part & 7, step = max(1, 32 / nr), lane = part & 31;
  const int b0 = nr < 32 ? slot / nr : 0, stride = nr * 128;
  int* s_exp = reinterpret_cast<int*>(smem + Smem::o_exp);
  uint32_t* s_top = reinterpret_cast<uint32_t*>(smem + Smem::o_top);
  const bool here = warp_wait(full, 0, abort) && b0 < step;
  for (int t = nr < 32 ? slot % nr : slot; here && t < nr; t += 32) {
    unsigned char* at = smem + Smem::o_x + t * 128 + c * 16;
    __nv_bfloat162 top = {0, 0};
#pragma unroll 4
    for (int b = b0; b < kn; b += step) {
      uint4* chunk = reinterpret_cast<uint4*>(at + b * stride);
      const uint4 v = *chunk;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(w + i)));
        const __half2 two = __floats2half2_rn(bf16lo(w[i]), bf16hi(w[i]));
        h[i] = *reinterpret_cast<const uint32_t*>(&two);
      }
      *chunk = make_uint4(h[0], h[1], h[2], h[3]);
    }
    const uint32_t both = *reinterpret_cast<const uint32_t*>(&top);
    atomicMax(s_top + t, max(both & 0xffffu, both >> 16));
    if (nr < 32) break;
  }
  tc::fence_smem_to_async();
  asm volatile("bar.sync 1, 256;" ::: "memory");
  auto as_is = [&](int t) { return s_top[t] == 0 || (s_top[t] >= kLeast && s_top[t] < kMost); };
  if (__all_sync(0xffffffffu, as_is(lane) && as_is(lane + 32))) return;   // all warps alike
  // Largest finite magnitudes, then f16 by them, both from memory.
  for (int pass = 0; pass < 2; ++pass) {
    for (int t = nr < 32 ? slot % nr : slot; here && t < p.T; t += 32) {
      const __nv_bfloat16* row = p.x + (int64_t)t * p.x_stride;
      const int e = x_exponent((uint32_t)s_exp[t]);
      uint32_t top = 0;
      if (!as_is(t))
        for (int b = b0; b < kn; b += step) {
          const uint4 v = load8(row, (k0 + b) * kK + ((c ^ (t & 7)) << 3), p.K);
          if (pass == 0) top = max(top, finite_top8(v));
          else *reinterpret_cast<uint4*>(smem + Smem::o_x + t * 128 + c * 16 + b * stride) = to_half8(v, pow2(-e));
        }
      if (pass == 0) atomicMax(s_exp + t, (int)top);
      if (nr < 32) break;
    }
    tc::fence_smem_to_async();
    asm volatile("bar.sync 1, 256;" ::: "memory");
  }
  if (part < p.T && !as_is(part)) s_exp[part] = x_exponent((uint32_t)s_exp[part]);
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

template <int kTurns>
__global__ void __launch_bounds__(few_threads(kTurns), 1)
w4_few_kernel(const __grid_constant__ Args p, const __grid_constant__ CUtensorMap x_map) {
  constexpr int kResults = 4 + 4 * kTurns;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* w_full = reinterpret_cast<uint64_t*>(smem + Smem::o_bar);
  uint64_t* w_empty = w_full + kMaxWStages;
  uint64_t* a_empty = w_empty + kMaxWStages;
  uint64_t* d_full = a_empty + kABufs;   // [2]
  uint64_t* d_empty = d_full + 2;        // [2]
  uint64_t* parts_full = d_empty + 2;    // all parts of this CTA's tokens are here
  uint64_t* parts_empty = parts_full + 1;  // this CTA's parts have been added everywhere
  uint64_t* x_full = parts_empty + 1;
  uint64_t* drained = x_full + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Smem::o_misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Smem::o_misc + 4);
  float* s_part = reinterpret_cast<float*>(smem + p.o_part);
  int* s_exps = reinterpret_cast<int*>(smem + Smem::o_exps);
  float* s_weight = reinterpret_cast<float*>(smem + Smem::o_share);
  int* s_most = reinterpret_cast<int*>(s_weight + kMaxParts * kFewTokens);
  int* s_exp = reinterpret_cast<int*>(smem + Smem::o_exp);
  uint32_t* s_top = reinterpret_cast<uint32_t*>(smem + Smem::o_top);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t P;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(P));
  const int rank = (int)cluster_rank(), clusters = gridDim.x / P, cid = blockIdx.x / P;
  // This CTA's slice of K, in tiles, and its row tiles: cid, cid + clusters, ...
  const int k0 = (int)((int64_t)p.kb * rank / P), kn = (int)((int64_t)p.kb * (rank + 1) / P) - k0;
  const int rows = (p.rt - cid + clusters - 1) / clusters;
  const int x_tile = p.nr * 128;

  if (tid == 0) {
    for (int i = 0; i < p.w_stages; ++i) {
      tc::mbar_init(w_full + i, 1);
      tc::mbar_init(w_empty + i, 4);
    }
    for (int i = 0; i < kABufs; ++i) {
      tc::mbar_init(a_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(d_full + i, 1);
      tc::mbar_init(d_empty + i, 4);
    }
    tc::mbar_init(parts_full, 1);
    tc::mbar_init(parts_empty, 4 * P);
    tc::mbar_init(x_full, 1);
    tc::mbar_init(drained, 1);
    *s_abort = 0;
  }
  if (tid < kFewTokens) s_top[tid] = s_exp[tid] = 0;
  if (warp == 1) {
    tc::tmem_alloc(s_tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  cluster_sync();
  tc::fence_after_sync();
  // All 512 columns begin at address 0. (A constant, so that the MMAs' operands stay in
  // uniform registers.)
  constexpr uint32_t tmem = 0;
  const uint32_t a_base = tmem + kAFirst;

  // Warps 1 to 3, and those behind the ones that widen.
  auto convert = [&]() {
    convert_x(smem, p, k0, kn, warp < 4 ? tid - 32 : tid - (kResults - 3) * 32, x_full, s_abort);
  };
  const unsigned char* codes = p.packed + ((size_t)cid * p.kb + k0) * kTileBytes;
  // (A hint may come before the wait: L2 is where writes meet.)
  if (tid == 64) asm volatile("prefetch.tensormap [%0];" :: "l"(&x_map) : "memory");
  if (tid == 0) bulk_prefetch_l2(codes, min(kn, p.w_stages * kWTiles) * kTileBytes);
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ======================= codes =================================================
    int issued = 0, ws = 0, b = 0, row = 0;
    uint32_t w_phase = 1;
    auto post = [&]() {
      const int m = min(kWTiles, kn - b);
      tc::mbar_arrive_expect_tx(w_full + ws, m * kTileBytes);
      tc::bulk_g2s(smem + p.o_w + ws * kWStageBytes, codes + (size_t)b * kTileBytes, m * kTileBytes,
                   w_full + ws);
      ++issued;
      if (++ws == p.w_stages) {
        ws = 0;
        w_phase ^= 1;
      }
      if ((b += m) == kn) {
        b = 0;
        ++row;
        codes += (size_t)clusters * p.kb * kTileBytes;
      }
    };
    if (lane == 0) {
      while (issued < p.w_stages && row < rows) post();
      while (row < rows) {
        if (!mbar_wait_abortable(w_empty + ws, w_phase, s_abort, 64)) break;
        post();
      }
      if (*s_abort)                      // copies in flight land before the CTA ends
        for (int i = max(0, issued - p.w_stages); i < issued; ++i)
          tc::mbar_wait(w_full + i % p.w_stages, (i / p.w_stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA ===================================================
    const bool one = tc::elect_one();
    const uint32_t id = idesc_f16(p.nt);
    const uint64_t xd = x_desc(tc::smem_u32(smem + Smem::o_x));
    const int x_step = x_tile / 16;
    // It waits for a buffer at a named barrier, where the warps that fill it arrive: no
    // polls beside theirs. A named barrier knows no limit, so every step is passed, in
    // order, also when a wait has run out: the buffer is then given back as it is.
    int ab = 0;
    convert();
    for (int row = 0; row < rows; ++row) {
      const int db = row & 1;
      const uint32_t d = tmem + db * kFewTokens;
      const bool ok = warp_wait(d_empty + db, ((row >> 1) & 1) ^ 1, s_abort);
      uint64_t x = xd;
      for (int b = 0; b < kn; b += S) {
        filled_sync(ab);
        tc::fence_after_sync();
        const int n = min(S, kn - b);
        if (one && ok) {
          const uint32_t a = a_base + ab * kACols;
          if (n == S) {
#pragma unroll
            for (int k = 0; k < S * 4; ++k)
              tc::mma_bf16_tmem_a(d, a + k * 8, x + (uint32_t)(k / 4 * x_step) + k % 4 * 2, id, b + k > 0);
          } else {
#pragma unroll 1
            for (int k = 0; k < n * 4; ++k)
              tc::mma_bf16_tmem_a(d, a + k * 8, x + (uint32_t)(k / 4 * x_step) + k % 4 * 2, id, b + k > 0);
          }
          tc::mma_commit(a_empty + ab);
          if (b + S >= kn) tc::mma_commit(d_full + db);
        } else if (one) {
          tc::mbar_arrive(a_empty + ab);
        }
        x += (uint32_t)(S * x_step);
        if (++ab == kABufs) ab = 0;
      }
    }
    // Nothing is in flight when tensor memory is freed.
    if (one) tc::mma_commit(drained);
    if (!tc::mbar_wait(drained, 0)) record_device_status(GDN_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp >= 4 && warp < kResults) {
    // ======================= codes to f16 ==========================================
    // The warpgroups take turns; a thread has the row of its lane in tensor memory. (One
    // tile's instructions, looped over: those of a whole step do not stay in the
    // instruction cache beside the other roles'.)
    const int r = (warp & 3) * 32 + lane;
    int b = 0, row = 0, s = 0, ab = 0;
    uint32_t wp = 0, ap = 1;
    auto stage = [&]() {
      if (++s == p.w_stages) {
        s = 0;
        wp ^= 1;
      }
    };
    auto buffer = [&]() {
      if (++ab == kABufs) {
        ab = 0;
        ap ^= 1;
      }
      if ((b += S) >= kn) {
        b = 0;
        ++row;
      }
    };
    auto pass = [&](int steps) {         // steps of the other warpgroups
      for (; steps > 0; --steps) {
        stage();
        buffer();
      }
    };
    pass((warp >> 2) - 1);
    Asked place_ready = ask(a_empty + ab, ap);
    bool ok = true;
    while (row < rows) {
      const int m = min(S, kn - b), filled = ab;
      uint32_t to = tc::tmem_warp_addr(a_base, ab * kACols);
      // (Not without the place, whatever has run out: two buffers' arrivals at one named
      // barrier would leave the warp of the MMAs there for good. It passes every step.)
      ok = ok && granted(place_ready, s_abort);
      if (!ok) place_wait(place_ready.bar, place_ready.parity);
      tc::fence_after_sync();
      // (Codes are asked for from here on: the place is free, so three steps back all have
      // been widened, and no stage is more than one phase away from what is asked.)
      static_assert(kMinWStages >= kABufs && kTurns <= kABufs, "no stage more than a phase away");
      Asked codes_ready = ask(w_full + s, wp);
      ok = ok && granted(codes_ready, s_abort);
      const unsigned char* tile = smem + p.o_w + s * kWStageBytes;
      uint64_t* emptied = w_empty + s;
      stage();
      buffer();
      pass(kTurns - 1);
      place_ready = ask(a_empty + ab, ap);
      if (ok) {
        // Two tiles at a time, the next two read meanwhile.
        Codes a = load_codes(tile, r), b = load_codes(tile + (m > 1 ? kTileBytes : 0), r);
#pragma unroll 1
        for (int k = m; k > 0; k -= 2) {
          const Codes c = a, d = b;
          tile += 2 * kTileBytes;
          if (k > 2) {
            a = load_codes(tile, r);
            b = load_codes(tile + (k > 3 ? kTileBytes : 0), r);
          }
          widen_codes(c, to);
          if (k > 1) widen_codes(d, to + 32);
          to += 64;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(emptied);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      filled_arrive(filled);
    }
  } else if (warp >= kResults && warp < kResults + 4) {
    // ======================= results ===============================================
    const int r = (warp & 3) * 32 + lane;
    const int own0 = rank * p.share, own = max(0, min(p.share, p.T - own0));
    // Bytes that come in for a row tile: 16 for 4 tokens of each row, of each CTA.
    const uint32_t expected = P * ((own + 3) / 4) * kRows * 16;
    convert();
    if (warp == kResults && P > 1) {       // the slice's exponents, to every CTA
      if (lane == 0) tc::mbar_arrive_expect_tx(parts_full, expected + P * p.T * 4);
      for (int q = 0; q < (int)P; ++q)
        for (int t = lane; t < p.T; t += 32)
          send(remote(s_exps + rank * kFewTokens + t, q), s_exp[t], remote(parts_full, q));
    }
    for (int row = 0; row < rows; ++row) {
      const int n = (cid + row * clusters) * kRows + r, db = row & 1;
      const int e_n = exponent(p.powers[n]);
      if (!warp_wait(d_full + db, (row >> 1) & 1, s_abort, 100)) break;
      if (__any_sync(0xffffffffu, *s_abort)) break;      // (MMAs of a buffer that was not filled)
      tc::fence_after_sync();
      const uint32_t d = tc::tmem_warp_addr(tmem, db * kFewTokens);
      if (P == 1) {
        for (int t = 0; t < p.T; t += 16) {
          float v[16];
          tc::tmem_ld16(d + t, v);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (t + k < p.T && n < p.N)
              store(p.y, p.f32, (int64_t)(t + k) * p.y_stride + n, scaled(v[k], e_n + s_exp[t + k]));
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(d_empty + db);
        continue;
      }
      // The places of the parts are free again.
      if (row > 0) {
        if (!cluster_wait(parts_empty, (row - 1) & 1, s_abort)) break;
        if (warp == kResults && lane == 0) tc::mbar_arrive_expect_tx(parts_full, expected);
      }
      // Parts of a CTA's tokens: [P][share / 4][128 rows][4].
      int q = 0, left = p.share;
      uint32_t to = remote(s_part + rank * p.share * kRows + r * 4, 0), bar = remote(parts_full, 0);
      for (int t = 0; t < p.T; t += 16) {
        float v[16];
        tc::tmem_ld16(d + t, v);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          if (t + k >= p.T) break;
          send4(to, v + k, bar);
          to += kRows * 16;
          if ((left -= 4) == 0 && t + k + 4 < p.T) {
            left = p.share;
            ++q;
            to = remote(s_part + rank * p.share * kRows + r * 4, q);
            bar = remote(parts_full, q);
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(d_empty + db);
      if (!cluster_wait(parts_full, row & 1, s_abort)) break;
      if (row == 0) {
        // What a part counts beside the one with the largest x of its token. (Each of the
        // four warps writes all of it, and reads what it wrote.)
        for (int t = lane; t < own; t += 32) {
          int most = s_exps[own0 + t];
          for (int q = 1; q < (int)P; ++q) most = max(most, s_exps[q * kFewTokens + own0 + t]);
          s_most[t] = most;
          for (int q = 0; q < (int)P; ++q)
            s_weight[q * kFewTokens + t] = weight_of(s_exps[q * kFewTokens + own0 + t] - most);
        }
        __syncwarp();
      }
      // 16 tokens at a time, their loads all on the way together (beside the stores to
      // tensor memory one takes some 400 cycles). The parts are given back before the
      // last stores to y, which the release would wait for.
      for (int t = 0; t < max(own, 1); t += 16) {
        float sum[16] = {};
        const float* part = s_part + t * kRows + r * 4;
#pragma unroll 1
        for (int q = 0; q < (int)P; ++q, part += p.share * kRows) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            if (t + k < own) {
              const float4 v = *reinterpret_cast<const float4*>(part + k * kRows);
              const float4 w = *reinterpret_cast<const float4*>(s_weight + q * kFewTokens + t + k);
              sum[k] = fmaf(v.x, w.x, sum[k]);
              sum[k + 1] = fmaf(v.y, w.y, sum[k + 1]);
              sum[k + 2] = fmaf(v.z, w.z, sum[k + 2]);
              sum[k + 3] = fmaf(v.w, w.w, sum[k + 3]);
            }
        }
        if (t + 16 >= own && row + 1 < rows) {
          __syncwarp();
          if (lane < (int)P) remote_arrive(remote(parts_empty, lane));
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (t + k < own && n < p.N)
            store(p.y, p.f32, (int64_t)(own0 + t + k) * p.y_stride + n, scaled(sum[k], e_n + s_most[t + k]));
      }
    }
  } else {
    if (warp == 2) {
      if (lane == 0) tc::mbar_arrive_expect_tx(x_full, kn * x_tile);
      __syncwarp();
      for (int i = lane; i < kn; i += 32) tma_x(smem + Smem::o_x + i * x_tile, &x_map, (k0 + i) * kK, x_full);
      __syncwarp();
    }
    convert();
    if (warp == 2 && *s_abort) tc::mbar_wait(x_full, 0);
  }
  // Every role of every CTA is here, done or given up.
  tc::fence_before_sync();
  __syncthreads();
  cluster_end();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// Clusters of P CTAs that the device holds at a time (0: unknown).
// (The shared memory decides, not the number of threads.)
int max_clusters(int device, int P) {
  static DeviceNumber counts[kMaxParts + 1];
  return counts[P](device, [&] { return clusters_of(w4_few_kernel<3>, P, few_threads(3), Smem::total); });
}

// Tokens whose results a CTA of the cluster adds up.
int few_share(int T, int P) { return ((T + P - 1) / P + 3) / 4 * 4; }
// Warpgroups that widen, for CTAs with `rows` row tiles of kn tiles of 64 k. A third one
// hides more of a step's chain of waits where a CTA has many steps, and comes late where it
// has few or where x and the results of more than 16 tokens are the work. us by two and
// three, 1 token: 131,072 x 4,096 66.1 and 61.1, 131,072 x 1,024 19.8 and 19.1, 20,000 x 4,096
// 22.4 and 21.6; 60,000 x 512 (4 x 8 tiles) 8.7 and 9.1, 4,096 x 4,096 (a row) 8.0 and 8.2; 24
// tokens: 131,072 x 1,024 23.4 and 24.0.
int few_turns(int T, int rows, int kn) { return T <= 16 && rows > 1 && rows * kn >= 64 ? 3 : 2; }
// What x's slice and the parts leave for the codes, in stages.
int few_stages(int T, int kn, int P) {
  const int left = Smem::total - Smem::o_x - kn * ((T + 7) / 8 * 8) * 128 - 1024 - (P > 1 ? P * few_share(T, P) * kRows * 4 : 0);
  return left < 0 ? 0 : std::min(kMaxWStages, left / kWStageBytes);
}

// x as (k, token), boxes of 64 k and `rows` tokens; zeros outside.
bool x_tensor(CUtensorMap* map, const void* x, int64_t stride, int T, int K, int rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  // (A single row's stride says nothing, and may be more than a tensor map takes.)
  if (T == 1) stride = (K + 7) / 8 * 8;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)T}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {kK, (cuuint32_t)rows}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool launch_w4_few(const void* x, int64_t x_stride, const void* packed, void* y, int64_t y_stride, int32_t y_type,
                   int32_t T, int32_t N, int32_t K, cudaStream_t st, gdn_status_t* rc) {
  if (T > kFewTokens) return false;
  static DeviceOnce once[2];
  if (allow_smem(once[0], w4_few_kernel<2>, Smem::total) != cudaSuccess ||
      allow_smem(once[1], w4_few_kernel<3>, Smem::total) != cudaSuccess) {
    cudaGetLastError();                  // clear it
    return false;
  }
  const int device = current_device();
  const Shape s(N, K);
  Args a;
  a.nr = (T + 7) / 8 * 8;
  // The cluster that takes least, or the general kernel, in the time of a tile of 64 k
  // (some 0.13 us): rounds of row tiles, x, and the last round's results. What the parts of
  // a round cost: 32 x 131,072 x 4,096 by pairs takes 95 us, 14 rounds of 52 tiles' time
  // for 32 tiles; the general kernel, which has x's kernel before it, 71. 1 x 4,096 x 8,192
  // by fours takes 10.8, by the general kernel 17.5.
  int parts = 0;
  double least = w4_general_cost(T, N, K);
  for (int P = 1; P <= std::min(kMaxParts, s.kb); ++P) {
    const int kn = (s.kb + P - 1) / P, clusters = max_clusters(device, P);
    if (clusters == 0 || few_stages(T, kn, P) < kMinWStages) continue;
    const double cost = (double)((s.rt + clusters - 1) / clusters) * (kn + (P > 1 ? 20 : 1)) + kn * a.nr * 128 / 10000.0 +
                        (P > 1 ? 40 : 20);
    if (cost < least) {
      parts = P;
      least = cost;
    }
  }
  if (parts == 0) return false;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.x_stride = x_stride;
  a.packed = static_cast<const unsigned char*>(packed);
  a.powers = reinterpret_cast<const float*>(a.packed + s.powers());
  a.y = y;
  a.y_stride = y_stride;
  a.T = T;
  a.N = N;
  a.K = K;
  a.rt = s.rt;
  a.kb = s.kb;
  a.nt = (T + 15) / 16 * 16;
  a.share = few_share(T, parts);
  const int kn = (s.kb + parts - 1) / parts;
  a.w_stages = few_stages(T, kn, parts);
  a.o_part = Smem::o_x + kn * a.nr * 128;
  a.o_w = (a.o_part + (parts > 1 ? parts * a.share * kRows * 4 : 0) + 1023) / 1024 * 1024;   // room behind x: its last rows
  a.f32 = y_type == GDN_TYPE_F32;
  CUtensorMap map;
  if (!x_tensor(&map, x, x_stride, T, K, a.nr)) {
    set_cuda_error(cudaErrorInvalidValue);
    *rc = GDN_ERR_CUDA;
    return true;
  }
  const int clusters = std::min(s.rt, max_clusters(device, parts));
  const int turns = few_turns(T, (s.rt + clusters - 1) / clusters, kn);
  *rc = check_launch(launch_clusters(turns == 3 ? w4_few_kernel<3> : w4_few_kernel<2>, clusters, parts,
                                     few_threads(turns), Smem::total, st, a, map));
  return true;
}

GDN_DEFINE_STATUS_GATHER(gather_status_w4_few)

}  // namespace gdn
