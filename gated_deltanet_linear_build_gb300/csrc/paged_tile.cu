// Attention of many query rows over a paged 8-bit cache, on the 5th-generation
// tensor cores.
//
// Bound: 4 d operations per visible (query row, key) pair at the BF16 rate, as
// long as the softmax (one exponential a pair) and the widening of V keep up.
// One CTA per SM; a tile is 256 rows (d <= 128: two 128-row halves that take
// turns on the tensor core) or 128 rows (d = 256, whose float32 output fills
// half of the tensor memory). Scores are kept two units of 64 keys ahead of the
// softmax, so that neither it nor the tensor core waits for the other's
// latency. Per unit:
//
// * S = Q K^T as e4m3 MMAs (kind::f8f6f4): K as it lies in the cache, Q as the
//   sum of two e4m3 parts hi + lo, which hold BF16's 8 significand bits. Two
//   passes at twice the BF16 rate cost what one BF16 pass would, without
//   widening K.
// * softmax: one thread per row, scores read once from tensor memory; P goes
//   back as f16 over the scores' columns and is the A operand of
// * O += P V (kind::f16). V's codes become f16 (exact) in the registers of the
//   loading warps on their way to shared memory.
// * Scales: K's joins the score's factor, V's the exponent, P' = 2^(s + log2 vs
//   - m), with P' / vs in the sum, per 16 keys (the smallest block). O is
//   rescaled only when a row's maximum grows by more than 2^8.
//
// Work split: where items are many or alike enough, whole items are dealt out by
// length (the plan compares the two). Otherwise, as in the split kernel, all (tile,
// kv head, 64 keys) units form one line cut into pieces of equal cost, one per SM;
// a tile cut by the end of a piece leaves float32 partial results, which another
// kernel joins in CTA order.
//
// Measured: 4,096 tokens of a 16,384-token prompt, 32 + 8 heads of 128: 733 us, 1,312
// TFLOP/s, 69% of the BF16 rate (the MMAs with a softmax that does nothing: 667
// us). 8,192-token prompt: 461 us; 16 + 2 heads of 256: 380 us, 1,445 TFLOP/s. 2,048
// tokens of 4 prompts, 16 + 2 heads of 256: 35 us (planned once a step: 30.6), latency.
//
// Roles (four warpgroups): 0 .. kM - 1: softmax of one 128-row tile each; the
// others up to 2: Q, widening of V; warps 12 and 15: MMAs of a tile each; warp
// 13: TMA copies of K, and the blocks' scales; warp 14: TMA copies of V's codes.
// K and V's codes lie as TMA leaves them, rows of 128 (64 for d = 64) bytes
// with their 16-byte chunks XOR-swizzled; Q and the widened V as 8 x 16-byte
// core matrices. Copies issued by threads instead (cp.async and register
// prefetches of 16 bytes each) held the tensor cores to a fifth of their rate.
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_attn.cuh"

namespace gdn {
namespace {
using namespace attn;

constexpr int kThreads = 512;
constexpr int kKeys = kTileKeys;         // keys per unit
// Registers: four warpgroups are launched with 128 a thread; their shares add
// up to no more than 4 x 128.
constexpr int kLaunchRegs = 128;

template <int D>
struct TC {
  static constexpr int M = D == 256 ? 1 : 2;            // 128-row tiles
  static constexpr int KS = D == 256 ? 4 : 6;           // K stages
  static constexpr int VR = D == 256 ? 2 : 4;           // stages of V's codes
  static constexpr int VS = D == 256 ? 2 : 4;           // and of V widened
  static constexpr int loaders = (3 - M) * 128;
  static constexpr int row = box_row(D);                // bytes of a row in a TMA box
  static constexpr int boxes = D / row;                 // boxes across a cache row
  static constexpr int q_part = 128 * D;                // one part (hi or lo) of one tile
  static constexpr int c_stage = kKeys * D;             // a unit's codes of K or V
  static constexpr int v_stage = kKeys * D * 2;
  static constexpr int o_q = 0;
  static constexpr int o_k = o_q + M * 2 * q_part;
  static constexpr int o_vr = o_k + KS * c_stage;
  static constexpr int o_v = o_vr + VR * c_stage;
  // Scales of a unit's 4 groups of 16 keys, float [8 units][ks | log2 vs | kSumScale /
  // vs][4]; the last is negative in units whose V scales lie far apart (kFarApart).
  // Unit n + KS is copied once the scores of n are done, so once the softmax of
  // n - 2 is: KS + 2 units are alive.
  static constexpr int o_sc = o_v + VS * v_stage;
  static_assert(KS + 2 <= 8, "ring of scales");
  // First key of a segment whose V is NaN in a column, uint16 [NR segments][D]. V
  // is widened at most VS units, hence segments, ahead of the results.
  static constexpr int NR = D == 256 ? 3 : 8;
  static_assert(VS < NR, "ring of NaN marks");
  static constexpr int o_nan = o_sc + 8 * 12 * 4;
  // Exponents of the rows' scales, int8 [2 segments][rows].
  static constexpr int o_ex = o_nan + NR * D * 2;
  static constexpr int o_bar = o_ex + 2 * M * 128;
  static constexpr int n_bar = 2 * KS + 2 * VR + 2 * VS + 8 + 4 + 4 + 4 + 2 + 2 + 3;
  static constexpr int o_misc = o_bar + n_bar * 8;      // tmem base, abort, flags
  static constexpr int total = o_misc + 32;
  static_assert(total <= 232448, "shared memory of one CTA");
  static constexpr int regs = 144, mma_regs = 80;
  static_assert(3 * regs + mma_regs <= 4 * kLaunchRegs, "registers of the launch");
  // Tensor-memory columns: two score buffers of 64 keys per tile, then O.
  static constexpr int c_s(int m, int b) { return m * 128 + b * 64; }
  static constexpr int c_o(int m) { return 256 + m * D; }
  // With one tile there is room for Q as well (hi, then lo): a 128 x 64 score
  // product then reads 2 KB of shared memory instead of 6, and 33 cycles are the
  // tensor core's instead of 49 (an 8,192-token prompt, 16 heads: 446 -> 381 us).
  // It also frees Q's place at once, so that the next segment's Q is prepared
  // during this one.
  static constexpr bool q_in_tmem = M == 1;
  static constexpr int c_q(int part) { return 128 + part * (D / 4); }
};

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
      :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// A in tensor memory: row m in lane m, four K elements a column.
__device__ __forceinline__ void mma_f8_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// 128 rows x 32 bytes of a K-major tile to 8 columns of tensor memory.
__device__ __forceinline__ void copy_128x256b(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" :: "r"(tmem), "l"(desc) : "memory");
}
// kind::f8f6f4: e4m3 A and B (format 0), float32 D. kind::f16: f16 A and B.
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Factor of a score: kept from 0, which would turn a masked score's -inf into
// NaN (a row's or block's scale may be that small); NaN marks a row and stays.
__device__ __forceinline__ float factor(float a) { return a < 1e-37f ? 1e-37f : a; }

// 32 columns of this warp's 32 lanes, without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}
// 16 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32_async(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
         "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
         "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
         "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
         "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r) : "r"(two));
  return r;
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegs));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}

// A bounded wait of a whole warp: all lanes go on, or none does.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_abortable(bar, parity, abort));
}

// One contiguous run of units of one (tile, head).
struct Seg {
  int seq, row0, n_units, cum, first_unit, count;
  Seq s;
  int n_rows, key_end;
};

// This CTA's work: a piece of the line of units (lo, head, it and s are those of
// its next unit), or whole items dealt out from the list sorted by length.
struct Line {
  int num, units1, lo, head, deal;     // deal: round of the dealing, -1 for a piece
  Item it;
  Seq s;
  long long u, u_end;
  __device__ bool more() const { return u < u_end; }
};

__device__ __forceinline__ Line line_of(const Args& p) {
  const Start at = read_start(p.tile_starts + blockIdx.x);
  Line l;
  l.num = at.num_items;
  l.units1 = at.units;
  l.lo = at.item;
  l.head = at.head;
  l.deal = at.c0 < 0 ? 0 : -1;
  l.it = at.it;
  l.s = {at.first, at.len, at.kv};
  l.u = at.u;
  l.u_end = at.u + at.count;
  return l;
}

__device__ __forceinline__ Seg seg_at(const Args& p, const Line& l, int tile_rows) {
  Seg g;
  g.seq = l.it.seq;
  g.row0 = l.it.row0;
  g.n_units = l.it.units;
  g.cum = l.it.cum;
  g.first_unit = l.deal >= 0 ? 0 : (int)(l.u - (long long)l.head * l.units1) - g.cum;
  g.count = l.deal >= 0 ? g.n_units : (int)min((long long)(g.n_units - g.first_unit), l.u_end - l.u);
  g.s = l.s;
  const int G = p.Hq / p.Hk;
  g.n_rows = min(tile_rows, g.s.len * G - g.row0);
  g.key_end = visible(g.s, (g.row0 + g.n_rows - 1) / G);
  return g;
}

__device__ __forceinline__ void pass(const Args& p, Line& l, const Seg& g) {
  const Item* from = p.tiles;
  if (l.deal >= 0) {
    // Back and forth over the CTAs: the longest with the shortest.
    ++l.deal;
    ++l.u;
    const int grid = gridDim.x, c = blockIdx.x;
    const int at = l.deal * grid + ((l.deal & 1) ? grid - 1 - c : c);
    l.lo = at / p.Hk;
    l.head = at - l.lo * p.Hk;
    from = p.sorted_tiles;
  } else {
    l.u += g.count;
    if (g.first_unit + g.count == g.n_units && ++l.lo == l.num) {
      l.lo = 0;
      ++l.head;
    }
  }
  if (l.more()) {
    const int4 raw = reinterpret_cast<const int4*>(from)[l.lo];
    l.it = {raw.x, raw.y, raw.z, raw.w};
    l.s = seq_of<true>(p.cu, p.kv, l.it.seq, p.T, (int64_t)p.max_blocks << p.log_b);
  }
}

// One 32-byte store of 16 BF16 values (or two of 16 bytes where o is not aligned
// for it): a row's sectors are written whole.
__device__ __forceinline__ void store16(__nv_bfloat16* at, const float* v, bool wide) {
  const uint4 a = pack8(v), b = pack8(v + 8);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(at), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z),
                    "r"(b.w) : "memory");
  } else {
    *reinterpret_cast<uint4*>(at) = a;
    *reinterpret_cast<uint4*>(at + 8) = b;
  }
}

// The NaNs of 16 codes of V taken out, and the first key of each of their columns
// kept. (Out of line: few units need it.)
__device__ __noinline__ uint4 take_nans(uint4 v, unsigned short* first_nan, int key) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll 1
    for (int b = 0; b < 4; ++b)
      if (((w[k] >> (8 * b)) & 0x7fu) == 0x7fu) {
        unsigned short* at = first_nan + k * 4 + b;
        unsigned short old = *reinterpret_cast<volatile unsigned short*>(at);
        while ((unsigned short)key < old) {
          const unsigned short was = atomicCAS(at, old, (unsigned short)key);
          if (was == old) break;
          old = was;
        }
        w[k] &= ~(0xffu << (8 * b));
      }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kAfterSplit: launched behind the split kernel (24 sequences, a fifth of them
// prompts of 300-600 tokens: 154 -> 142 us together with one join for both; as a
// run-time flag it cost d = 256 its registers, 381 -> 402 us for 8,192 tokens).
template <int D, bool kAfterSplit>
__global__ void __launch_bounds__(kThreads, 1)
attn_tile_kernel(const Args p, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  using C = TC<D>;
  constexpr int kM = C::M, kRows = kM * 128;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::o_bar);
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + C::KS;
  uint64_t* vr_full = k_empty + C::KS;
  uint64_t* vr_empty = vr_full + C::VR;
  uint64_t* v_full = vr_empty + C::VR;
  uint64_t* v_empty = v_full + C::VS;
  uint64_t* sc_full = v_empty + C::VS;       // [8]
  uint64_t* s_full = sc_full + 8;            // [kM][2] score buffers
  uint64_t* p_full = s_full + 4;             // [kM][2]
  // Products done, [kM][2] by the unit's parity, and Q, [2] by the segment's: the
  // softmax does not wait for every one of them, and with two barriers none is
  // more than one phase away from what it waits for.
  uint64_t* o_done = p_full + 4;
  uint64_t* q_full = o_done + 4;
  uint64_t* q_empty = q_full + 2;            // [2] by the segment's parity
  uint64_t* nan_sync = q_empty + 2;          // the widening threads among themselves
  uint64_t* drained = nan_sync + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::o_misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::o_misc + 4);
  volatile int* s_any_nan = reinterpret_cast<volatile int*>(smem + C::o_misc + 16);
  float* s_sc = reinterpret_cast<float*>(smem + C::o_sc);
  signed char* s_ex = reinterpret_cast<signed char*>(smem + C::o_ex);
  unsigned short* s_nan = reinterpret_cast<unsigned short*>(smem + C::o_nan);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = tid >> 7;
  const int G = p.Hq / p.Hk, B = 1 << p.log_b;

  if (tid == 0) {
    for (int i = 0; i < C::KS; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(k_empty + i, kM);
    }
    for (int i = 0; i < C::VR; ++i) {
      tc::mbar_init(vr_full + i, 1);
      tc::mbar_init(vr_empty + i, C::loaders);
    }
    for (int i = 0; i < C::VS; ++i) {
      tc::mbar_init(v_full + i, C::loaders);
      tc::mbar_init(v_empty + i, kM);
    }
    for (int i = 0; i < 8; ++i) tc::mbar_init(sc_full + i, 4);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 128);
      tc::mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full + i, C::loaders);
      tc::mbar_init(q_empty + i, 1);
    }
    tc::mbar_init(nan_sync, C::loaders);
    for (int i = 0; i < 2; ++i) tc::mbar_init(drained + i, 1);
    *s_abort = 0;
    *s_any_nan = 0;
  }
  if (warp == 12) {
    tc::tmem_alloc(s_tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
  // Behind the split kernel, the plan and the step's inputs are two launches back:
  // this kernel goes on as soon as it has an SM, and waits for the split kernel at its
  // end, for those that follow. Why it may: it can start only when every CTA of the
  // split kernel has let it, which each does behind its own wait, so all that this
  // kernel reads was complete, and in L2, before its first instruction; and what the
  // split kernel writes it does not read. TMA reads L2. What this SM's L1 holds from
  // earlier kernels the fence (an acquire at GPU scope) discards, and the loads behind
  // it are plain, coherent ones: no ld.global.nc, for which a fence promises nothing.
  if constexpr (kAfterSplit) {
    __threadfence();
  } else {
    pdl_wait();
    pdl_trigger();
  }
  Line l = line_of(p);

  if (wg == 3) {
    // ======================= MMA warp ==========================================
    regs_down<C::mma_regs>();
    // One warp per 128-row tile. The whole warp walks the role, so that descriptors
    // stay in uniform registers, and one elected lane issues: 66 cycles per 128 x
    // 128 MMA, the tensor core's own rate, where a lone lane's loop took above 200.
    // What the role does beside issuing is the tensor core's idle time: stages and
    // phases are counted along, not divided out, and two tiles have two warps
    // (4,096 tokens of 16,384, d = 128: 797 -> 731 us).
    if (warp == 12 || (kM == 2 && warp == 15)) {
      const int m = warp == 12 ? 0 : 1;
      const bool one = elect_one();
      constexpr uint32_t id_qk = idesc_f32(128, kKeys), id_pv = idesc_f32(128, D) | tc::kTransB;
      const uint32_t s_buf = tmem + m * 128, o_buf = tmem + C::c_o(0) + m * D;
      const uint64_t qd = tc::tile_desc(tc::smem_u32(smem + C::o_q) + m * 2 * C::q_part, D / 2, 0);
      const uint64_t kd = desc_swizzled<C::row>(tc::smem_u32(smem + C::o_k));
      const uint64_t vd = tc::mn_desc(tc::smem_u32(smem + C::o_v), D, 0);
      uint64_t* sf = s_full + m * 2;
      uint64_t* pf = p_full + m * 2;
      uint64_t* od = o_done + m * 2;
      // Stages and phases of the next unit to score and the next to add.
      int ks = 0, vs = 0, s_b = 0, p_b = 0, seg_b = 0;
      uint32_t kp = 0, vp = 0, pp = 0, qp = 0;
      bool ok = true;
      auto qk = [&]() {
        ok = ok && warp_wait(k_full + ks, kp, s_abort);
        tc::fence_after_sync();
        if (!ok) return;
        const uint32_t d = s_buf + s_b * 64;
        const uint64_t b = kd + ks * (C::c_stage / 16);
        if (one) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              const uint64_t bk = b + (k * 32 / C::row) * (kKeys * C::row / 16) + (k * 32 % C::row) / 16;
              if constexpr (C::q_in_tmem)
                mma_f8_tmem_a(d, tmem + C::c_q(part) + k * 8, bk, id_qk, part | k);
              else
                mma_f8(d, qd + part * (C::q_part / 16) + k * 16, bk, id_qk, part | k);
            }
          tc::mma_commit(sf + s_b);
          tc::mma_commit(k_empty + ks);
        }
        s_b ^= 1;
        if (++ks == C::KS) {
          ks = 0;
          kp ^= 1;
        }
      };
      while (ok && l.more()) {
        const Seg g = seg_at(p, l, kRows);
        ok = ok && warp_wait(q_full + seg_b, qp, s_abort);
        tc::fence_after_sync();
        if constexpr (C::q_in_tmem) {
          // The scores of the segment before are done, as their softmax is (p_full);
          // those of this one come behind the copy in the tensor core's order.
          if (ok && one) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                copy_128x256b(tmem + C::c_q(part) + k * 8, qd + part * (C::q_part / 16) + k * 16);
            tc::mma_commit(q_empty + seg_b);
          }
        }
        qp ^= seg_b;
        seg_b ^= 1;
        qk();
        if (g.count > 1) qk();
        for (int j = 0; ok && j < g.count; ++j) {
          ok = ok && warp_wait(v_full + vs, vp, s_abort);
          ok = ok && warp_wait(pf + p_b, pp, s_abort);
          tc::fence_after_sync();
          if (!ok) break;
          const uint32_t at = s_buf + p_b * 64;
          const uint64_t b = vd + vs * (C::v_stage / 16);
          if (one) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              tc::mma_bf16_tmem_a(o_buf, at + k * 8, b + k * 2 * D, id_pv, j > 0 || k > 0);
            tc::mma_commit(od + p_b);
            tc::mma_commit(v_empty + vs);
          }
          pp ^= p_b;
          p_b ^= 1;
          if (++vs == C::VS) {
            vs = 0;
            vp ^= 1;
          }
          if (j + 2 < g.count) qk();
        }
        pass(p, l, g);
      }
      // Nothing of this warp's tensor work is in flight when TMEM is freed.
      if (one) tc::mma_commit(drained + m);
      if (!tc::mbar_wait(drained + m, 0)) record_device_status(GDN_ERR_TIMEOUT);
      __syncwarp();
    } else if (warp == 13 || warp == 14) {
      // ===================== TMA copies ==========================================
      // Warp 13: K and the units' scales; warp 14: V's codes. Lane i posts box i:
      // one page (or its part in the unit) times one of the boxes across a row.
      const bool is_k = warp == 13;
      const int log_box = min(p.log_b, 6), box_keys = 1 << log_box;
      static_assert(kKeys == 64, "log_box");
      const int pages = kKeys >> log_box;
      const int page = lane % pages, bx = lane / pages;
      const bool posts = lane < pages * C::boxes;
      const CUtensorMap* map = is_k ? &k_map : &v_map;
      uint64_t* full = is_k ? k_full : vr_full;
      uint64_t* empty = is_k ? k_empty : vr_empty;
      const int stages = is_k ? C::KS : C::VR;
      unsigned char* base = smem + (is_k ? C::o_k : C::o_vr);
      const int absent = max(p.num_blocks * p.Hk, 1);   // a box past the end reads zeros
      int st = 0, round = 0, unit = 0;
      bool ok = true;
      while (ok && l.more()) {
        const Seg g = seg_at(p, l, kRows);
        const int32_t* table = p.table + (int64_t)g.seq * p.table_stride;
        const int key_first = g.first_unit * kKeys;
        const int n = g.count;
        auto id_at = [&](int i) {
          const int key = key_first + i * kKeys + page * box_keys;
          return i < n && key < g.key_end ? table[key >> p.log_b] : -1;
        };
        int next = id_at(0);
        for (int i = 0; i < n; ++i) {
          const int id = next;
          next = id_at(i + 1);
          if (round > 0) ok = ok && warp_wait(empty + st, (round - 1) & 1, s_abort);
          if (!ok) break;
          const int key0 = key_first + i * kKeys;
          const int key = key0 + page * box_keys;
          if (lane == 0) tc::mbar_arrive_expect_tx(full + st, C::c_stage);
          __syncwarp();
          if (posts) {
            const bool in = (unsigned)id < (unsigned)p.num_blocks;
            if (!in && is_k && key < g.key_end) record_device_status(GDN_ERR_INVALID_ARG);
            tma_box(base + st * C::c_stage + (bx * kKeys + page * box_keys) * C::row, map, bx * C::row,
                    key & (B - 1), in ? id * p.Hk + l.head : absent, full + st);
          }
          if (is_k) {
            // Scales of the unit's 4 groups of 16 keys.
            const int blk = __shfl_sync(0xffffffffu, id, ((lane & 3) * 16) >> log_box);
            if (lane < 4) {
              float a = 1.f, v = 1.f;
              if (key0 + lane * 16 < g.key_end && (unsigned)blk < (unsigned)p.num_blocks) {
                a = p.ks[(size_t)blk * p.Hk + l.head];
                v = p.vs[(size_t)blk * p.Hk + l.head];
              }
              v = fmaxf(v, 7.888609052210118e-31f);     // 2^-100
              float* sc = s_sc + (unit & 7) * 12;
              sc[lane] = a;
              sc[4 + lane] = lg2_approx(v);
              float iv = __fdividef(kSumScale, v);
              if (log_box < 6) {                        // several blocks
                const uint32_t ex = __float_as_uint(v) >> 23;
                if (__reduce_max_sync(0xfu, ex) - __reduce_min_sync(0xfu, ex) >= (uint32_t)kFarApart) iv = -iv;
              }
              sc[8 + lane] = iv;
              tc::mbar_arrive(sc_full + (unit & 7));
            }
            __syncwarp();
            ++unit;
          }
          if (++st == stages) {
            st = 0;
            ++round;
          }
        }
        pass(p, l, g);
      }
      // The copies in flight land before the CTA may end: a giving-up reader
      // would not have waited for them.
      if (*s_abort) {
        for (int i = 0; i < stages; ++i)
          if (round > 0 || i < st)
            tc::mbar_wait(full + i, (round - (i < st ? 0 : 1)) & 1);
      }
    }
  } else if (wg >= kM) {
    // ======================= Q, widening of V ====================================
    regs_up<C::regs>();
    const int dt = tid - kM * 128;                    // 0 .. loaders - 1
    constexpr int chunks = D / 16;
    constexpr int v_it = kKeys * chunks / C::loaders;
    const int r_in = dt & 7, c = (dt >> 3) % chunks;  // this thread's row of 8, its chunk
    const int rg_in = dt / (8 * chunks);              // and its group of 8 rows in a pass
    constexpr int rg_per = C::loaders / (8 * chunks); // groups of 8 rows per pass
    int unit = 0, nan_phase = 0, seg = 0;             // running counts
    bool ok = true;
    while (ok && l.more()) {
      const Seg g = seg_at(p, l, kRows);
      // ---- Q: hi and lo codes, one power-of-two scale per row ---------------------
      // 8 rows at a time, 4 lanes to 64 bytes of a row, so that loads use whole
      // sectors and the stores fill the core matrices in order. The next 8 rows are
      // on their way meanwhile. (A loop of small body: straight code that runs once
      // a segment is paid in instruction fetches.)
      {
        constexpr int passes = D / 32;
        constexpr int groups = kRows / 8 / (C::loaders / 32);       // of 8 rows, per warp
        const int rr = lane & 7, cq = lane >> 3;
        const float neg = p.scale_log2 < 0.f ? -1.f : 1.f;
        auto fetch = [&](int a, uint4 (&w)[passes]) {
          const int local = ((dt >> 5) * groups + a) * 8 + rr;
          const int qrow = g.row0 + local, qt = qrow / G;
          const __nv_bfloat16* src = p.q + (int64_t)(g.s.first + qt) * p.q_stride +
                                     (int64_t)(l.head * G + qrow - qt * G) * D + cq * 8;
#pragma unroll
          for (int k = 0; k < passes; ++k)
            w[k] = local < g.n_rows ? *reinterpret_cast<const uint4*>(src + k * 32) : make_uint4(0, 0, 0, 0);
        };
        uint4 w[passes], ahead[passes];
        fetch(0, ahead);
        // Q's place is free: copied on, or the last scores of the segment before done.
        if constexpr (C::q_in_tmem) {
          if (seg > 0) ok = ok && warp_wait(q_empty + ((seg - 1) & 1), ((seg - 1) >> 1) & 1, s_abort);
        } else {
          if (unit > 0) ok = ok && warp_wait(k_empty + (unit - 1) % C::KS, ((unit - 1) / C::KS) & 1, s_abort);
        }
#pragma unroll 1
        for (int a = 0; ok && a < groups; ++a) {
#pragma unroll
          for (int k = 0; k < passes; ++k) w[k] = ahead[k];
          if (a + 1 < groups) fetch(a + 1, ahead);
          const int local = ((dt >> 5) * groups + a) * 8 + rr;
          uint32_t top = 0;                          // largest magnitude, as bits
#pragma unroll
          for (int k = 0; k < passes; ++k) {
            const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = max(top, max((v[i] & 0x7fffu) << 16, v[i] & 0x7fff0000u));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
          // The row's largest magnitude goes to [128, 256). A row with an infinity
          // or NaN is zeros here, and marked by the exponent -128.
          const bool bad = top >= 0x7f800000u;
          const int ex = min(max((int)(top >> 23) - 127 - 7, -126), 126);
          const float inv = neg * __int_as_float((127 - ex) << 23);
          if (cq == 0) s_ex[(seg & 1) * kRows + local] = (signed char)(bad ? -128 : ex);
          unsigned char* hi = smem + C::o_q + (local >> 7) * 2 * C::q_part +
                              ((local & 127) >> 3) * (D * 8) + rr * 16 + (cq & 1) * 8 +
                              (cq >> 1) * 128;
#pragma unroll
          for (int k = 0; k < passes; ++k) {
            const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t h4[2] = {0, 0}, l4[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = bad ? 0u : v[i];
              const float x0 = bf16lo(x) * inv, x1 = bf16hi(x) * inv;
              const uint32_t h2 = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
              const uint32_t f = e4m3x2_half2(h2);
              const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&f));
              const uint32_t l2 = __nv_cvt_float2_to_fp8x2(make_float2(x0 - hf.x, x1 - hf.y),
                                                           __NV_SATFINITE, __NV_E4M3);
              h4[i >> 1] |= h2 << (16 * (i & 1));
              l4[i >> 1] |= l2 << (16 * (i & 1));
            }
            *reinterpret_cast<uint2*>(hi + k * 256) = make_uint2(h4[0], h4[1]);
            *reinterpret_cast<uint2*>(hi + C::q_part + k * 256) = make_uint2(l4[0], l4[1]);
          }
        }
        if (!ok) break;
        tc::fence_smem_to_async();
        tc::mbar_arrive(q_full + (seg & 1));
      }
      const int nan_base = visible(g.s, g.row0 / G) - kKeys;   // every row sees the unit behind it
      unsigned short* first_nan = s_nan + (seg % C::NR) * D;
      for (int i = 0; ok && i < g.count; ++i, ++unit) {
        const int key0 = (g.first_unit + i) * kKeys;
        const int sr = unit % C::VR, st = unit % C::VS;
        ok = ok && warp_wait(vr_full + sr, (unit / C::VR) & 1, s_abort);
        if (unit >= C::VS)
          ok = ok && warp_wait(v_empty + st, (unit / C::VS - 1) & 1, s_abort);
        if (!ok) break;
        if (i == 0) {
          for (int k = dt; k < D; k += C::loaders) first_nan[k] = 0xffff;
          tc::mbar_arrive(nan_sync);
          ok = warp_wait(nan_sync, nan_phase & 1, s_abort);
          ++nan_phase;
          if (!ok) break;
        }
        const unsigned char* src = smem + C::o_vr + sr * C::c_stage +
                                   (c * 16 / C::row) * (kKeys * C::row);
        uint4 raw[v_it];
#pragma unroll
        for (int it = 0; it < v_it; ++it)
          raw[it] = *reinterpret_cast<const uint4*>(
              src + swizzled<C::row>((it * rg_per + rg_in) * 8 + r_in, c % (C::row / 16)));
        unsigned char* dst = smem + C::o_v + st * C::v_stage;
        // Keys past the end hold stale bytes: zeros instead. And where the tile's
        // rows do not see the same keys, a weight of zero must not meet a NaN (0 x
        // NaN is NaN): a NaN of V is written as zero and kept as the first key
        // whose column has one.
        if (key0 > nan_base) {
          uint32_t any = 0;
#pragma unroll
          for (int it = 0; it < v_it; ++it) {
            if (key0 + (it * rg_per + rg_in) * 8 + r_in >= g.key_end) raw[it] = make_uint4(0, 0, 0, 0);
            any |= ((raw[it].x & 0x7f7f7f7fu) + 0x01010101u) | ((raw[it].y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((raw[it].z & 0x7f7f7f7fu) + 0x01010101u) | ((raw[it].w & 0x7f7f7f7fu) + 0x01010101u);
          }
          if ((any & 0x80808080u) != 0) {
#pragma unroll
            for (int it = 0; it < v_it; ++it)
              raw[it] = take_nans(raw[it], first_nan + c * 16,
                                  key0 + (it * rg_per + rg_in) * 8 + r_in - nan_base);
            *s_any_nan = 1;
          }
        }
#pragma unroll
        for (int it = 0; it < v_it; ++it) {
          const uint4 w = raw[it];
          unsigned char* at = dst + (it * rg_per + rg_in) * (D * 16) + c * 256 + r_in * 16;
          *reinterpret_cast<uint4*>(at) = make_uint4(e4m3x2_half2(w.x), e4m3x2_half2(w.x >> 16),
                                                     e4m3x2_half2(w.y), e4m3x2_half2(w.y >> 16));
          *reinterpret_cast<uint4*>(at + 128) = make_uint4(e4m3x2_half2(w.z), e4m3x2_half2(w.z >> 16),
                                                           e4m3x2_half2(w.w), e4m3x2_half2(w.w >> 16));
        }
        // Only now: an arrival right behind the loads overtook them, and a copy landed in
        // codes not yet read (one step in some thousands).
        tc::mbar_arrive(vr_empty + sr);
        tc::fence_smem_to_async();
        tc::mbar_arrive(v_full + st);
      }
      pass(p, l, g);
      ++seg;
    }
  } else {
    // ======================= softmax of 128 rows ================================
    regs_up<C::regs>();
    const int m = wg, r = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    int unit = 0, seg = 0;
    bool ok = true;
    while (ok && l.more()) {
      const Seg g = seg_at(p, l, kRows);
      const int row = g.row0 + m * 128 + r;
      const bool live = m * 128 + r < g.n_rows;
      const int tok = row / G, hq = l.head * G + row - tok * G;
      ok = ok && warp_wait(q_full + (seg & 1), (seg >> 1) & 1, s_abort);
      if (!ok) break;
      const int ex = s_ex[(seg & 1) * kRows + m * 128 + r];
      const int lim = live ? visible(g.s, tok) : 0;
      // A row without keys has zeros whatever its q holds: no NaN meets its masked scores.
      const float rs = lim == 0 ? 0.f : fabsf(p.scale_log2) * (ex == -128 ? __int_as_float(0x7fffffff)
                                                                          : __int_as_float((ex + 127) << 23));
      const int min_lim = visible(g.s, (g.row0 + m * 128) / G);
      const int nan_base = visible(g.s, g.row0 / G) - kKeys;
      const bool part_tile = m * 128 + 128 > g.n_rows;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < g.count; ++j, ++unit) {
        const int buf = m * 2 + (unit & 1);
        // The unit's scales, long there, before its scores.
        ok = ok && warp_wait(sc_full + (unit & 7), (unit >> 3) & 1, s_abort);
        const float* sc = s_sc + (unit & 7) * 12;
        float fa[4], fb[4], fi[4];
        *reinterpret_cast<float4*>(fa) = *reinterpret_cast<const float4*>(sc);
        *reinterpret_cast<float4*>(fb) = *reinterpret_cast<const float4*>(sc + 4);
        *reinterpret_cast<float4*>(fi) = *reinterpret_cast<const float4*>(sc + 8);
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) fa[gr] = factor(rs * fa[gr]);
        ok = ok && warp_wait(s_full + buf, (unit >> 1) & 1, s_abort);
        if (!ok) break;
        tc::fence_after_sync();
        float x[64];
        const uint32_t ts = tmem + lane_base + m * 128 + (unit & 1) * 64;
        tmem_ld32_async(ts, x);
        tmem_ld32_async(ts + 32, x + 32);
        tmem_wait_ld();
        const int key0 = (g.first_unit + j) * kKeys;
        if (part_tile || key0 + kKeys > min_lim) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (key0 + k >= lim) x[k] = -INFINITY;
        }
        // The weights on the running maximum as it was, beside this unit's maximum:
        // neither waits for the other. Where the maximum grew by more than 2^8 (the
        // first unit, and few others), once more on the new one.
        uint32_t pk[32];
        float lsum;
        bool again, far = false;
#pragma unroll 1
        do {
          const float ref = (m_run == -INFINITY ? 0.f : m_run) - 7.f;
          float mx = -INFINITY;
          lsum = 0.f;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr) {
            const float* y = x + gr * 16;
            const float2 a2 = make_float2(fa[gr], fa[gr]), b2 = make_float2(fb[gr] - ref, fb[gr] - ref);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 v = fma2(make_float2(y[2 * k], y[2 * k + 1]), a2, b2);
              v.x = ex2_approx(v.x);
              v.y = ex2_approx(v.y);
              sum = add2(sum, v);
              const __half2 h = __floats2half2_rn(v.x, v.y);
              pk[gr * 8 + k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            lsum = fmaf(sum.x + sum.y, fi[gr], lsum);
            const float t0 = max3(y[0], y[1], y[2]), t1 = max3(y[3], y[4], y[5]), t2 = max3(y[6], y[7], y[8]),
                        t3 = max3(y[9], y[10], y[11]), t4 = max3(y[12], y[13], y[14]);
            mx = fmaxf(mx, fmaf(max3(max3(t0, t1, t2), max3(t3, t4, y[15]), -INFINITY), fa[gr], fb[gr]));
          }
          again = false;
          // More than 8 above the running maximum, or kFarUnit below.
          const bool apart = fi[0] < 0.f;
          if (!__any_sync(0xffffffffu, apart || fabsf(mx - m_run + (kFarUnit - 8.f) * 0.5f) > (kFarUnit + 8.f) * 0.5f))
            break;
          again = __any_sync(0xffffffffu, mx > m_run + 8.f);
          if (!again) {
            far = __any_sync(0xffffffffu, apart || (mx < m_run - kFarUnit && mx > -INFINITY));
          } else {
            const float m_new = fmaxf(mx, m_run);
            const float x_al = m_new > m_run ? m_run - m_new : 0.f, al = ex2_approx(x_al);
            m_run = m_new;
            l_run = add_scaled(0.f, l_run, al, x_al);
            if (j > 0) {
              // The products of the unit before are in O; this unit's wait for P.
              ok = warp_wait(o_done + m * 2 + ((unit - 1) & 1), ((unit - 1) >> 1) & 1, s_abort);
              if (!ok) break;
              tc::fence_after_sync();
              const uint32_t to = tmem + lane_base + C::c_o(m);
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float v[16];
                tmem_ld16(to + c, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] *= al;
                tc::tmem_st16(to + c, *reinterpret_cast<uint32_t(*)[16]>(v));
              }
            }
          }
        } while (again);
        if (!ok) break;
        if (far) {                       // the sum anew, from the scores
          const float ref = (m_run == -INFINITY ? 0.f : m_run) - 7.f;
          lsum = 0.f;
#pragma unroll 1
          for (int gr = 0; gr < 4; ++gr) {
            float y[16];
            tmem_ld16(ts + gr * 16, y);
            const float iv = fabsf(sc[8 + gr]), a = factor(rs * sc[gr]), b = sc[4 + gr] - ref + far_shift(iv);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              sum += key0 + gr * 16 + k < lim ? ex2_approx(fmaf(y[k], a, b)) : 0.f;
            lsum = fmaf(sum, far_factor(iv), lsum);
          }
        }
        l_run += lsum;
        tmem_st32_async(ts, pk);
        tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(p_full + buf);
      }
      if (!ok) break;
      // ---- results -------------------------------------------------------------
      ok = warp_wait(o_done + m * 2 + ((unit - 1) & 1), ((unit - 1) >> 1) & 1, s_abort);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t to = tmem + lane_base + C::c_o(m);
      const bool whole = g.count == g.n_units;
      __nv_bfloat16* out = p.o + ((int64_t)(g.s.first + tok) * p.Hq + hq) * D;
      const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
      const float il = over_sum(l_run);
      const size_t part_sz = (size_t)(D + 2) * 128;
      float* part = p.tile_partials +
                    (((size_t)blockIdx.x * 2 + (g.first_unit == 0 ? 1 : 0)) * kM + m) * part_sz;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        tmem_ld32_async(to + c, v);
        tmem_wait_ld();
        if (*s_any_nan) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int first = s_nan[(seg % C::NR) * D + c + k];
            if (first != 0xffff && lim > nan_base + first) v[k] = NAN;
          }
        }
        if (whole) {
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = put_one(v[k], il);
            store16(out + c, v, wide);
            store16(out + c + 16, v + 16, wide);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) __stcg(part + (size_t)(2 + c + k) * 128 + r, v[k]);
        }
      }
      if (!whole) {
        __stcg(part + r, m_run);
        __stcg(part + 128 + r, l_run);
      }
      tc::fence_before_sync();
      pass(p, l, g);
      ++seg;
    }
  }
  // Every role is here, done or given up.
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 12) tc::tmem_dealloc(tmem, 512);
  if constexpr (kAfterSplit) {
    pdl_wait();
    pdl_trigger();
  }
}

template <int D, bool kAfterSplit>
gdn_status_t launch_tile(const Args& a, cudaStream_t st) {
  static const cudaError_t set = cudaFuncSetAttribute(
      attn_tile_kernel<D, kAfterSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, TC<D>::total);
  if (set != cudaSuccess) return check_launch(set);
  const int B = 1 << a.log_b;
  const int64_t pages = (int64_t)a.num_blocks * a.Hk;
  CUtensorMap k_map, v_map;
  if (!cache_map(&k_map, a.kc, D, B, pages, std::min(B, kKeys)) ||
      !cache_map(&v_map, a.vc, D, B, pages, std::min(B, kKeys))) {
    set_cuda_error(cudaErrorInvalidValue);
    return GDN_ERR_CUDA;
  }
  return check_launch(launch_pdl(attn_tile_kernel<D, kAfterSplit>, dim3(a.tile_grid), dim3(kThreads), TC<D>::total, st, a,
                                 k_map, v_map));
}

}  // namespace

namespace attn {

namespace {
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
}  // namespace

// The cache as (d, token of the block, block x head), boxes of `rows` tokens.
bool cache_map(CUtensorMap* map, const void* cache, int d, int B, int64_t pages, int rows) {
  const int row = box_row(d);
  static const EncodeTiled encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)B, (cuuint64_t)(pages > 0 ? pages : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)d * B};
  const cuuint32_t box[3] = {(cuuint32_t)row, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(cache), dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn

gdn_status_t launch_attn_tile(const Args& a, cudaStream_t st) {
  if (a.d == 64) return a.after_split ? launch_tile<64, true>(a, st) : launch_tile<64, false>(a, st);
  if (a.d == 128) return a.after_split ? launch_tile<128, true>(a, st) : launch_tile<128, false>(a, st);
  return a.after_split ? launch_tile<256, true>(a, st) : launch_tile<256, false>(a, st);
}

GDN_DEFINE_STATUS_GATHER(gather_status_attn_tile)

}  // namespace gdn
