// Attention of few query rows over a paged 8-bit cache, split over the keys.
//
// Bound: every K and V byte is read once (2 d bytes per token and kv head) for
// 4 d G operations, G <= 16 rows: 16 to 32 operations a byte, so HBM bounds it
// as long as the tensor cores do the products and few other instructions run
// per byte. Hence:
//
// * One unit = 32 keys. A warp owns whole units (running maximum, sum and
//   output of its own; no block barrier in the loop) and streams them through
//   a private ring of TMA slots, K and V alternating.
// * S = Q K^T on e4m3 MMAs (m16n8k32): K goes to the tensor core as it lies in
//   the cache. Q is split into two e4m3 parts, hi + lo, which together hold
//   BF16's 8 significand bits; hi is rows 0-7 of the A tile and lo rows 8-15,
//   so 8 query rows fill the 16-row MMA and both parts of a row's sum meet in
//   one thread.
// * O^T = V^T P^T on f16 MMAs (m16n8k16): V^T is the 16-row operand (no row is
//   wasted on few queries), P^T the 8-column one, whose register layout is
//   that of the scores. V codes become f16 exactly (e4m3 is a subset); P is
//   rounded to f16 (11 bits) on a scale of 2^7 to 2^15, so that a key whose
//   weight is 2^-21 of the largest one's still keeps its digits.
// * The block's V scale enters the exponent: P' = 2^(s + log2 vs - m), and the
//   sum takes P' / vs. Blocks of any scale then share one accumulator, and the
//   largest contribution, not the largest weight, sets the range. Where scales lie so
//   far apart that a P' leaves float32's range while P' / vs does not, the sum takes
//   it on another range (kFarUnit).
// * The accumulator is rescaled only when a row's maximum grows by more than
//   2^8 (the headroom of P's range): most units skip it.
//
// Work split: all units of all (tile, head) items form one line that is cut into
// pieces, one per CTA; a piece may end inside an item. Such items leave float32
// partial results in the workspace, which another kernel joins in a fixed order
// (equal inputs give equal bits). Joining inside this kernel, by the CTA that
// arrives last, took as long as that launch does, and its code cost the stream its
// registers (48 requests of 3k-30k tokens: 232 -> 335 us).
//
// Measured: 48 requests of 3k-30k tokens, 32 query and 8 kv heads of 128, 1.42 GB:
// 234 us, 6.1 TB/s, 90% of the copy rate. 16 rows a tile (12 heads a kv head) have
// twice the instructions a byte and half of the warps: 64%. 32 requests of 512 to
// 1,143 tokens, 16 + 2 heads of 256, 28 MB: 16.0 us (planned once a step: 14.2), of
// which 10.7 are there for a single request.
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_attn.cuh"

namespace gdn {

namespace {
using namespace attn;

// ---------------------------------------------------------------------------
// MMA and copy wrappers
// The MMAs are volatile: they stay in front of the copy that refills the slot whose
// keys they take (see `issue`).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The low (high) two e4m3 codes of a word as a pair of f16 (exact).
__device__ __forceinline__ uint32_t half2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t half2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// ---------------------------------------------------------------------------
// Split kernel
// ---------------------------------------------------------------------------

template <int D, int QM>
struct Cfg {
  static constexpr int rows = 8 * QM;
  // CTAs per SM, by registers: 128 a thread hold O of 8 rows up to d = 128 and of
  // 16 up to d = 64; the others have the SM to themselves.
  static constexpr int ctas = D * QM <= 128 ? 2 : 1;
  static constexpr int slots = D == 128 && QM == 2 ? 6 : 3;   // half units (K or V) in a warp's ring
  // Q's fragments stay in registers for 8 rows; for 16 they are read from shared
  // memory (100 requests of 3k-30k tokens, 12 heads a kv head of 128: 191 -> 184 us;
  // 16 of 64: 178 -> 168; for 8 rows of 128 233 -> 234), rows 64 bytes off a bank
  // line: two rows x four chunks at once.
  static constexpr bool q_in_regs = QM == 1;
  static constexpr int q_pitch = 2 * D + 64;
  static constexpr int slot_bytes = kUnit * D;
  static constexpr int row = box_row(D), boxes = D / row;
  static constexpr int ring = kWarps * slots * slot_bytes;
  static constexpr int q_bytes = rows * q_pitch;       // hi | lo codes of each row
  static constexpr int o_pitch = D + 4;                // of a row of O while the warps join
  static_assert(kWarps * rows * o_pitch * 4 <= ring, "the warps' O fits the rings");
  // ring | Q | Q row scales | m, l and factor of each warp's rows | joined m, l |
  // first key whose V is NaN in a column | barriers | flags
  static constexpr int o_q = ring;
  static constexpr int o_qs = o_q + q_bytes;
  static constexpr int o_ml = o_qs + rows * 4;
  static constexpr int o_l = o_ml + kWarps * rows * 3 * 4;
  static constexpr int o_nan = o_l + rows * 2 * 4;
  static constexpr int o_bar = o_nan + D * 4;
  static constexpr int o_flag = o_bar + kWarps * slots * 8;
  static constexpr int o_cum = o_flag + 16;            // units and pieces before each sequence (self plan)
  static constexpr int total = o_cum + (2 * kSelfPlan + 1) * 4;
};

// The K rows of an MMA's 8 columns and the V rows of its k index are free to
// choose, as long as both agree. Column n is key 8 j + n / 2 + 4 (n % 2) where
// rows are 128 bytes: with TMA's swizzle (chunk XOR row) the 8 lanes of a K read
// (2 rows x 4 chunks) and of a V read (4 rows x 2 chunks) then touch all banks
// once. 64-byte rows take key 8 j + n (their V reads take two passes).
template <int D>
__device__ __forceinline__ int key_of(int n) {
  if constexpr (D == 64) return n;
  return (n >> 1) + 4 * (n & 1);
}
// Takes this lane's NaNs of V out of a slot and keeps the first key of each of
// their columns; true if there were any. (Out of line: few units need it, and
// its registers are not the stream's.)
template <int D>
__device__ __noinline__ bool take_nans(unsigned char* slot, int* first_nan, int key0) {
  constexpr int row = box_row(D);
  bool any = false;
#pragma unroll 1
  for (int at = (threadIdx.x & 31) * 4; at < kUnit * D; at += 128) {
    const uint32_t word = *reinterpret_cast<const uint32_t*>(slot + at);
    if ((((word & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) == 0) continue;
    const int box = at / (kUnit * row), r = at / row % kUnit;
    // The swizzle is its own inverse.
    const int col = box * row + swizzled<row>(r, at % row / 16) - r * row + at % 16;
    for (int c = 0; c < 4; ++c)
      if (((word >> (8 * c)) & 0x7fu) == 0x7fu) {
        atomicMin(first_nan + col + c, key0 + r);
        slot[at + c] = 0;
      }
    any = true;
  }
  return any;
}

// This lane's sum of a unit's weights where V scales lie far apart (kFarUnit).
__device__ __forceinline__ float far_sum(float4 x0, float4 x1, float ref, float iv0, float iv1) {
  auto e = [](float x) { return ex2_approx(x); };
  const float a = ref - far_shift(iv0), b = ref - far_shift(iv1);
  return fmaf(e(x0.x - a) + e(x0.y - a) + e(x0.z - a) + e(x0.w - a), far_factor(iv0),
              (e(x1.x - b) + e(x1.y - b) + e(x1.z - b) + e(x1.w - b)) * far_factor(iv1));
}

// Largest value of the block. (Out of line: few steps need it.)
__device__ __noinline__ int block_max(int x, int* warps) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = x;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) x = max(x, warps[k]);
  return x;
}

template <int D, int QM>
__global__ void __launch_bounds__(kWarps * 32, Cfg<D, QM>::ctas)
attn_split_kernel(const Args p, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D, QM>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_q = smem + C::o_q;
  float* s_qs = reinterpret_cast<float*>(smem + C::o_qs);
  float* s_ml = reinterpret_cast<float*>(smem + C::o_ml);
  float* s_l = reinterpret_cast<float*>(smem + C::o_l);
  int* s_nan = reinterpret_cast<int*>(smem + C::o_nan);
  int* s_flag = reinterpret_cast<int*>(smem + C::o_flag);   // a NaN in V | gave up
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  unsigned char* ring = smem + w * (C::slots * C::slot_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::o_bar) + w * C::slots;
  const int G = p.Hq / p.Hk, B = 1 << p.log_b;
  const int log_box = min(p.log_b, 5);                 // tokens of a TMA box, and boxes of a half unit
  const int pages = kUnit >> log_box;
  const int page = lane & (pages - 1), bx = lane >> (5 - log_box);
  const bool posts = bx < C::boxes;
  const int absent = max(p.num_blocks * p.Hk, 1);      // a box past the end reads zeros

  if (lane < C::slots) tc::mbar_init(full + lane, 1);
  if (tid == 0) s_flag[1] = 0;
  __syncwarp();
  bool dead = false;                                   // a wait of this warp ran out
  int posted = 0, taken = 0;                           // half units, over all segments
  pdl_wait();
  pdl_trigger();
  Start start;
  int* s_cum = reinterpret_cast<int*>(smem + C::o_cum);
  if (p.self_plan) {
    // One tile a sequence: every CTA forms the line itself (one round of loads and
    // a scan or two), which is sooner than a kernel before this one.
    int2* sums = reinterpret_cast<int2*>(s_ml);
    int* s_pieces = s_cum + kSelfPlan + 1;
    constexpr int per = kSelfPlan / (kWarps * 32);
    int u4[per];
    int2 mine = make_int2(0, 0), total;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int n = tid * per + k;
      u4[k] = 0;
      if (n < p.N) {
        const Seq q = seq_of(p.cu, p.kv, n, p.T, (int64_t)p.max_blocks << p.log_b);
        if (q.len > 0) u4[k] = max(1, (visible(q, q.len - 1) + kUnit - 1) / kUnit);
      }
      mine.x += u4[k];
      mine.y += u4[k] > 0;
    }
    // Exclusive sums of a pair over the block.
    auto scan = [&](int2 v, int2& tot) {
      int2 inc = v;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, k), y = __shfl_up_sync(0xffffffffu, inc.y, k);
        if (lane >= k) { inc.x += x; inc.y += y; }
      }
      __syncthreads();
      if (lane == 31) sums[w] = inc;
      __syncthreads();
      int2 before = make_int2(inc.x - v.x, inc.y - v.y);
      tot = make_int2(0, 0);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        if (k < w) { before.x += sums[k].x; before.y += sums[k].y; }
        tot.x += sums[k].x;
        tot.y += sums[k].y;
      }
      return before;
    };
    const int2 both = scan(mine, total);
    int before = both.x, cost = both.x + both.y * kSplitOver;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      s_cum[tid * per + k] = before;
      s_pieces[tid * per + k] = cost;
      before += u4[k];
      cost += u4[k] + (u4[k] > 0 ? kSplitOver : 0);
    }
    if (tid == 0) s_cum[kSelfPlan] = total.x;
    const long long all = (long long)total.x * p.Hk;
    int longest = 0;
    if (by_longest((long long)total.y * p.Hk, gridDim.x)) {
#pragma unroll
      for (int k = 0; k < per; ++k) longest = max(longest, u4[k]);
      longest = block_max(longest, reinterpret_cast<int*>(sums + kWarps));
    }
    const Cut cut = cut_of(all, (long long)total.y * p.Hk, longest, gridDim.x, kWarps, kSplitOver);
    const int cost_all = total.x + total.y * kSplitOver;
    int pieces = 0;                      // of one head
    if (cut.target) {
      int2 n = make_int2(0, 0), tot;
#pragma unroll
      for (int k = 0; k < per; ++k) n.x += (u4[k] + cut.target - 1) / cut.target;
      before = scan(n, tot).x;
#pragma unroll
      for (int k = 0; k < per; ++k) {
        s_pieces[tid * per + k] = before;
        before += (u4[k] + cut.target - 1) / cut.target;
      }
      pieces = tot.x;
    }
    __syncthreads();
    const int c = blockIdx.x;
    start.num_items = p.N;
    start.units = total.x;
    start.u = all;
    start.item = start.head = start.count = start.pieces = start.first = start.len = start.kv = start.c0 = 0;
    start.it = {0, 0, 0, 0};
    int y = 0;
    bool work;
    if (cut.target) {
      work = pieces > 0 && c < pieces * p.Hk;
      if (work) {
        start.head = c / pieces;
        y = c - start.head * pieces;
        start.item = find_item(p.N, y, [&](int i) { return s_pieces[i]; });
      }
    } else {
      work = piece_of_line(start, c, p.Hk, cost_all, cut.per_cta, kSplitOver,
                           [&](int i) { return s_pieces[i]; }, [&](int i) { return s_cum[i]; });
    }
    if (work) {
      const int i = start.item;
      start.it = {i, 0, s_cum[i + 1] - s_cum[i], s_cum[i]};
      const Seq q = seq_of(p.cu, p.kv, i, p.T, (int64_t)p.max_blocks << p.log_b);
      start.first = q.first;
      start.len = q.len;
      start.kv = q.kv;
      if (cut.target) piece_of(start, c, y - s_pieces[i], (start.it.units + cut.target - 1) / cut.target);
      else pieces_of_line(start, (long long)start.head * cost_all + s_pieces[i], cut.per_cta, kSplitOver);
    }
    if (tid < 4)                         // for the joining kernel
      reinterpret_cast<int4*>(p.starts + blockIdx.x)[tid] = reinterpret_cast<const int4*>(&start)[tid];
  } else {
    start = read_start(p.starts + blockIdx.x);
  }
  const int num_items = start.num_items, units1 = start.units;
  long long u = start.u;
  const long long u_end = u + start.count;
  int lo = start.item, head = start.head;
  Item it = start.it;
  Seq s = {start.first, start.len, start.kv};

  while (u < u_end) {
    const int x = (int)(u - (long long)head * units1);
    const int seq = it.seq, row0 = it.row0, n_units = it.units, cum = it.cum;
    const int first_unit = x - cum;
    const int seg = (int)min((long long)(n_units - first_unit), u_end - u);
    const int n_rows = min(C::rows, s.len * G - row0);
    const int key_end = visible(s, (row0 + n_rows - 1) / G);      // keys of the last row
    const int32_t* table = p.table + (int64_t)seq * p.table_stride;

    // ---- this warp's units: first_unit + w, + 8, ... --------------------------
    const int mine = seg > w ? (seg - w + kWarps - 1) / kWarps : 0;
    // Q's rows of this warp, on their way before the first table read is waited for.
    constexpr int per = D / 32;
    uint32_t q_raw[QM][per / 2];
#pragma unroll
    for (int rq = 0; rq < QM; ++rq) {
      const int r = w + rq * kWarps;
      const int row = row0 + r, tok = row / G;
      const __nv_bfloat16* src = p.q + (int64_t)(s.first + tok) * p.q_stride +
                                 (int64_t)(head * G + row - tok * G) * D + lane * per;
#pragma unroll
      for (int i = 0; i < per / 2; ++i)
        q_raw[rq][i] = r < n_rows ? __ldg(reinterpret_cast<const uint32_t*>(src) + i) : 0u;
    }
    // Block of this lane's box of unit i; read a unit before it is needed.
    auto block_of = [&](int i) {
      const int key = (first_unit + w + i * kWarps) * kUnit + (page << log_box);
      return i < mine && key < key_end ? __ldg(table + (key >> p.log_b)) : -1;
    };
    int blk = -1, blk_next = block_of(0);
    // Scales of the units being copied, in order: lane l & 3 holds K's of the unit's
    // two halves and V's.
    constexpr int kAhead = C::slots / 2;
    float sc_q[kAhead];
    // Half unit h into the ring's next slot, whose last one this warp has read: the
    // copy must not land before those reads have their data, and it is not ordered
    // behind loads that are merely issued. It need not be: every load from a slot feeds
    // an MMA of the same half unit, a warp issues in program order, and an MMA issues
    // only once its registers have arrived. So it is enough that a slot's MMAs stand in
    // front of its refill: they and the copy are volatile, with the wait for the next
    // half unit between them, and __syncwarp() joins the lanes.
    auto issue = [&](int h, int q) {
      const int i = h >> 1, is_v = h & 1;
      if (i >= mine || dead) return;
      const int key0 = (first_unit + w + i * kWarps) * kUnit;
      if (!is_v) {
        blk = blk_next;
        blk_next = block_of(i + 1);
        const int half = lane & 1;
        const int b = __shfl_sync(0xffffffffu, blk, pages == 2 ? half : 0);
        sc_q[q] = 1.f;
        if (key0 + half * 16 < key_end) {
          if ((unsigned)b < (unsigned)p.num_blocks)
            sc_q[q] = __ldg(((lane & 2) ? p.vs : p.ks) + (size_t)b * p.Hk + head);
          else
            record_device_status(GDN_ERR_INVALID_ARG);
        }
      }
      const int st = posted % C::slots;
      if (lane == 0) tc::mbar_arrive_expect_tx(full + st, C::slot_bytes);
      __syncwarp();
      if (posts)
        tma_box(ring + st * C::slot_bytes + (bx * kUnit + (page << log_box)) * C::row,
                is_v ? &v_map : &k_map, bx * C::row, (key0 + (page << log_box)) & (B - 1),
                (unsigned)blk < (unsigned)p.num_blocks ? blk * p.Hk + head : absent, full + st);
      ++posted;
    };
    // The next half unit in order; its slot.
    auto take = [&]() {
      const int st = taken % C::slots;
      if (!dead && !__all_sync(0xffffffffu, tc::mbar_wait(full + st, (taken / C::slots) & 1))) {
        dead = true;
        s_flag[1] = 1;
        record_device_status(GDN_ERR_TIMEOUT);
      }
      ++taken;
      return ring + st * C::slot_bytes;
    };
#pragma unroll
    for (int h = 0; h < C::slots - 1; ++h) issue(h, h >> 1);

    for (int i = tid; i < D; i += kWarps * 32) s_nan[i] = 0x7fffffff;
    if (tid == 0) s_flag[0] = 0;

    // ---- Q of the tile: hi and lo codes, one power-of-two scale per row -------
#pragma unroll
    for (int rq = 0; rq < QM; ++rq) {
      const int r = w + rq * kWarps;
      float v[per];
      float top = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < per; i += 2) {
        v[i] = bf16lo(q_raw[rq][i / 2]);
        v[i + 1] = bf16hi(q_raw[rq][i / 2]);
      }
#pragma unroll
      for (int i = 0; i < per; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        bad |= !(fabsf(v[i]) <= 3.4e38f);
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      bad = __any_sync(0xffffffffu, bad);
      // Bring the row's largest magnitude into [128, 256); rows of zeros (and of
      // values below 2^-119) keep the smallest scale.
      const int ex = max((int)((__float_as_uint(top) >> 23) & 255) - 127 - 7, -126);
      const float inv = __int_as_float((127 - min(ex, 126)) << 23);
#pragma unroll
      for (int i = 0; i < per; i += 2) {
        const float a = bad ? 0.f : v[i] * inv, b = bad ? 0.f : v[i + 1] * inv;
        const uint32_t h2 = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t f = half2_lo(h2);
        const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&f));
        const uint32_t l2 = __nv_cvt_float2_to_fp8x2(make_float2(a - hf.x, b - hf.y),
                                                     __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint16_t*>(s_q + r * C::q_pitch + lane * per + i) = (uint16_t)h2;
        *reinterpret_cast<uint16_t*>(s_q + r * C::q_pitch + D + lane * per + i) = (uint16_t)l2;
      }
      // A row with an infinity or NaN has no finite softmax: its scores are NaN.
      if (lane == 0)
        s_qs[r] = bad ? __int_as_float(0x7fffffff) : __int_as_float((ex + 127) << 23);
    }
    __syncthreads();

    // ---- Q fragments: chunk t4 + 4 c of a row, hi and lo, as K's chunks below -----
    uint4 qf[C::q_in_regs ? QM : 1][C::q_in_regs ? D / 64 : 1][2];
    float rs[QM];
    int lim[QM];
    int min_lim = 0x7fffffff;
#pragma unroll
    for (int m = 0; m < QM; ++m) {
      if constexpr (C::q_in_regs) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const unsigned char* at = s_q + (m * 8 + g) * C::q_pitch + 16 * (t4 + 4 * c);
          qf[m][c][0] = *reinterpret_cast<const uint4*>(at);
          qf[m][c][1] = *reinterpret_cast<const uint4*>(at + D);
        }
      }
      rs[m] = s_qs[m * 8 + g] * p.scale_log2;
      const int r = m * 8 + g;
      lim[m] = visible(s, (row0 + min(r, n_rows - 1)) / G);
      if (r < n_rows) min_lim = min(min_lim, lim[m]);
    }
    min_lim = __reduce_min_sync(0xffffffffu, min_lim);

    // ---- the stream ----------------------------------------------------------
    float acc[QM][D / 16][4];            // O^T: (d row g | g + 8, query 2 t4 | 2 t4 + 1)
    float m_run[QM], l_run[QM];
#pragma unroll
    for (int m = 0; m < QM; ++m) {
      m_run[m] = -INFINITY;
      l_run[m] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][i][c] = 0.f;
    }

    for (int i = 0; i < mine && !dead; ++i) {
      const int unit = first_unit + w + i * kWarps;
      // The unit's scales, before those of the next one replace them.
      float ksc[2], lvs[2], ivs[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ksc[k] = __shfl_sync(0xffffffffu, sc_q[0], k);
        const float v = fmaxf(__shfl_sync(0xffffffffu, sc_q[0], 2 + k), 7.888609052210118e-31f);   // 2^-100
        lvs[k] = lg2_approx(v);
        ivs[k] = __fdividef(kSumScale, v);
      }
      const bool apart = fabsf(lvs[0] - lvs[1]) > kFarApart;
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) sc_q[k] = sc_q[k + 1];
      // K of unit i has landed, and the slot before it is free again.
      float sc[QM][4][2];
      {
        const unsigned char* slot = take();
        issue(2 * i + C::slots - 1, kAhead - 1);
        float c4[QM][4][4];
#pragma unroll
        for (int m = 0; m < QM; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) c4[m][j][c] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 qh[QM], ql[QM];
          if constexpr (!C::q_in_regs) {
#pragma unroll
            for (int m = 0; m < QM; ++m) {
              const unsigned char* at = s_q + (m * 8 + g) * C::q_pitch + 16 * (t4 + 4 * c);
              qh[m] = *reinterpret_cast<const uint4*>(at);
              ql[m] = *reinterpret_cast<const uint4*>(at + D);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + key_of<D>(g);
            const uint4 kk = *reinterpret_cast<const uint4*>(
                slot + (c >> 1) * (kUnit * C::row) + swizzled<C::row>(r, t4 + 4 * (c & 1)));
#pragma unroll
            for (int m = 0; m < QM; ++m) {
              if constexpr (C::q_in_regs) {
                mma_e4m3(c4[m][j], qf[m][c][0].x, qf[m][c][1].x, qf[m][c][0].y, qf[m][c][1].y, kk.x, kk.y);
                mma_e4m3(c4[m][j], qf[m][c][0].z, qf[m][c][1].z, qf[m][c][0].w, qf[m][c][1].w, kk.z, kk.w);
              } else {
                mma_e4m3(c4[m][j], qh[m].x, ql[m].x, qh[m].y, ql[m].y, kk.x, kk.y);
                mma_e4m3(c4[m][j], qh[m].z, ql[m].z, qh[m].w, ql[m].w, kk.z, kk.w);
              }
            }
          }
        }
#pragma unroll
        for (int m = 0; m < QM; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sc[m][j][0] = c4[m][j][0] + c4[m][j][2];
            sc[m][j][1] = c4[m][j][1] + c4[m][j][3];
          }
      }
      __syncwarp();
      unsigned char* slot = take();                      // V of unit i
      issue(2 * i + C::slots, kAhead - 1);
      const bool cut = unit * kUnit + kUnit > min_lim;
      // Keys past the end hold stale bytes: zeros instead.
      if (unit * kUnit + kUnit > key_end) {
        const int past = max(0, key_end - unit * kUnit) * C::row;       // bytes of the rows before
#pragma unroll 1
        for (int box = 0; box < C::boxes; ++box)
#pragma unroll 1
          for (int at = past + lane * 16; at < kUnit * C::row; at += 512)
            *reinterpret_cast<uint4*>(slot + box * (kUnit * C::row) + at) = make_uint4(0, 0, 0, 0);
        tc::fence_smem_to_async();                       // before the next copy into the slot
        __syncwarp();
      }
      // Where the rows of the tile do not see the same keys, a weight of zero must not
      // meet a NaN (0 x NaN is NaN): a NaN of V is taken out of the slot and kept as
      // the first key whose column has one.
      if (cut && min_lim < key_end) {
        if (take_nans<D>(slot, s_nan, unit * kUnit)) s_flag[0] = 1;
        tc::fence_smem_to_async();
        __syncwarp();
      }
      uint32_t pf[QM][4];
#pragma unroll
      for (int m = 0; m < QM; ++m) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float xx = fmaf(sc[m][j][e], rs[m] * ksc[j >> 1], lvs[j >> 1]);
            if (cut && unit * kUnit + 8 * j + key_of<D>(2 * t4 + e) >= lim[m]) xx = -INFINITY;
            sc[m][j][e] = xx;
            mx = fmaxf(mx, xx);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // More than 8 above the running maximum, or kFarUnit below.
        float far = 0.f;
        if (__any_sync(0xffffffffu, apart || fabsf(mx - m_run[m] + (kFarUnit - 8.f) * 0.5f) > (kFarUnit + 8.f) * 0.5f)) {
          const float m_old = m_run[m], m_new = fmaxf(mx, m_old);
          const float al = m_new > m_old ? ex2_approx(m_old - m_new) : 1.f;
          m_run[m] = m_new;
          l_run[m] = add_scaled(0.f, l_run[m], al, m_new > m_old ? m_old - m_new : 0.f);
          const float a0 = __shfl_sync(0xffffffffu, al, 8 * t4);
          const float a1 = __shfl_sync(0xffffffffu, al, 8 * t4 + 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            acc[m][k][0] *= a0;
            acc[m][k][1] *= a1;
            acc[m][k][2] *= a0;
            acc[m][k][3] *= a1;
          }
          if (__any_sync(0xffffffffu, apart || (mx < m_new - kFarUnit && mx > -INFINITY)))
            far = far_sum(make_float4(sc[m][0][0], sc[m][0][1], sc[m][1][0], sc[m][1][1]),
                          make_float4(sc[m][2][0], sc[m][2][1], sc[m][3][0], sc[m][3][1]),
                          (m_new == -INFINITY ? 0.f : m_new) - 7.f, ivs[0], ivs[1]);
        }
        const float ref = (m_run[m] == -INFINITY ? 0.f : m_run[m]) - 7.f;
        float lsum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p0 = ex2_approx(sc[m][j][0] - ref), p1 = ex2_approx(sc[m][j][1] - ref);
          lsum = fmaf(p0 + p1, ivs[j >> 1], lsum);
          pf[m][j] = pack_half2(p0, p1);
        }
        l_run[m] += far == 0.f ? lsum : far;
      }
      // O^T += V^T P^T: the two rows of m-tile k are bytes 2k and 2k + 1 of the
      // lane's own 16-byte chunk (8-byte one for d = 64) of the V rows.
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (D == 64) {
          uint2 va[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 16 * ks + 8 * (k >> 1) + key_of<D>(2 * t4 + (k & 1));
            va[k] = *reinterpret_cast<const uint2*>(slot + swizzled<C::row>(r, g >> 1) + (g & 1) * 8);
          }
          const uint32_t wv[4][2] = {{va[0].x, va[0].y}, {va[1].x, va[1].y},
                                     {va[2].x, va[2].y}, {va[3].x, va[3].y}};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t xa = __byte_perm(wv[0][q], wv[1][q], 0x5140);
            const uint32_t xb = __byte_perm(wv[0][q], wv[1][q], 0x7362);
            const uint32_t ya = __byte_perm(wv[2][q], wv[3][q], 0x5140);
            const uint32_t yb = __byte_perm(wv[2][q], wv[3][q], 0x7362);
#pragma unroll
            for (int m = 0; m < QM; ++m) {
              mma_f16(acc[m][2 * q], half2_lo(xa), half2_hi(xa), half2_lo(ya), half2_hi(ya),
                      pf[m][2 * ks], pf[m][2 * ks + 1]);
              mma_f16(acc[m][2 * q + 1], half2_lo(xb), half2_hi(xb), half2_lo(yb), half2_hi(yb),
                      pf[m][2 * ks], pf[m][2 * ks + 1]);
            }
          }
        } else {
#pragma unroll
          for (int cc = 0; cc < D / 128; ++cc) {
            uint4 va[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 16 * ks + 8 * (k >> 1) + key_of<D>(2 * t4 + (k & 1));
              va[k] = *reinterpret_cast<const uint4*>(slot + cc * (kUnit * C::row) +
                                                      swizzled<C::row>(r, v_chunk(g)));
            }
            const uint32_t wv[4][4] = {{va[0].x, va[0].y, va[0].z, va[0].w},
                                       {va[1].x, va[1].y, va[1].z, va[1].w},
                                       {va[2].x, va[2].y, va[2].z, va[2].w},
                                       {va[3].x, va[3].y, va[3].z, va[3].w}};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t xa = __byte_perm(wv[0][q], wv[1][q], 0x5140);
              const uint32_t xb = __byte_perm(wv[0][q], wv[1][q], 0x7362);
              const uint32_t ya = __byte_perm(wv[2][q], wv[3][q], 0x5140);
              const uint32_t yb = __byte_perm(wv[2][q], wv[3][q], 0x7362);
              const uint32_t f0 = half2_lo(xa), f1 = half2_hi(xa), f2 = half2_lo(ya), f3 = half2_hi(ya);
              const uint32_t h0 = half2_lo(xb), h1 = half2_hi(xb), h2 = half2_lo(yb), h3 = half2_hi(yb);
#pragma unroll
              for (int m = 0; m < QM; ++m) {
                mma_f16(acc[m][8 * cc + 2 * q], f0, f1, f2, f3, pf[m][2 * ks], pf[m][2 * ks + 1]);
                mma_f16(acc[m][8 * cc + 2 * q + 1], h0, h1, h2, h3, pf[m][2 * ks], pf[m][2 * ks + 1]);
              }
            }
          }
        }
      }
      __syncwarp();
    }

    // ---- join the warps ------------------------------------------------------
#pragma unroll
    for (int m = 0; m < QM; ++m) {
      l_run[m] += __shfl_xor_sync(0xffffffffu, l_run[m], 1);
      l_run[m] += __shfl_xor_sync(0xffffffffu, l_run[m], 2);
      if (t4 == 0)
        *reinterpret_cast<float2*>(s_ml + (w * C::rows + m * 8 + g) * 2) = make_float2(m_run[m], l_run[m]);
    }
    __syncthreads();                     // also: every warp is done with its ring
    float* s_f = s_ml + kWarps * C::rows * 2;            // factors to the common maximum
    if (tid < C::rows) {
      float top = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_ml[(k * C::rows + tid) * 2]);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = *reinterpret_cast<const float2*>(s_ml + (k * C::rows + tid) * 2);
        // A warp without keys has zeros; a NaN row keeps m = -inf and its l, a NaN.
        const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
        s_f[k * C::rows + tid] = f;
        l = add_scaled(l, ml.y, f, ml.x - top);
      }
      s_l[tid * 2] = top;
      s_l[tid * 2 + 1] = l;
    }
    __syncthreads();
    // Each warp leaves its O, on the common maximum, as [row][m-tile][g][2]: rows
    // D + 4 floats apart, so that a store's 16 lanes touch all banks.
    float* s_o = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < QM; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = m * 8 + 2 * t4 + e;
        const float f = s_f[w * C::rows + r];
        float* dst = s_o + (w * C::rows + r) * C::o_pitch + 2 * g;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          *reinterpret_cast<float2*>(dst + 16 * k) = make_float2(acc[m][k][e] * f, acc[m][k][2 + e] * f);
      }
    __syncthreads();
    const bool whole = seg == n_units, gave_up = s_flag[1] != 0;
    float* part = p.partials + ((size_t)blockIdx.x * 2 + (first_unit == 0 ? 1 : 0)) * C::rows * (D + 2);
    const RowsOut out = {p.o, s.first, row0, gave_up ? 0 : n_rows, G, p.Hq, head};
#pragma unroll
    for (int e = tid * 4; e < C::rows * D; e += kWarps * 32 * 4) {
      const int r = e / D, pos = e % D;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(s_o + (k * C::rows + r) * C::o_pitch + pos);
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      if (s_flag[0] && r < n_rows) {
        const int lim_r = visible(s, (row0 + r) / G);
        if (lim_r > s_nan[d_of<D>(pos)]) o.x = NAN;
        if (lim_r > s_nan[d_of<D>(pos + 1)]) o.y = NAN;
        if (lim_r > s_nan[d_of<D>(pos + 2)]) o.z = NAN;
        if (lim_r > s_nan[d_of<D>(pos + 3)]) o.w = NAN;
      }
      if (whole) put_row4<D>(out, r, pos, o, s_l[r * 2 + 1]);
      else __stcg(reinterpret_cast<float4*>(part + 2 * C::rows + e), o);
    }
    if (!whole && tid < C::rows)
      __stcg(reinterpret_cast<float2*>(part) + tid, *reinterpret_cast<const float2*>(s_l + tid * 2));
    tc::fence_smem_to_async();           // before the next copies into the ring
    __syncthreads();                     // the ring, Q and s_ml are free again
    u += seg;
    if (u < u_end) {                     // the piece goes on with the next item
      if (++lo == num_items) {
        lo = 0;
        ++head;
      }
      if (p.self_plan) {
        while (s_cum[lo + 1] == s_cum[lo])               // sequences without new tokens
          if (++lo == num_items) {
            lo = 0;
            ++head;
          }
        it = {lo, 0, s_cum[lo + 1] - s_cum[lo], s_cum[lo]};
      } else {
        const int4 raw = __ldg(reinterpret_cast<const int4*>(p.items) + lo);
        it = {raw.x, raw.y, raw.z, raw.w};
      }
      s = seq_of(p.cu, p.kv, it.seq, p.T, (int64_t)p.max_blocks << p.log_b);
    }
  }
  // Copies of a warp that gave up land before its CTA may end.
  if (dead)
    for (int h = max(0, posted - C::slots); h < posted; ++h)
      tc::mbar_wait(full + h % C::slots, (h / C::slots) & 1);
}

template <int D, int QM>
gdn_status_t launch_split(const Args& a, cudaStream_t st) {
  static const cudaError_t set = cudaFuncSetAttribute(
      attn_split_kernel<D, QM>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, QM>::total);
  if (set != cudaSuccess) return check_launch(set);
  const int B = 1 << a.log_b;
  const int64_t pages = (int64_t)a.num_blocks * a.Hk;
  CUtensorMap k_map, v_map;
  if (!cache_map(&k_map, a.kc, D, B, pages, std::min(B, kUnit)) ||
      !cache_map(&v_map, a.vc, D, B, pages, std::min(B, kUnit))) {
    set_cuda_error(cudaErrorInvalidValue);
    return GDN_ERR_CUDA;
  }
  return check_launch(launch_pdl(attn_split_kernel<D, QM>, dim3(a.split_grid), dim3(kWarps * 32),
                                 Cfg<D, QM>::total, st, a, k_map, v_map));
}

}  // namespace

gdn_status_t launch_attn_split(const Args& a, cudaStream_t st) {
  const bool two = a.split_rows == 16;
  if (a.d == 64) return two ? launch_split<64, 2>(a, st) : launch_split<64, 1>(a, st);
  if (a.d == 128) return two ? launch_split<128, 2>(a, st) : launch_split<128, 1>(a, st);
  return two ? launch_split<256, 2>(a, st) : launch_split<256, 1>(a, st);
}

GDN_DEFINE_STATUS_GATHER(gather_status_attn_split)

}  // namespace gdn
