// Attention of few query rows over a paged 8-bit cache, split over the keys.
//
// Bound: every K and V byte is read once (2 d bytes per token and kv head) for
// 4 d G operations, G <= 16 rows: 16 to 32 operations a byte, so HBM bounds it
// as long as the tensor cores do the products and few other instructions run
// per byte. Hence:
//
// * One unit = 32 keys. A warp owns whole units (running maximum, sum and
//   output of its own; no block barrier in the loop) and streams them through
//   a private ring of cp.async slots, K and V alternating.
// * S = Q K^T on e4m3 MMAs (m16n8k32): K goes to the tensor core as it lies in
//   the cache. Q is split into two e4m3 parts, hi + lo, which together hold
//   BF16's 8 significand bits; hi is rows 0-7 of the A tile and lo rows 8-15,
//   so 8 query rows fill the 16-row MMA and both parts of a row's sum meet in
//   one thread.
// * O^T = V^T P^T on f16 MMAs (m16n8k16): V^T is the 16-row operand (no row is
//   wasted on few queries), P^T the 8-column one, whose register layout is
//   that of the scores. V codes become f16 exactly (e4m3 is a subset); P is
//   rounded to f16 (11 bits) on a scale of 2^7 to 2^15, so that a key whose
//   weight is 2^-29 of the largest one's still keeps its digits.
// * The block's V scale enters the exponent: P' = 2^(s + log2 vs - m), and the
//   sum takes P' / vs. Blocks of any scale then share one accumulator, and the
//   largest contribution, not the largest weight, sets the range.
// * The accumulator is rescaled only when a row's maximum grows by more than
//   2^8 (the headroom of P's range): most units skip it.
//
// Work split: all units of all (tile, head) items form one line that is cut
// into equal pieces, one per CTA; a piece may end inside an item. Such items
// leave float32 partial results in the workspace, and the CTA that arrives
// last at the item's counter joins them in CTA order (a fixed order, so that
// equal inputs give equal bits).
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_attn.cuh"

namespace gdn {

namespace attn {

Layout layout(int T, int N, int Hq, int Hk, int d) {
  Layout l;
  const int64_t G = Hq / Hk;
  l.split_rows = split_rows((int)G);
  l.item_cap = (int)std::min<int64_t>((int64_t)T * G / l.split_rows + N, 0x7fffffff / 16);
  l.tile_rows = tile_rows(d);
  l.tile_cap = (int)std::min<int64_t>((int64_t)T * G / l.tile_rows + N, 0x7fffffff / 16);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t at = 0;
  l.starts = at;
  at += kSplitGridMax * sizeof(Start);
  l.tile_starts = at;
  at = up(at + tile_grid() * sizeof(Start));
  l.items = at;
  at = up(at + (size_t)l.item_cap * sizeof(Item));
  l.counters = at;
  at = up(at + ((size_t)l.item_cap * Hk + 2 * kSplitGridMax) * sizeof(int));
  l.tiles = at;
  at = up(at + (size_t)l.tile_cap * sizeof(Item));
  l.partials = at;
  at = up(at + (size_t)kSplitGridMax * 2 * (size_t)l.split_rows * (d + 2) * sizeof(float));
  l.tile_partials = at;
  at = up(at + (size_t)tile_grid() * 2 * (size_t)l.tile_rows * (d + 2) * sizeof(float));
  l.total = at;
  return l;
}

}  // namespace attn

namespace {
using namespace attn;

// ---------------------------------------------------------------------------
// Plan: the row tiles of the step, in sequence order, with the running sum of
// their kv units. One CTA; a few thousand tiles at most.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t *cu, *kv;
  int N, T, G, Hk, limit;
  int64_t kv_max;
  int rows, item_cap, grid;            // split kernel
  int tile_rows, tile_cap, tile_grid;  // tensor-core kernel
  Item *items, *tiles;
  int* counters;
  Start *starts, *tile_starts;
};

__device__ __forceinline__ int block_scan(int v, int* sums, int& tot) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += a;
  }
  __syncthreads();
  if (lane == 31) sums[w] = v;
  __syncthreads();
  if (w == 0) {
    int s = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += a;
    }
    sums[lane] = s;
  }
  __syncthreads();
  tot = sums[31];
  return v + (w > 0 ? sums[w - 1] : 0);
}

// Row tiles of `rows` rows, with units of `keys` keys, of the sequences with
// more than `above` and at most `upto` rows.
struct ListArgs {
  int rows, keys, above, upto, cap;
  Item* items;
};

__device__ void build_list(const PlanArgs& p, const ListArgs& a, int* sums, int* s_first,
                           int& items, int& units) {
  const int tid = threadIdx.x;
  items = units = 0;
  for (int n0 = 0; n0 < p.N; n0 += kPlanThreads) {
    // Tiles of this thread's sequence, then one thread per tile.
    int tiles = 0;
    if (n0 + tid < p.N) {
      const Seq s = seq_of(p.cu, p.kv, n0 + tid, p.T, p.kv_max);
      const int64_t r = (int64_t)s.len * p.G;
      if (r > a.above && r <= a.upto) tiles = (int)((r + a.rows - 1) / a.rows);
    }
    int tot;
    const int inc = block_scan(tiles, sums, tot);
    s_first[tid] = inc - tiles;
    __syncthreads();
    for (int i0 = 0; i0 < tot; i0 += kPlanThreads) {
      const int i = i0 + tid;
      Item it = {0, 0, 0, 0};
      if (i < tot) {
        int lo = 0, hi = kPlanThreads - 1;    // last sequence whose first tile is <= i
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_first[mid] <= i) lo = mid; else hi = mid - 1;
        }
        it.seq = n0 + lo;
        it.row0 = (i - s_first[lo]) * a.rows;
        const Seq s = seq_of(p.cu, p.kv, it.seq, p.T, p.kv_max);
        const int last = min(s.len - 1, (it.row0 + a.rows - 1) / p.G);
        // An item without keys still has one unit, which writes its zeros.
        it.units = max(1, (visible(s, last) + a.keys - 1) / a.keys);
        if (items + i >= a.cap) it.units = 0;      // malformed offsets only
      }
      int tot_units;
      const int cum = block_scan(it.units, sums, tot_units);
      it.cum = units + cum - it.units;
      if (i < tot && items + i < a.cap) a.items[items + i] = it;
      units += tot_units;
    }
    items += tot;
    __syncthreads();
  }
  items = min(items, a.cap);
}

// Every CTA's piece of the line, of at least `least` units.
__device__ void cut_line(const PlanArgs& p, const Item* items, int num, int units, int grid, int least,
                         Start* starts) {
  const int64_t all = (int64_t)units * p.Hk;
  const int per_cta = (int)max((int64_t)least, (all + grid - 1) / grid);
  __syncthreads();                              // the list is written
  for (int c = threadIdx.x; c < grid; c += kPlanThreads) {
    Start at;
    at.u = min((long long)all, (long long)c * per_cta);
    at.u_end = min((long long)all, at.u + per_cta);
    at.item = at.head = 0;
    at.num_items = num;
    at.units = units;
    at.per_cta = per_cta;
    at.it = {0, 0, 0, 0};
    at.first = at.len = at.kv = 0;
    if (at.u < all) {
      at.head = (int)(at.u / units);
      const int x = (int)(at.u - (int64_t)at.head * units);
      int lo = 0, hi = num - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (items[mid].cum <= x) lo = mid; else hi = mid - 1;
      }
      at.item = lo;
      at.it = items[lo];
      const Seq s = seq_of(p.cu, p.kv, at.it.seq, p.T, p.kv_max);
      at.first = s.first;
      at.len = s.len;
      at.kv = s.kv;
    }
    starts[c] = at;
  }
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const PlanArgs p) {
  __shared__ int sums[32];
  __shared__ int s_first[kPlanThreads];
  pdl_wait();
  pdl_trigger();
  int items, units, tiles, tile_units;
  build_list(p, {p.rows, kUnit, 0, p.limit, p.item_cap, p.items}, sums, s_first, items, units);
  build_list(p, {p.tile_rows, kTileKeys, p.limit, 0x7fffffff, p.tile_cap, p.tiles}, sums, s_first,
             tiles, tile_units);
  for (int i = threadIdx.x; i < items * p.Hk + 2 * kSplitGridMax; i += kPlanThreads) p.counters[i] = 0;
  // A piece of the split kernel gives each of its warps a unit at least.
  cut_line(p, p.items, items, units, p.grid, 8, p.starts);
  cut_line(p, p.tiles, tiles, tile_units, p.tile_grid, 1, p.tile_starts);
}

// ---------------------------------------------------------------------------
// MMA and copy wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
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
__device__ __forceinline__ void cp_async4(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
               :: "r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------------------
// Split kernel
// ---------------------------------------------------------------------------
constexpr int kWarps = 8;
constexpr int kJoin = 16;                // partial results joined by one CTA
constexpr int kJoinMax = (kSplitGridMax + kJoin - 1) / kJoin > kJoin ? (kSplitGridMax + kJoin - 1) / kJoin : kJoin;

template <int D, int QM>
struct Cfg {
  static constexpr int rows = 8 * QM;
  static constexpr int slots = 3;                      // half units in a warp's ring
  static constexpr int slot_bytes = kUnit * D;
  static constexpr int chunks = D / 16;                // 16-byte chunks of a cache row
  static constexpr int ring = kWarps * slots * slot_bytes;
  static constexpr int q_bytes = rows * 2 * D;         // hi | lo codes of each row
  // ring | Q | Q row scales | scales of the ring's units | per-warp m, l | abort flag
  static constexpr int o_q = ring;
  static constexpr int o_qs = o_q + q_bytes;
  static constexpr int o_sc = o_qs + rows * 4;
  static constexpr int o_ml = o_sc + kWarps * slots * 2 * 4;
  static constexpr int o_flag = o_ml + kWarps * rows * 2 * 4;
  static constexpr int o_nan = o_flag + 16;            // [D]: first key whose V is NaN there
  static constexpr int total = o_nan + D * 4;
};

// Chunk swizzle of a row inside a slot: the K reads (8 lanes: 2 neighbouring
// rows x 4 chunks) and the V reads (4 rows two apart x 2 chunks) both touch all
// 32 banks once. 64-byte rows pair up in a 128-byte line, so their K reads need
// none and their V reads settle for two passes.
template <int D>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (D == 64) return chunk ^ (2 * ((row >> 1) & 1));
  return chunk ^ ((2 * ((row >> 1) & 3)) ^ (4 * (row & 1)));
}

template <int D, int QM>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 1 : 2)
attn_split_kernel(const Args p) {
  using C = Cfg<D, QM>;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* s_q = smem + C::o_q;
  float* s_qs = reinterpret_cast<float*>(smem + C::o_qs);
  float* s_ml = reinterpret_cast<float*>(smem + C::o_ml);
  int* s_flag = reinterpret_cast<int*>(smem + C::o_flag);   // [0] last to arrive, [1] a NaN in V
  int* s_nan = reinterpret_cast<int*>(smem + C::o_nan);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  unsigned char* ring = smem + w * (C::slots * C::slot_bytes);
  float* ring_sc = reinterpret_cast<float*>(smem + C::o_sc) + w * C::slots * 2;
  const int G = p.Hq / p.Hk, B = 1 << p.log_b;
  const size_t block_bytes = (size_t)B * D;

  pdl_wait();
  pdl_trigger();
  const Start start = read_start(p.starts + blockIdx.x);
  const int num_items = start.num_items, units1 = start.units, per_cta = start.per_cta;
  long long u = start.u;
  const long long u_end = start.u_end;
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
    const int halves = 2 * mine;
    // Blocks of the two 16-token halves of the next unit to be copied.
    auto block_at = [&](int unit, int half) {
      const int tok = unit * kUnit + half * 16;
      return tok < key_end ? __ldg(table + (tok >> p.log_b)) : 0;
    };
    int cur0 = 0, cur1 = 0, nxt0 = 0, nxt1 = 0;
    if (mine > 0) {
      nxt0 = block_at(first_unit + w, 0);
      nxt1 = block_at(first_unit + w, 1);
    }
    auto issue = [&](int h) {
      if (h < halves) {
        const int i = h >> 1, is_v = h & 1;
        const int unit = first_unit + w + i * kWarps;
        if (!is_v) {
          cur0 = nxt0;
          cur1 = nxt1;
          if (i + 1 < mine) {
            nxt0 = block_at(unit + kWarps, 0);
            nxt1 = block_at(unit + kWarps, 1);
          }
          if ((unsigned)cur0 >= (unsigned)p.num_blocks || (unsigned)cur1 >= (unsigned)p.num_blocks)
            record_device_status(GDN_ERR_INVALID_ARG);
        }
        const uint8_t* base = is_v ? p.vc : p.kc;
        unsigned char* slot = ring + (h % C::slots) * C::slot_bytes;
        constexpr int rows_per = 32 / C::chunks;                 // rows per warp-wide copy
        const int c = lane % C::chunks, r_in = lane / C::chunks;
#pragma unroll
        for (int k = 0; k < kUnit / rows_per; ++k) {
          const int r = k * rows_per + r_in;
          const int tok = unit * kUnit + r;
          const int blk = r < 16 ? cur0 : cur1;
          const bool ok = tok < key_end && (unsigned)blk < (unsigned)p.num_blocks;
          const uint8_t* src = base;
          if (ok) src += ((size_t)blk * p.Hk + head) * block_bytes + (size_t)(tok & (B - 1)) * D + c * 16;
          tc::cp_async16(slot + r * D + swz<D>(r, c) * 16, src, ok ? 16u : 0u);
        }
        if (lane < 2) {
          const int blk = lane ? cur1 : cur0;
          const bool ok = unit * kUnit + lane * 16 < key_end && (unsigned)blk < (unsigned)p.num_blocks;
          const float* sc = is_v ? p.vs : p.ks;
          cp_async4(ring_sc + (h % C::slots) * 2 + lane, ok ? sc + (size_t)blk * p.Hk + head : sc,
                    ok ? 4u : 0u);
        }
      }
      tc::cp_async_commit();
    };
#pragma unroll
    for (int h = 0; h < C::slots - 1; ++h) issue(h);

    for (int i = tid; i < D; i += kWarps * 32) s_nan[i] = 0x7fffffff;
    if (tid == 0) s_flag[1] = 0;

    // ---- Q of the tile: hi and lo codes, one power-of-two scale per row -------
    for (int r = w; r < C::rows; r += kWarps) {
      constexpr int per = D / 32;
      float v[per];
      float top = 0.f;
      bool bad = false;
      if (r < n_rows) {
        const int row = row0 + r, tok = s.first + row / G, hq = head * G + row % G;
        const __nv_bfloat16* src = p.q + (int64_t)tok * p.q_stride + (int64_t)hq * D + lane * per;
#pragma unroll
        for (int i = 0; i < per; i += 2) {
          const uint32_t two = __ldg(reinterpret_cast<const uint32_t*>(src + i));
          v[i] = bf16lo(two);
          v[i + 1] = bf16hi(two);
        }
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) v[i] = 0.f;
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
        *reinterpret_cast<uint16_t*>(s_q + r * 2 * D + lane * per + i) = (uint16_t)h2;
        *reinterpret_cast<uint16_t*>(s_q + r * 2 * D + D + lane * per + i) = (uint16_t)l2;
      }
      // A row with an infinity or NaN has no finite softmax: its scores are NaN.
      if (lane == 0)
        s_qs[r] = bad ? __int_as_float(0x7fffffff) : __int_as_float((ex + 127) << 23);
    }
    __syncthreads();

    // ---- Q fragments: k index (t4, i) of step s <-> the K chunk layout below ---
    uint32_t qf[QM][D / 32][4];
    float rs[QM];
    int lim[QM];
    int min_lim = 0x7fffffff;
#pragma unroll
    for (int m = 0; m < QM; ++m) {
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const unsigned char* at = s_q + (m * 8 + g) * 2 * D + 16 * (t4 + 4 * (k >> 1)) + 8 * (k & 1);
        const uint2 h2 = *reinterpret_cast<const uint2*>(at);
        const uint2 l2 = *reinterpret_cast<const uint2*>(at + D);
        qf[m][k][0] = h2.x;
        qf[m][k][1] = l2.x;
        qf[m][k][2] = h2.y;
        qf[m][k][3] = l2.y;
      }
      rs[m] = s_qs[m * 8 + g] * p.scale_log2;
      const int r = m * 8 + g;
      lim[m] = r < n_rows ? visible(s, (row0 + r) / G) : 0;
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

    for (int i = 0; i < mine; ++i) {
      const int unit = first_unit + w + i * kWarps;
      // K of unit i has landed; its slot's predecessor is free again.
      tc::cp_async_wait_group<C::slots - 2>();
      __syncwarp();
      issue(2 * i + C::slots - 1);
      float sc[QM][4][2];
      float ksc[2];
      {
        const int sl = (2 * i) % C::slots;
        const unsigned char* slot = ring + sl * C::slot_bytes;
        ksc[0] = ring_sc[sl * 2];
        ksc[1] = ring_sc[sl * 2 + 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float c4[QM][4];
#pragma unroll
          for (int m = 0; m < QM; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) c4[m][c] = 0.f;
          const int r = 8 * j + g;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 kk = *reinterpret_cast<const uint4*>(slot + r * D + swz<D>(r, t4 + 4 * c) * 16);
#pragma unroll
            for (int m = 0; m < QM; ++m) {
              mma_e4m3(c4[m], qf[m][2 * c][0], qf[m][2 * c][1], qf[m][2 * c][2], qf[m][2 * c][3],
                       kk.x, kk.y);
              mma_e4m3(c4[m], qf[m][2 * c + 1][0], qf[m][2 * c + 1][1], qf[m][2 * c + 1][2],
                       qf[m][2 * c + 1][3], kk.z, kk.w);
            }
          }
#pragma unroll
          for (int m = 0; m < QM; ++m) {
            sc[m][j][0] = c4[m][0] + c4[m][2];
            sc[m][j][1] = c4[m][1] + c4[m][3];
          }
        }
      }
      // V of unit i has landed.
      tc::cp_async_wait_group<C::slots - 2>();
      __syncwarp();
      issue(2 * i + C::slots);
      const int sl = (2 * i + 1) % C::slots;
      const unsigned char* slot = ring + sl * C::slot_bytes;
      float lvs[2], ivs[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float vsc = fmaxf(ring_sc[sl * 2 + k], 7.888609052210118e-31f);   // 2^-100
        lvs[k] = lg2_approx(vsc);
        ivs[k] = __fdividef(1.f, vsc);
      }
      const bool cut = unit * kUnit + kUnit > min_lim;
      // Where the rows of the tile do not see the same keys, a weight of zero
      // must not meet a NaN (0 x NaN is NaN): a NaN of V is taken out of the
      // slot and kept as the first key whose column has one.
      if (cut && min_lim < key_end) {
        unsigned char* vs_ = ring + sl * C::slot_bytes;
        for (int k = lane; k < C::slot_bytes / 4; k += 32) {
          const uint32_t word = *reinterpret_cast<const uint32_t*>(vs_ + 4 * k);
          if ((((word & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0) {
            const int r = 4 * k / D, at = 4 * k % D;
            const int col = swz<D>(r, at / 16) * 16 + at % 16;      // the swizzle is its own inverse
            uint32_t clean = word;
            for (int c = 0; c < 4; ++c) {
              if (((word >> (8 * c)) & 0x7fu) == 0x7fu) {
                atomicMin(s_nan + col + c, unit * kUnit + r);
                clean &= ~(0xffu << (8 * c));
              }
            }
            *reinterpret_cast<uint32_t*>(vs_ + 4 * k) = clean;
            s_flag[1] = 1;
          }
        }
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
            if (cut && unit * kUnit + 8 * j + 2 * t4 + e >= lim[m]) xx = -INFINITY;
            sc[m][j][e] = xx;
            mx = fmaxf(mx, xx);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (__any_sync(0xffffffffu, mx > m_run[m] + 8.f)) {
          const float m_new = fmaxf(mx, m_run[m]);
          const float al = m_new > m_run[m] ? ex2_approx(m_run[m] - m_new) : 1.f;
          m_run[m] = m_new;
          l_run[m] *= al;
          const float a0 = __shfl_sync(0xffffffffu, al, 8 * t4);
          const float a1 = __shfl_sync(0xffffffffu, al, 8 * t4 + 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            acc[m][k][0] *= a0;
            acc[m][k][1] *= a1;
            acc[m][k][2] *= a0;
            acc[m][k][3] *= a1;
          }
        }
        const float ref = (m_run[m] == -INFINITY ? 0.f : m_run[m]) - 7.f;
        float lsum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p0 = ex2_approx(sc[m][j][0] - ref), p1 = ex2_approx(sc[m][j][1] - ref);
          lsum = fmaf(p0 + p1, ivs[j >> 1], lsum);
          pf[m][j] = pack_half2(p0, p1);
        }
        l_run[m] += lsum;
      }
      // O^T += V^T P^T: lane (g, t4) holds d = 16 chunk + byte, 16 chunk(g): the
      // two rows of m-tile b are bytes 2b and 2b + 1 of the lane's own chunk.
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int r0 = 16 * ks + 2 * t4;
        if constexpr (D == 64) {
          uint2 va[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r0 + (k & 1) + 8 * (k >> 1);
            va[k] = *reinterpret_cast<const uint2*>(slot + r * D + swz<D>(r, g >> 1) * 16 + (g & 1) * 8);
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
              const int r = r0 + (k & 1) + 8 * (k >> 1);
              va[k] = *reinterpret_cast<const uint4*>(slot + r * D + swz<D>(r, g + 8 * cc) * 16);
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
    tc::cp_async_wait_group<0>();

    // ---- join the warps ------------------------------------------------------
#pragma unroll
    for (int m = 0; m < QM; ++m) {
      l_run[m] += __shfl_xor_sync(0xffffffffu, l_run[m], 1);
      l_run[m] += __shfl_xor_sync(0xffffffffu, l_run[m], 2);
      if (t4 == 0) {
        s_ml[(w * C::rows + m * 8 + g) * 2] = m_run[m];
        s_ml[(w * C::rows + m * 8 + g) * 2 + 1] = l_run[m];
      }
    }
    __syncthreads();                     // also: every warp is done with its ring
    // Warp w leaves its rows of O, on the common maximum, in its ring:
    // float32 [rows][D], 16-byte chunks XOR-ed by the row.
    float* s_o = reinterpret_cast<float*>(smem);
    static_assert(kWarps * C::rows * D * 4 <= C::ring, "the warps' O fits the rings");
    constexpr int n_el = C::rows * D / (kWarps * 32);
#pragma unroll
    for (int m = 0; m < QM; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = m * 8 + 2 * t4 + e;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_ml[(k * C::rows + r) * 2]);
        const float mw = s_ml[(w * C::rows + r) * 2];
        // A warp without keys has f = 0; its accumulator is zero as well.
        const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - top);
        float* dst = s_o + (w * C::rows + r) * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // m-tile k: d of its rows g and g + 8.
          int d0;
          if constexpr (D == 64) d0 = g * 8 + 2 * k;
          else d0 = 128 * (k >> 3) + g * 16 + 2 * (k & 7);
          *reinterpret_cast<float2*>(dst + (d0 ^ (8 * (r & 3)))) =
              make_float2(acc[m][k][e] * f, acc[m][k][2 + e] * f);
        }
      }
    }
    __syncthreads();
    float sum_o[n_el];
#pragma unroll
    for (int i = 0; i < n_el; ++i) {
      const int at = i * kWarps * 32 + tid, r = at / D, dd = at % D;
      sum_o[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) sum_o[i] += s_o[(k * C::rows + r) * D + (dd ^ (8 * (r & 3)))];
      if (s_flag[1] && r < n_rows && visible(s, (row0 + r) / G) > s_nan[dd]) sum_o[i] = NAN;
    }
    // Row r's joined maximum and sum (each thread for the rows that it holds).
    const bool whole = seg == n_units;
    float* part = nullptr;
    if (!whole)
      part = p.partials + ((size_t)blockIdx.x * 2 + (first_unit == 0 ? 1 : 0)) * C::rows * (D + 2);
#pragma unroll
    for (int i = 0; i < n_el; ++i) {
      const int at = i * kWarps * 32 + tid, r = at / D, dd = at % D;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_ml[(k * C::rows + r) * 2]);
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float mw = s_ml[(k * C::rows + r) * 2];
        // NaN sums pass on: a NaN row keeps m = -inf, so its l is added as it is.
        const float lw = s_ml[(k * C::rows + r) * 2 + 1];
        l += mw == -INFINITY ? lw : lw * ex2_approx(mw - top);
      }
      if (whole) {
        if (r < n_rows) {
          const int row = row0 + r;
          const float o = l == 0.f ? 0.f : sum_o[i] / l;
          p.o[((int64_t)(s.first + row / G) * p.Hq + head * G + row % G) * D + dd] = __float2bfloat16_rn(o);
        }
      } else {
        __stcg(part + 2 * C::rows + r * D + dd, sum_o[i]);
        if (dd == 0) {
          __stcg(part + r * 2, top);
          __stcg(part + r * 2 + 1, l);
        }
      }
    }
    if (!whole) {
      // The item's CTAs are those of its first and last unit and all between, in
      // groups of kJoin: the last of a group joins it in place of its first
      // member's partial, the last group's joins the groups.
      const long long at0 = (long long)head * units1 + cum;
      const int c0 = (int)(at0 / per_cta), c1 = (int)((at0 + n_units - 1) / per_cta);
      const int grp = ((int)blockIdx.x - c0) / kJoin, groups = (c1 - c0) / kJoin + 1;
      const int ga = c0 + grp * kJoin, gb = min(c1, ga + kJoin - 1);
      const size_t psz = C::rows * (D + 2);
      float* fs = reinterpret_cast<float*>(smem);             // factors, [n][rows]
      float* s_l = fs + kJoinMax * C::rows;
      auto slot = [&](int c) { return p.partials + ((size_t)c * 2 + (c == c0)) * psz; };
      // Joins the partials of CTAs a, a + step, ... (n of them); `out` or the output.
      auto join = [&](int a, int step, int n, float* out) {
        for (int r = w; r < C::rows; r += kWarps) {
          float top = -INFINITY, l = 0.f;
          for (int c = lane; c < n; c += 32) top = fmaxf(top, __ldcg(slot(a + c * step) + r * 2));
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
          for (int c = lane; c < n; c += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot(a + c * step)) + r);
            // NaN sums pass on: a NaN row has m = -inf and its l as it is.
            const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
            fs[c * C::rows + r] = f;
            l += ml.y * f;
          }
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
          if (lane == 0) {
            s_l[r * 2] = top;
            s_l[r * 2 + 1] = l;
          }
        }
        __syncthreads();
#pragma unroll 1
        for (int e = tid * 4; e < C::rows * D; e += kWarps * 32 * 4) {
          const int r = e / D, dd = e % D;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int c = 0; c < n; ++c) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(a + c * step) + 2 * C::rows + e));
            const float f = fs[c * C::rows + r];
            o.x = fmaf(v.x, f, o.x);
            o.y = fmaf(v.y, f, o.y);
            o.z = fmaf(v.z, f, o.z);
            o.w = fmaf(v.w, f, o.w);
          }
          if (out) {
            __stcg(reinterpret_cast<float4*>(out + 2 * C::rows + e), o);
          } else if (r < n_rows) {
            const int row = row0 + r;
            const float l = s_l[r * 2 + 1], il = l == 0.f ? 0.f : 1.f / l;
            uint2 b;
            b.x = pack_bf16x2(o.x * il, o.y * il);
            b.y = pack_bf16x2(o.z * il, o.w * il);
            *reinterpret_cast<uint2*>(p.o + ((int64_t)(s.first + row / G) * p.Hq + head * G + row % G) * D + dd) = b;
          }
        }
        if (out && tid < C::rows)
          __stcg(reinterpret_cast<float2*>(out) + tid, make_float2(s_l[tid * 2], s_l[tid * 2 + 1]));
      };
      // One more arrival of `of` at the counter; true for the whole CTA at the last.
      auto last = [&](int* counter, int of) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int seen = atomicAdd(counter, 1);
          s_flag[0] = seen == of - 1;
          if (seen == of - 1) *counter = 0;        // ready for the next call on this plan
        }
        __syncthreads();
        if (s_flag[0]) __threadfence();
        return s_flag[0] != 0;
      };
      int* item_counter = p.counters + 2 * kSplitGridMax + (size_t)lo * p.Hk + head;
      if (groups == 1) {
        if (last(item_counter, gb - ga + 1)) join(ga, 1, gb - ga + 1, nullptr);
      } else if (last(p.counters + ga * 2 + (ga == c0), gb - ga + 1)) {
        join(ga, 1, gb - ga + 1, slot(ga));
        if (last(item_counter, groups)) join(c0, kJoin, groups, nullptr);
      }
    }
    __syncthreads();                     // the ring, Q and s_ml are free again
    u += seg;
    if (first_unit + seg == n_units && ++lo == num_items) {
      lo = 0;
      ++head;
    }
    if (u < u_end) {
      const int4 raw = __ldg(reinterpret_cast<const int4*>(p.items) + lo);
      it = {raw.x, raw.y, raw.z, raw.w};
      s = seq_of(p.cu, p.kv, it.seq, p.T, (int64_t)p.max_blocks << p.log_b);
    }
  }
}

template <int D, int QM>
gdn_status_t launch_split(const Args& a, cudaStream_t st) {
  static const cudaError_t set = cudaFuncSetAttribute(
      attn_split_kernel<D, QM>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, QM>::total);
  if (set != cudaSuccess) return check_launch(set);
  return check_launch(launch_pdl(attn_split_kernel<D, QM>, dim3(a.split_grid), dim3(kWarps * 32),
                                 Cfg<D, QM>::total, st, a));
}

}  // namespace

gdn_status_t launch_attn_plan(const int32_t* cu, const int32_t* kv, int N, int T, int Hq, int Hk,
                              int d, int64_t kv_max, void* workspace, cudaStream_t st) {
  const Layout l = layout(T, N, Hq, Hk, d);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  PlanArgs p;
  p.cu = cu;
  p.kv = kv;
  p.N = N;
  p.T = T;
  p.G = Hq / Hk;
  p.Hk = Hk;
  p.rows = l.split_rows;
  p.item_cap = l.item_cap;
  p.grid = split_grid(d);
  p.kv_max = kv_max;
  p.items = reinterpret_cast<Item*>(ws + l.items);
  p.counters = reinterpret_cast<int*>(ws + l.counters);
  p.limit = split_limit(p.G);
  p.tile_rows = l.tile_rows;
  p.tile_cap = l.tile_cap;
  p.tile_grid = tile_grid();
  p.tiles = reinterpret_cast<Item*>(ws + l.tiles);
  p.starts = reinterpret_cast<Start*>(ws + l.starts);
  p.tile_starts = reinterpret_cast<Start*>(ws + l.tile_starts);
  return check_launch(launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p));
}

gdn_status_t launch_attn_split(const Args& a, cudaStream_t st) {
  const bool two = a.split_rows == 16;
  if (a.d == 64) return two ? launch_split<64, 2>(a, st) : launch_split<64, 1>(a, st);
  if (a.d == 128) return two ? launch_split<128, 2>(a, st) : launch_split<128, 1>(a, st);
  return two ? launch_split<256, 2>(a, st) : launch_split<256, 1>(a, st);
}

GDN_DEFINE_STATUS_GATHER(gather_status_attn_split)

}  // namespace gdn
