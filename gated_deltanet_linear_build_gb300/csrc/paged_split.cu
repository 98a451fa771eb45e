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
//   weight is 2^-29 of the largest one's still keeps its digits.
// * The block's V scale enters the exponent: P' = 2^(s + log2 vs - m), and the
//   sum takes P' / vs. Blocks of any scale then share one accumulator, and the
//   largest contribution, not the largest weight, sets the range.
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
// 233 us, 6.1 TB/s, 90% of the copy rate. 16 rows a tile (12 heads a kv head) have
// twice the instructions a byte and half of the warps: 66%. 32 requests of 100 to
// 1,900 tokens, 28 MB: 15.7 us, of which 9 are there for a single short request.
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
  l.self_starts = at;
  at += kSplitGridMax * sizeof(Start);
  l.tile_starts = at;
  at = up(at + tile_grid() * sizeof(Start));
  l.items = at;
  at = up(at + (size_t)l.item_cap * sizeof(Item));
  l.tiles = at;
  at = up(at + (size_t)l.tile_cap * sizeof(Item));
  l.sorted_tiles = at;
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
// their kv units, and the pieces that the line of units is cut into. One CTA a
// list: latency bounds it (two rounds of dependent loads and a scan each).
// ---------------------------------------------------------------------------

// What an item costs beside its units, in units: a segment's start and end. (Split
// kernel, 0 / 8 / 16 / 32: 256 decode requests of up to 1,000 tokens 77 / 69 / 66
// / 68 us, 400 of up to 2,000 at d = 256 95 / 84 / 81 / 85 us. Tensor-core kernel,
// 5 / 8 / 12: 4,096 tokens behind 4,000, d = 256, 294 / 288 / 286 us.)
constexpr int kSplitOver = 16, kItemCost = 10;

struct ListArgs {
  int rows, keys, above, upto, cap, grid;          // tiles of the sequences with above < rows <= upto
  int least, over;                                 // units of a piece; of an item's overhead (Cut)
  Item *items, *sorted;                            // sorted: room for the items by length, or null
  Start* starts;
};
struct PlanArgs {
  const int32_t *cu, *kv;
  int N, T, G, Hk;
  int64_t kv_max;
  ListArgs list[2];                    // of the kernels that the step launches
};

// A list's first kPlanThreads items stay here: the plan's steps follow one another
// through global memory at 0.4 us each otherwise (2,048 tokens in 4 prompts: 7.9
// us).
template <int kPlanThreads>
struct PlanShared {
  int2 sums[32];
  int first[kPlanThreads];
  Item items[kPlanThreads], sorted[kPlanThreads];
};
template <int kPlanThreads>
__device__ __forceinline__ Item item_at(const PlanShared<kPlanThreads>& sh, const ListArgs& a, int i) {
  return i < kPlanThreads ? sh.items[i] : a.items[i];
}
template <int kPlanThreads>
__device__ __forceinline__ Item sorted_at(const PlanShared<kPlanThreads>& sh, const ListArgs& a, int i) {
  return i < kPlanThreads ? sh.sorted[i] : a.sorted[i];
}

// Inclusive scan of a pair over the block; the total in tot.
template <int kPlanThreads>
__device__ __forceinline__ int2 block_scan(int2 v, int2* sums, int2& tot) {
  constexpr int kLast = kPlanThreads / 32 - 1;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v.x, d), b = __shfl_up_sync(0xffffffffu, v.y, d);
    if (lane >= d) { v.x += a; v.y += b; }
  }
  __syncthreads();                     // earlier readers of sums are done
  if (lane == 31) sums[w] = v;
  __syncthreads();
  // Every warp scans the warps' sums itself.
  int2 s = lane <= kLast ? sums[lane] : make_int2(0, 0);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, s.y, d);
    if (lane >= d) { s.x += a; s.y += b; }
  }
  tot.x = __shfl_sync(0xffffffffu, s.x, kLast);
  tot.y = __shfl_sync(0xffffffffu, s.y, kLast);
  const int bx = __shfl_sync(0xffffffffu, s.x, (w + 31) & 31), by = __shfl_sync(0xffffffffu, s.y, (w + 31) & 31);
  if (w > 0) { v.x += bx; v.y += by; }
  return v;
}

__device__ __forceinline__ Item item_of(const PlanArgs& p, const ListArgs& a, const Seq& s, int seq,
                                        int tile) {
  Item it = {seq, tile * a.rows, 0, 0};
  const int last = min(s.len - 1, (it.row0 + a.rows - 1) / p.G);
  // An item without keys still has one unit, which writes its zeros.
  it.units = max(1, (visible(s, last) + a.keys - 1) / a.keys);
  return it;
}

template <int kPlanThreads>
__device__ void build_list(const PlanArgs& p, const ListArgs& a, PlanShared<kPlanThreads>& sh, int& items, int& units) {
  const int tid = threadIdx.x;
  int2* sums = sh.sums;
  int* s_first = sh.first;
  items = units = 0;
  for (int n0 = 0; n0 < p.N; n0 += kPlanThreads) {
    int tiles = 0;
    Seq s = {0, 0, 0};
    if (n0 + tid < p.N) {
      s = seq_of(p.cu, p.kv, n0 + tid, p.T, p.kv_max);
      const int64_t r = (int64_t)s.len * p.G;
      if (r > a.above && r <= a.upto) tiles = (int)((r + a.rows - 1) / a.rows);
    }
    if (!__syncthreads_or(tiles > 1)) {
      // One tile a sequence: one scan gives its place and its units.
      Item it = {0, 0, 0, 0};
      if (tiles) it = item_of(p, a, s, n0 + tid, 0);
      int2 tot;
      const int2 inc = block_scan<kPlanThreads>(make_int2(tiles, it.units), sums, tot);
      it.cum = units + inc.y - it.units;
      const int at = items + inc.x - 1;
      if (tiles && at < a.cap) {
        a.items[at] = it;
        if (at < kPlanThreads) sh.items[at] = it;
      }
      items += tot.x;
      units += tot.y;
      continue;
    }
    int2 tot;
    const int2 inc = block_scan<kPlanThreads>(make_int2(tiles, 0), sums, tot);
    s_first[tid] = inc.x - tiles;
    __syncthreads();
    for (int i0 = 0; i0 < tot.x; i0 += kPlanThreads) {
      const int i = i0 + tid;
      Item it = {0, 0, 0, 0};
      if (i < tot.x && items + i < a.cap) {    // beyond: malformed offsets only
        int lo = 0, hi = kPlanThreads - 1;     // last sequence whose first tile is <= i
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_first[mid] <= i) lo = mid; else hi = mid - 1;
        }
        it = item_of(p, a, seq_of(p.cu, p.kv, n0 + lo, p.T, p.kv_max), n0 + lo, i - s_first[lo]);
      }
      int2 tot_units;
      const int2 cum = block_scan<kPlanThreads>(make_int2(0, it.units), sums, tot_units);
      it.cum = units + cum.y - it.units;
      if (i < tot.x && items + i < a.cap) {
        a.items[items + i] = it;
        if (items + i < kPlanThreads) sh.items[items + i] = it;
      }
      units += tot_units.y;
    }
    items += tot.x;
    __syncthreads();                           // s_first is free again
  }
  items = min(items, a.cap);
}

// The line is cut in one of two ways. Into pieces of equal cost, which may end
// inside an item and go on with the next: no SM is idle. An item costs its units
// and `over` more (a segment's start and end). Or, where items are no more than
// half as many as CTAs, each item by itself into pieces of about `target` units:
// a piece then is one segment (a CTA with two held up a step of one 16,000-token
// request by 4 of 10 us). With target >= all / (grid - items) the pieces are no
// more than the CTAs.
struct Cut {
  int per_cta, target;                 // target 0: pieces of equal cost
};
__device__ __forceinline__ Cut cut_of(long long all, long long items, int grid, int least, int over) {
  Cut c;
  c.per_cta = (int)max((long long)least, (all + items * over + grid - 1) / grid);
  c.target = 0;
  if (2 * items <= grid) c.target = (int)max((long long)least, (all + grid - items - 1) / (grid - items));
  return c;
}
// Piece k of the n that an item of `units` units is cut into.
__device__ __forceinline__ void piece_of(Start& at, int c, int k, int n) {
  const int from = (int)((long long)at.it.units * k / n), to = (int)((long long)at.it.units * (k + 1) / n);
  at.u = (long long)at.head * at.units + at.it.cum + from;
  at.count = to - from;
  at.c0 = c - k;
  at.pieces = n;
}
// Largest i < num with cum(i) <= x.
template <typename F>
__device__ __forceinline__ int find_item(int num, long long x, F cum) {
  int lo = 0, hi = num - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// CTA c's piece of equal cost: at.u, at.count and, if that is not 0, at.item and
// at.head. cost(i) and units(i): of one head's items before item i; cost_all: of
// one head. The first unit of item i is at cost(i) + over.
template <typename FC, typename FU>
__device__ __forceinline__ bool piece_of_line(Start& at, int c, int Hk, long long cost_all, int per_cta, int over,
                                              FC cost, FU units) {
  auto unit_at = [&](long long x, int& item, int& head) {
    head = Hk;
    item = 0;
    if (x >= cost_all * Hk) return (long long)at.units * Hk;
    head = (int)((unsigned long long)x / (unsigned long long)cost_all);
    const long long y = x - head * cost_all;
    item = find_item(at.num_items, y, cost);
    return (long long)head * at.units + units(item) + (int)max(0ll, (long long)(y - cost(item) - over));
  };
  int item, head;
  at.u = unit_at((long long)c * per_cta, at.item, at.head);
  at.count = (int)(unit_at((long long)(c + 1) * per_cta, item, head) - at.u);
  return at.count > 0;
}
// The pieces of its item, which takes cost_before of the line before it.
__device__ __forceinline__ void pieces_of_line(Start& at, long long cost_before, int per_cta, int over) {
  const long long first = cost_before + over;
  at.c0 = (int)(first / per_cta);
  at.pieces = (int)((first + at.it.units - 1) / per_cta) - at.c0 + 1;
}

// Every CTA's piece of the list's line.
template <int kPlanThreads>
__device__ void cut_line(const PlanArgs& p, const ListArgs& a, PlanShared<kPlanThreads>& sh, int num, int units) {
  int2* sums = sh.sums;
  int* s_pieces = sh.first;
  const long long all = (long long)units * p.Hk;
  const Cut cut = cut_of(all, (long long)num * p.Hk, a.grid, a.least, a.over);
  const long long cost_all = units + (long long)num * a.over;   // of one head
  __syncthreads();                              // the list is written
  int pieces = 0;                               // of one head
  if (cut.target) {
    const int n = threadIdx.x < num ? (sh.items[threadIdx.x].units + cut.target - 1) / cut.target : 0;
    int2 tot;
    const int2 inc = block_scan<kPlanThreads>(make_int2(n, 0), sums, tot);
    s_pieces[threadIdx.x] = inc.x - n;
    pieces = tot.x;
    __syncthreads();
  }
  for (int c = threadIdx.x; c < a.grid; c += kPlanThreads) {
    Start at;
    at.u = all;
    at.item = at.head = at.count = at.pieces = at.first = at.len = at.kv = at.c0 = 0;
    at.num_items = num;
    at.units = units;
    at.it = {0, 0, 0, 0};
    int y = 0;
    bool work;
    if (cut.target) {
      work = pieces > 0 && c < pieces * p.Hk;
      if (work) {
        at.head = c / pieces;
        y = c - at.head * pieces;
        at.item = find_item(num, y, [&](int i) { return s_pieces[i]; });
      }
    } else {
      auto before = [&](int i) { return item_at(sh, a, i).cum; };
      work = piece_of_line(at, c, p.Hk, cost_all, cut.per_cta, a.over,
                           [&](int i) { return before(i) + (long long)i * a.over; }, before);
    }
    if (work) {
      at.it = item_at(sh, a, at.item);
      const Seq s = seq_of(p.cu, p.kv, at.it.seq, p.T, p.kv_max);
      at.first = s.first;
      at.len = s.len;
      at.kv = s.kv;
      if (cut.target) {
        const int k = y - s_pieces[at.item];
        piece_of(at, c, k, (at.it.units + cut.target - 1) / cut.target);
      } else {
        pieces_of_line(at, (long long)at.head * cost_all + at.it.cum + (long long)at.item * a.over, cut.per_cta, a.over);
      }
    }
    a.starts[c] = at;
  }
}

// Whole items, longest first, dealt out back and forth over the CTAs: without
// cuts there are no partial results to write and join. Taken where the most
// loaded CTA then ends before an even cut of the line would, with kCutCost for the
// partial results and their join (4: 8 prompts of 100-500 tokens behind up to
// 3,000 take 104 us instead of 97).
constexpr int kCutCost = 16, kMaxRounds = 12;
template <int kPlanThreads>
__device__ bool deal_items(const PlanArgs& p, const ListArgs& a, PlanShared<kPlanThreads>& sh, int num, int units) {
  int2* sums = sh.sums;
  int* s_hist = sh.first;
  const int tid = threadIdx.x;
  const int64_t total = (int64_t)num * p.Hk;
  // Counting sort by length, in kPlanThreads classes up to the longest.
  __syncthreads();                              // the list is written
  int longest = 1;
  for (int i = tid; i < num; i += kPlanThreads) longest = max(longest, item_at(sh, a, i).units);
  s_hist[tid] = 0;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, k));
  if ((tid & 31) == 0) sums[tid >> 5].x = longest;
  __syncthreads();
  longest = sums[tid & (kPlanThreads / 32 - 1)].x;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, k));
  const float per = (kPlanThreads - 1) / (float)longest;
  auto cls = [&](int u) { return min((int)((longest - u) * per), kPlanThreads - 1); };
  for (int i = tid; i < num; i += kPlanThreads) atomicAdd(s_hist + cls(item_at(sh, a, i).units), 1);
  __syncthreads();
  const int mine = s_hist[tid];
  int2 tot;
  const int2 inc = block_scan<kPlanThreads>(make_int2(mine, 0), sums, tot);
  s_hist[tid] = inc.x - mine;
  __syncthreads();
  for (int i = tid; i < num; i += kPlanThreads) {
    const Item it = item_at(sh, a, i);
    const int at = atomicAdd(s_hist + cls(it.units), 1);
    a.sorted[at] = it;
    if (at < kPlanThreads) sh.sorted[at] = it;
  }
  __syncthreads();
  if (total > (int64_t)kMaxRounds * a.grid) return true;        // many: any deal is even
  int load = 0;
  static_assert(kPlanThreads >= 160, "a thread per CTA");
  if (tid < a.grid)
    for (int k = 0; k < kMaxRounds; ++k) {
      const int at = k * a.grid + ((k & 1) ? a.grid - 1 - tid : tid);
      if (at >= total) break;
      load += sorted_at(sh, a, at / p.Hk).units + kItemCost;
    }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) load = max(load, __shfl_xor_sync(0xffffffffu, load, k));
  if ((tid & 31) == 0) sums[tid >> 5].y = load;
  __syncthreads();
  load = sums[tid & (kPlanThreads / 32 - 1)].y;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) load = max(load, __shfl_xor_sync(0xffffffffu, load, k));
  const int64_t even = ((int64_t)units * p.Hk + kItemCost * total) / a.grid + kItemCost + kCutCost;
  return load <= even;
}

template <int kPlanThreads>
__device__ void deal_starts(const PlanArgs& p, const ListArgs& a, const PlanShared<kPlanThreads>& sh, int num) {
  const int64_t total = (int64_t)num * p.Hk;
  for (int c = threadIdx.x; c < a.grid; c += kPlanThreads) {
    Start at;
    at.num_items = num;
    at.units = at.pieces = 0;
    at.u = 0;
    at.c0 = -1;
    // Rounds in which this CTA has an item.
    const int64_t full = total / a.grid;
    const int rest = (int)(total - full * a.grid);
    at.count = (int)full + (((full & 1) ? a.grid - 1 - c : c) < rest ? 1 : 0);
    at.it = {0, 0, 0, 0};
    at.item = at.head = at.first = at.len = at.kv = 0;
    if (at.count > 0) {
      at.item = c / p.Hk;
      at.head = c - at.item * p.Hk;
      at.it = sorted_at(sh, a, at.item);
      const Seq s = seq_of(p.cu, p.kv, at.it.seq, p.T, p.kv_max);
      at.first = s.first;
      at.len = s.len;
      at.kv = s.kv;
    }
    a.starts[c] = at;
  }
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const PlanArgs p) {
  __shared__ PlanShared<kPlanThreads> sh;
  pdl_wait();
  pdl_trigger();
  const ListArgs& a = p.list[blockIdx.x];
  int items, units;
  build_list(p, a, sh, items, units);
  if (a.sorted && deal_items(p, a, sh, items, units)) deal_starts(p, a, sh, items);
  else cut_line(p, a, sh, items, units);
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
// ---------------------------------------------------------------------------
// Split kernel
// ---------------------------------------------------------------------------
constexpr int kWarps = 8;

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
    const Cut cut = cut_of(all, (long long)total.y * p.Hk, gridDim.x, kWarps, kSplitOver);
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

    for (int i = 0; i < mine && !dead; ++i) {
      const int unit = first_unit + w + i * kWarps;
      // The unit's scales, before those of the next one replace them.
      float ksc[2], lvs[2], ivs[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ksc[k] = __shfl_sync(0xffffffffu, sc_q[0], k);
        const float v = fmaxf(__shfl_sync(0xffffffffu, sc_q[0], 2 + k), 7.888609052210118e-31f);   // 2^-100
        lvs[k] = lg2_approx(v);
        ivs[k] = __fdividef(1.f, v);
      }
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
        l += ml.y * f;
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

gdn_status_t launch_attn_plan(const int32_t* cu, const int32_t* kv, int N, int T, int Hq, int Hk,
                              int d, int64_t kv_max, int max_new_tokens, void* workspace,
                              cudaStream_t st) {
  const Layout l = layout(T, N, Hq, Hk, d);
  const int G = Hq / Hk;
  const Kernels use = kernels_of(N, T, G, Hk, max_new_tokens, kv_max);
  const int limit = use.limit;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  PlanArgs p;
  p.cu = cu;
  p.kv = kv;
  p.N = N;
  p.T = T;
  p.G = G;
  p.Hk = Hk;
  p.kv_max = kv_max;
  int lists = 0;
  // A piece of the split kernel gives each of its 8 warps a unit at least.
  if (use.split)
    p.list[lists++] = {l.split_rows, kUnit, 0, limit, l.item_cap, split_grid(d, l.split_rows), kWarps,
                       kSplitOver,                        reinterpret_cast<Item*>(ws + l.items), nullptr, reinterpret_cast<Start*>(ws + l.starts)};
  if (use.tile)
    p.list[lists++] = {l.tile_rows, kTileKeys, limit, 0x7fffffff, l.tile_cap, tile_grid(), 1,
                       kItemCost,                        reinterpret_cast<Item*>(ws + l.tiles), reinterpret_cast<Item*>(ws + l.sorted_tiles),
                       reinterpret_cast<Start*>(ws + l.tile_starts)};
  // A warp more is a turn more for every instruction of the others: 256 threads
  // where they hold the sequences and the items (4 prompts: 6.1 -> 4.7 us).
  const int64_t rows = (int64_t)T * G;
  const bool small = N <= 256 && (!use.split || rows / l.split_rows + N <= 256) &&
                     (!use.tile || rows / l.tile_rows + N <= 256);
  return check_launch(small ? launch_pdl(attn_plan_kernel<256>, dim3(lists), dim3(256), 0, st, p)
                            : launch_pdl(attn_plan_kernel<1024>, dim3(lists), dim3(1024), 0, st, p));
}

gdn_status_t launch_attn_split(const Args& a, cudaStream_t st) {
  const bool two = a.split_rows == 16;
  if (a.d == 64) return two ? launch_split<64, 2>(a, st) : launch_split<64, 1>(a, st);
  if (a.d == 128) return two ? launch_split<128, 2>(a, st) : launch_split<128, 1>(a, st);
  return two ? launch_split<256, 2>(a, st) : launch_split<256, 1>(a, st);
}

GDN_DEFINE_STATUS_GATHER(gather_status_attn_split)

}  // namespace gdn
