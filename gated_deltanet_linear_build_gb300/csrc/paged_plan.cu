// The plan of an attention step: which tiles of query rows there are, and which
// CTA takes which part of them.
//
// The tiles of a step, in sequence order, with the running sum of their kv units,
// and the pieces that the line of units is cut into (or the order in which whole
// tiles are dealt out). One CTA a list: latency bounds it (two rounds of dependent
// loads and a scan each). Measured: 2,048 tokens of 4 prompts 4.7 us, 48 requests 4.3
// us; decode steps of one tile a request need no plan of their own.
#include <algorithm>

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

struct ListArgs {
  int rows, keys, above, upto, cap, grid;          // tiles of the sequences with above < rows <= upto
  int least, over;                                 // units of a piece; of an item's overhead (Cut)
  int wide;                                        // the units may pass 32 bits
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

// Whether `units` more of each thread keep the list's costs within 32 bits; `all` is
// their sum, over all calls.
template <int kPlanThreads>
__device__ bool room_for(const PlanArgs& p, const ListArgs& a, int2* sums, int units, long long& all) {
  int2 tot;
  block_scan<kPlanThreads>(make_int2(units & 0xfff, units >> 12), sums, tot);
  all += tot.x + ((long long)tot.y << 12);
  return all <= kMaxUnits && all * p.Hk <= kMaxUnits * a.grid;
}

template <int kPlanThreads>
__device__ void build_list(const PlanArgs& p, const ListArgs& a, PlanShared<kPlanThreads>& sh, int& items, int& units) {
  const int tid = threadIdx.x;
  int2* sums = sh.sums;
  int* s_first = sh.first;
  items = units = 0;
  long long all = 0;                   // units as a 64-bit number, of wide lists
  // A list whose units do not fit is left empty, and the step with it unwritten.
  auto fits = [&](int more) {
    if (!a.wide || room_for<kPlanThreads>(p, a, sums, more, all)) return true;
    items = units = 0;
    if (tid == 0) record_device_status(GDN_ERR_UNSUPPORTED);
    return false;
  };
  // Well-formed offsets have no more tiles than the list has room for. With others,
  // sequences may overlap: tiles beyond the room are dropped, and their units with
  // them, so that the line is as long as its items.
  for (int n0 = 0; n0 < p.N && items < a.cap; n0 += kPlanThreads) {
    int tiles = 0;
    Seq s = {0, 0, 0};
    if (n0 + tid < p.N) {
      s = seq_of(p.cu, p.kv, n0 + tid, p.T, p.kv_max);
      const int64_t r = (int64_t)s.len * p.G;
      if (r > a.above && r <= a.upto) tiles = (int)((r + a.rows - 1) / a.rows);
    }
    if (!__syncthreads_or(tiles > 1) && min(kPlanThreads, p.N - n0) <= a.cap - items) {
      // One tile a sequence: one scan gives its place and its units.
      Item it = {0, 0, 0, 0};
      if (tiles) it = item_of(p, a, s, n0 + tid, 0);
      if (!fits(it.units)) return;
      int2 tot;
      const int2 inc = block_scan<kPlanThreads>(make_int2(tiles, it.units), sums, tot);
      it.cum = units + inc.y - it.units;
      const int at = items + inc.x - 1;
      if (tiles) {
        a.items[at] = it;
        if (at < kPlanThreads) sh.items[at] = it;
      }
      items += tot.x;
      units += tot.y;
      continue;
    }
    // The tiles' sum in two parts: with overlapping sequences it may pass 32 bits.
    int2 tot;
    const int2 inc = block_scan<kPlanThreads>(make_int2(tiles & 0xfff, tiles >> 12), sums, tot);
    s_first[tid] = (int)min(inc.x + ((long long)inc.y << 12) - tiles, 0x7fffffffll);
    const int here = (int)min(tot.x + ((long long)tot.y << 12), (long long)(a.cap - items));
    __syncthreads();
    for (int i0 = 0; i0 < here; i0 += kPlanThreads) {
      const int i = i0 + tid;
      Item it = {0, 0, 0, 0};
      if (i < here) {
        int lo = 0, hi = kPlanThreads - 1;     // last sequence whose first tile is <= i
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_first[mid] <= i) lo = mid; else hi = mid - 1;
        }
        it = item_of(p, a, seq_of(p.cu, p.kv, n0 + lo, p.T, p.kv_max), n0 + lo, i - s_first[lo]);
      }
      if (!fits(it.units)) return;
      int2 tot_units;
      const int2 cum = block_scan<kPlanThreads>(make_int2(0, it.units), sums, tot_units);
      it.cum = units + cum.y - it.units;
      if (i < here) {
        a.items[items + i] = it;
        if (items + i < kPlanThreads) sh.items[items + i] = it;
      }
      units += tot_units.y;
    }
    items += here;
    __syncthreads();                           // s_first is free again
  }
}

// Every CTA's piece of the list's line.
template <int kPlanThreads>
__device__ void cut_line(const PlanArgs& p, const ListArgs& a, PlanShared<kPlanThreads>& sh, int num, int units) {
  int2* sums = sh.sums;
  int* s_pieces = sh.first;
  const long long all = (long long)units * p.Hk;
  int longest = 0;
  if (by_longest((long long)num * p.Hk, a.grid)) {   // no more items than threads, then
    __syncthreads();                             // the list is written
    longest = __reduce_max_sync(0xffffffffu, threadIdx.x < num ? sh.items[threadIdx.x].units : 0);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5].x = longest;
    __syncthreads();
    longest = __reduce_max_sync(0xffffffffu, sums[threadIdx.x & (kPlanThreads / 32 - 1)].x);
  }
  const Cut cut = cut_of(all, (long long)num * p.Hk, longest, a.grid, a.least, a.over);
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
  const int64_t rows = (int64_t)T * G;
  auto wide = [&](int tile_rows, int keys, int grid) {
    const int64_t most = most_units(rows / tile_rows + N, kv_max, keys);
    return most > kMaxUnits || most * Hk > kMaxUnits * grid;
  };
  // A piece of the split kernel gives each of its 8 warps a unit at least.
  if (use.split)
    p.list[lists++] = {l.split_rows, kUnit, 0, limit, l.item_cap, split_grid(d, l.split_rows), kWarps,
                       kSplitOver, wide(l.split_rows, kUnit, split_grid(d, l.split_rows)), reinterpret_cast<Item*>(ws + l.items), nullptr,
                       reinterpret_cast<Start*>(ws + l.starts)};
  if (use.tile)
    p.list[lists++] = {l.tile_rows, kTileKeys, limit, 0x7fffffff, l.tile_cap, tile_grid(), 1,
                       kItemCost, wide(l.tile_rows, kTileKeys, tile_grid()), reinterpret_cast<Item*>(ws + l.tiles),
                       reinterpret_cast<Item*>(ws + l.sorted_tiles),
                       reinterpret_cast<Start*>(ws + l.tile_starts)};
  // A warp more is a turn more for every instruction of the others: 256 threads
  // where they hold the sequences and the items (4 prompts: 6.1 -> 4.7 us).
  const bool small = N <= 256 && (!use.split || rows / l.split_rows + N <= 256) &&
                     (!use.tile || rows / l.tile_rows + N <= 256);
  return check_launch(small ? launch_pdl(attn_plan_kernel<256>, dim3(lists), dim3(256), 0, st, p)
                            : launch_pdl(attn_plan_kernel<1024>, dim3(lists), dim3(1024), 0, st, p));
}

GDN_DEFINE_STATUS_GATHER(gather_status_attn_plan)

}  // namespace gdn
