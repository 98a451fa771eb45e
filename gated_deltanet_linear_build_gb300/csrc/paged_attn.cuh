// Shared by the paged-attention units: the plan that one launch builds from
// the step's lengths and the others read, and its layout in the workspace.
#pragma once

#include <cuda.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace attn {

// A query row of (sequence, kv head) is r = token * G + g: G = Hq / Hk query
// heads share the kv head, so their rows share every K and V byte read.

// One row tile of a sequence; it stands for Hk items, one per kv head.
struct Item {
  int seq;
  int row0;      // first row of the tile
  int units;     // kv units that the tile's last row sees
  int cum;       // units of the tiles before it
};

constexpr int kUnit = 32;              // keys per unit of the split kernel
constexpr int kTileKeys = 64;         // keys per unit of the tensor-core kernel

// A CTA's piece of the work line (units of all heads), `count` units from u, with
// all that its first segment needs: one 64-byte line instead of a chain of loads.
struct alignas(64) Start {
  int item, head, num_items, units;   // of unit u; of the list: tiles, one head's units
  Item it;
  int first, len, kv;                 // the item's sequence
  int c0;                             // the CTA that begins the item (-1: whole items are dealt)
  long long u;
  int count, pieces;                  // pieces of the item
};

struct Layout {
  size_t starts, self_starts, tile_starts, items, partials, tiles, sorted_tiles, tile_partials, total;
  int item_cap, tile_cap, split_rows, tile_rows;
};

// Rows of a split tile: 16 where the query heads of a token need more than 8.
inline int split_rows(int G) { return G > 8 ? 16 : 8; }

// Rows of a tile of the tensor-core kernel.
inline int tile_rows(int d) { return d == 256 ? 128 : 256; }
inline int tile_grid() { return num_sms() < 160 ? num_sms() : 160; }

// Sequences of at most this many rows (new tokens x G) go to the split kernel.
inline int split_limit(int G) { return 64; }

// Which kernels a step's lengths leave work for, and the most rows that go to the
// split kernel. One sequence is exactly as long as the step. A step with longer
// sequences whose short ones cannot hold up the tensor-core kernel (all of them
// with full tables are two units an SM at most) leaves the split kernel out: two
// launches with next to nothing to do are 5 us.
struct Kernels {
  bool split, tile;
  int limit;
};
inline Kernels kernels_of(int N, int T, int G, int Hk, int max_new_tokens, int64_t kv_max) {
  const int64_t longest = N == 1 ? T : max_new_tokens;
  Kernels k = {true, longest * G > split_limit(G), split_limit(G)};
  const int64_t short_units = (int64_t)N * Hk * ((kv_max + kTileKeys - 1) / kTileKeys);
  if (k.tile && (N == 1 || short_units <= 2 * tile_grid())) {
    k.split = false;
    k.limit = 0;
  }
  return k;
}
// A list's units and costs are 32-bit numbers. Units that one head's line may have
// (kv_max: the table's width), in sequences of any length up to it.
inline int64_t most_units(int64_t tiles, int64_t kv_max, int keys) {
  const int64_t kv = kv_max < 0x7fffffff ? kv_max : 0x7fffffff;
  return tiles * ((kv + keys - 1) / keys);
}
constexpr int64_t kMaxUnits = 1 << 30;
constexpr int kSelfPlan = 512;
// Whether the split kernel's CTAs can plan the step by themselves: one tile a
// sequence, no more of them than one block scans. A decode step of 32 requests
// takes 17.0 us with a plan of its own, and 19.4 us with the
// plan's kernel.
inline bool self_planned(int N, int T, int G, int Hk, int max_new_tokens, int64_t kv_max) {
  const int64_t longest = N == 1 ? T : max_new_tokens;
  return N <= kSelfPlan && longest * G <= split_rows(G) && most_units(N, kv_max, kUnit) * Hk <= kMaxUnits;
}

// CTAs of the split kernel: one wave.
constexpr int kSplitGridMax = 320;
inline int split_grid(int d, int rows) {
  const int n = num_sms() * (d * rows <= 8 * 128 ? 2 : 1);
  return n < kSplitGridMax ? n : kSplitGridMax;
}

Layout layout(int T, int N, int Hq, int Hk, int d);

constexpr int kWarps = 8;              // warps of a CTA of the split kernel

// Bytes of a cache row in one TMA box: the widest swizzle.
__host__ __device__ constexpr int box_row(int d) { return d == 64 ? 64 : 128; }
// The cache as (d, token of the block, block x head), boxes of `rows` tokens.
bool cache_map(CUtensorMap* map, const void* cache, int d, int B, int64_t pages, int rows);

// TMA box: rows of one (block, head) to shared memory.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, int z,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(tc::smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
// K-major operand of 128-byte (64-byte) swizzled rows: 8-row groups 8 rows apart.
template <int kRow>
__device__ __forceinline__ uint64_t desc_swizzled(uint32_t addr) {
  return tc::smem_desc(addr, 16, 8 * kRow) | ((uint64_t)(kRow == 128 ? 2 : 4) << 61);
}
// Byte of chunk c of row r under that swizzle.
template <int kRow>
__device__ __forceinline__ int swizzled(int r, int c) {
  if constexpr (kRow == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}


struct Args {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t* table;
  int64_t table_stride;
  const int32_t *cu, *kv;
  __nv_bfloat16* o;
  int N, T, Hq, Hk, d, log_b, num_blocks, max_blocks;
  float scale_log2;                    // softmax scale x log2 e
  Item* items;
  float* partials;
  Item *tiles, *sorted_tiles;          // in sequence order; by length
  int split_rows, split_grid, tile_grid;
  Start* starts;
  const Start* tile_starts;
  int self_plan;                       // the split kernel's CTAs plan by themselves
  int after_split;                     // the tensor-core kernel is launched behind the split kernel
  float* tile_partials;
};

// Lengths of sequence n, malformed ones as an empty sequence. kPlain: without
// ld.global.nc, for a kernel that reads them without a wait of its own.
struct Seq {
  int first, len, kv;
};
template <bool kPlain = false>
__device__ __forceinline__ Seq seq_of(const int32_t* cu, const int32_t* kv, int n, int T,
                                      int64_t kv_max) {
  auto at = [](const int32_t* p) { return kPlain ? *p : __ldg(p); };
  Seq s;
  s.first = at(cu + n);
  s.len = at(cu + n + 1) - s.first;
  if (s.first < 0 || s.len < 0 || s.first > T - s.len) s.first = s.len = 0;
  const int64_t k = at(kv + n);
  s.kv = (int)(k < 0 ? 0 : k > kv_max ? kv_max : k);
  return s;
}
__device__ __forceinline__ Start read_start(const Start* at) {
  union {
    int4 v[4];
    Start s;
  } x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = reinterpret_cast<const int4*>(at)[i];
  return x.s;
}
// Keys that row r of the sequence sees: [0, visible).
__device__ __forceinline__ int visible(const Seq& s, int token) {
  return max(0, s.kv - s.len + token + 1);
}

// What an item costs beside its units, in units: a segment's start and end. (Split
// kernel, 0 / 8 / 16 / 32: 256 decode requests of up to 1,000 tokens 77 / 69 / 66
// / 68 us, 400 of up to 2,000 at d = 256 95 / 84 / 81 / 85 us. Tensor-core kernel,
// 5 / 8 / 12: 4,096 tokens behind 4,000, d = 256, 294 / 288 / 286 us.)
constexpr int kSplitOver = 16, kItemCost = 10;

// The line is cut in one of two ways. Into pieces of equal cost, which may end
// inside an item and go on with the next: no SM is idle. An item costs its units
// and `over` more (a segment's start and end). Or, where there are fewer items than
// CTAs, each item by itself into pieces of at most `target` units: a piece then is
// one segment (a CTA with two held up a step of one 16,000-token request by 4 of 10
// us). With target >= all / (grid - items) the pieces are no more than the CTAs.
// Taken where items are no more than half as many as CTAs, or their longest piece
// is not much above the other way's share, which has some of a segment's overhead
// more to bear. (d = 256, 2 kv heads, 60 requests of 512-1,143 tokens: 18.7 us by
// items, 20.4 in equal pieces; 75 requests: 19.0, 22.7.)
struct Cut {
  int per_cta, target;                 // target 0: pieces of equal cost
};
// Whether cut_of needs the longest item.
__device__ __forceinline__ bool by_longest(long long items, int grid) { return 2 * items > grid && items < grid; }
__device__ __forceinline__ Cut cut_of(long long all, long long items, int longest, int grid, int least, int over) {
  Cut c;
  c.per_cta = (int)max((long long)least, (all + items * over + grid - 1) / grid);
  c.target = 0;
  if (items < grid) {
    const int target = (int)max((long long)least, (all + grid - items - 1) / (grid - items));
    if (2 * items <= grid || min(target, longest) <= c.per_cta + over / 4) c.target = target;
  }
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

// sum + y 2^x, with f = ex2_approx(x): 2^x alone may lie below float32's range where
// the blocks' V scales lie far apart, and y above it by as much.
__device__ __forceinline__ float add_scaled(float sum, float y, float f, float x) {
  const float h = ex2_approx(0.5f * x);
  return x < -100.f ? fmaf(y * h, h, sum) : fmaf(y, f, sum);
}
// The sum of the weights P' / vs is kept 2^-16 times: P' reaches 2^15 and 1 / vs 2^100,
// so that 4,096 keys of the smallest scale would pass float32's range.
constexpr float kSumScale = 1.f / 65536.f;
// What a row's outputs are to be multiplied by, for its sum l; put_one does.
__device__ __forceinline__ float over_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float put_one(float o, float il) { return o * kSumScale * il; }
// A weight P' = 2^(s + log2 vs - m) of a small vs may be below float32's range though
// P' / vs is as large as any. Where a unit's largest P' is 2^-kFarUnit or more, and the
// V scales within it are within 2^kFarApart, what is lost is below 2^(kFarUnit +
// kFarApart - 133) = 2^-33 of the unit's largest weight. In other units the sum takes
// P' 2^100 instead, where 1 / vs makes room for that.
constexpr float kFarUnit = 60.f, kFarApart = 40.f;
// What the sum's exponents and factors change by, for a block of kSumScale / vs = iv.
__device__ __forceinline__ float far_shift(float iv) { return iv >= kSumScale ? 100.f : 0.f; }
__device__ __forceinline__ float far_factor(float iv) { return iv >= kSumScale ? iv * 7.888609052210118e-31f : iv; }

// The split kernel's V chunk of lane group g.
__device__ __forceinline__ int v_chunk(int g) { return (g >> 1) | ((g & 1) << 2); }
// d of element `pos` of a row of O as the warps leave it: [m-tile k][g][2].
template <int D>
__device__ __forceinline__ int d_of(int pos) {
  const int k = pos >> 4, g = (pos >> 1) & 7, b = pos & 1;
  if constexpr (D == 64) return g * 8 + 2 * k + b;
  return 128 * (k >> 3) + 16 * v_chunk(g) + 2 * (k & 7) + b;
}

// Where the rows of a tile go.
struct RowsOut {
  __nv_bfloat16* o;
  int first, row0, n_rows, G, Hq, head;
};
// Four elements of row r, from position pos, over their sum l.
template <int D>
__device__ __forceinline__ void put_row4(const RowsOut& t, int r, int pos, float4 o, float l) {
  if (r >= t.n_rows) return;
  const int row = t.row0 + r, tok = row / t.G;
  const float il = over_sum(l);
  __nv_bfloat16* at = t.o + ((int64_t)(t.first + tok) * t.Hq + t.head * t.G + row - tok * t.G) * D;
  *reinterpret_cast<uint32_t*>(at + d_of<D>(pos)) = pack_bf16x2(put_one(o.x, il), put_one(o.y, il));
  *reinterpret_cast<uint32_t*>(at + d_of<D>(pos + 2)) = pack_bf16x2(put_one(o.z, il), put_one(o.w, il));
}

}  // namespace attn

gdn_status_t launch_attn_plan(const int32_t* cu, const int32_t* kv, int N, int T, int Hq, int Hk,
                              int d, int64_t kv_max, int max_new_tokens, void* workspace,
                              cudaStream_t st);
gdn_status_t launch_attn_split(const attn::Args& a, cudaStream_t st);
gdn_status_t launch_attn_tile(const attn::Args& a, cudaStream_t st);
// Joins what the kernels that ran (split, tile) have cut.
gdn_status_t launch_attn_join(const attn::Args& a, bool split, bool tile, cudaStream_t st);

}  // namespace gdn
