// Joins the float32 partial results of items that the attention kernels cut.
//
// Bound: latency (two rounds of dependent loads, a sum over an item's pieces),
// or the partial results' bytes, which are in L2. One launch for both kernels,
// and a grid bounded by the step's items, few CTAs where they are few: 1,216 CTAs
// of which most had nothing to do cost a step 12 us.
// Measured: 8 heads' tiles of 19 pieces 3 us (64 tokens behind 30,000), 40 MB of
// partial results of 4,096 tokens 10 us.
#include <algorithm>

#include "paged_attn.cuh"

namespace gdn {
namespace {
using namespace attn;

constexpr int kJoinThreads = 256;
constexpr int kTileGridMax = 160;
// Up to this many cut tiles the form for few. 64 tokens a sequence behind 20,000,
// step in us, few / many: 1 sequence x 8 heads (16 tiles at most) 40 / 54, 2 (32)
// 64.6 / 64.5, 3 (48) 82 / 80; d = 256, 1 x 2 heads (10) 40 / 71, 4 (40) 88 / 90,
// 8 (80) 148 / 146.
constexpr int kFewTiles = 32;

struct JoinShared {
  int count[kJoinThreads / 32], c0;
  Start next;
  union {
    struct {
      float f[kSplitGridMax * 16];     // factors [partial][row]
      float l[16];
      float4 o[kJoinThreads];
    } split;
    float2 ml[kTileGridMax * 32];      // maximum and sum [partial][row]
  };
};

// The k-th piece that begins an item and ends inside it: its CTA in sh.c0 and the
// next CTA's piece in sh.next; false if there are no more.
__device__ __forceinline__ bool find_cut(JoinShared& sh, const Start* starts, int pieces, int k) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int base = 0; base + 1 < pieces; base += kJoinThreads) {
    const int c = base + tid;
    bool cut = false;
    Start next;
    if (c + 1 < pieces) {
      next = read_start(starts + c + 1);
      cut = next.count > 0 && next.c0 == c && next.u != (long long)next.head * next.units + next.it.cum;
    }
    const unsigned vote = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) sh.count[w] = __popc(vote);
    if (tid == 0) sh.c0 = -1;
    __syncthreads();
    int before = __popc(vote & ((1u << lane) - 1)), total = 0;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) {
      if (i < w) before += sh.count[i];
      total += sh.count[i];
    }
    if (cut && before == k) {
      sh.c0 = c;
      sh.next = next;
    }
    __syncthreads();
    if (sh.c0 >= 0) return true;
    k -= total;
    __syncthreads();
  }
  return false;
}

// Split kernel: the k-th cut item, the y-th of COLS shares of its elements. Thread
// groups share a long item's partials; each adds its own in CTA order, and the
// groups are added in order: the order is fixed.
template <int D, int QM, int COLS>
__device__ __forceinline__ void join_split(const Args& p, JoinShared& sh, int k0, int y) {
  constexpr int rows = 8 * QM, elems = rows * D / 4 / COLS;           // float4 of this CTA
  constexpr int lanes = elems < kJoinThreads ? elems : kJoinThreads;  // threads of a group
  constexpr int groups = kJoinThreads / lanes;
  static_assert(kJoinThreads % lanes == 0 && elems % lanes == 0, "whole groups");
  if (!find_cut(sh, p.starts, p.split_grid, k0)) return;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const Start& next = sh.next;
  const int n = next.pieces;
  const float* base = p.partials + ((size_t)sh.c0 * 2 + 1) * (rows * (D + 2));
  auto part = [&](int c) { return base + (c == 0 ? 0 : (size_t)(2 * c - 1) * (rows * (D + 2))); };
  const int group = tid / lanes, from = n * group / groups, to = n * (group + 1) / groups;
  // Eight loads at a time (a chain of single ones would take 0.5 us each), the
  // first of them before the factors are known.
  float4 v[8];
  auto fetch = [&](int e, int c) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < to) v[k] = __ldcg(reinterpret_cast<const float4*>(part(c + k) + 2 * rows + e));
  };
  const int e0 = (y * elems + tid % lanes) * 4;
  fetch(e0, from);
  for (int r = w; r < rows; r += kJoinThreads / 32) {
    float top = -INFINITY, l = 0.f;
    constexpr int per = (kSplitGridMax + 31) / 32;
    float2 ml[per];
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int c = lane + 32 * k;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (c < n) ml[k] = __ldcg(reinterpret_cast<const float2*>(part(c)) + r);
      top = fmaxf(top, ml[k].x);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int c = lane + 32 * k;
      // NaN sums pass on: a NaN row has m = -inf and its l as it is.
      const float f = ml[k].x == -INFINITY ? 1.f : ex2_approx(ml[k].x - top);
      if (c < n) sh.split.f[c * rows + r] = f;
      l = add_scaled(l, ml[k].y, f, ml[k].x - top);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    if (lane == 0) sh.split.l[r] = l;
  }
  __syncthreads();
  const int G = p.Hq / p.Hk;
  const RowsOut out = {p.o, next.first, next.it.row0, min(rows, next.len * G - next.it.row0), G, p.Hq, next.head};
#pragma unroll 1
  for (int i = 0; i < elems; i += lanes) {
    const int e = e0 + i * 4, r = e / D;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = from; c < to; c += 8) {
      if (c > from || i > 0) fetch(e, c);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < to) {
          const float f = sh.split.f[(c + k) * rows + r];
          o.x = fmaf(v[k].x, f, o.x);
          o.y = fmaf(v[k].y, f, o.y);
          o.z = fmaf(v[k].z, f, o.z);
          o.w = fmaf(v[k].w, f, o.w);
        }
    }
    if constexpr (groups > 1) {
      sh.split.o[tid] = o;
      __syncthreads();
      if (group > 0) return;                   // elems == lanes here
#pragma unroll
      for (int k = 1; k < groups; ++k) {
        const float4 a = sh.split.o[k * lanes + tid];
        o.x += a.x;
        o.y += a.y;
        o.z += a.z;
        o.w += a.w;
      }
    }
    put_row4<D>(out, r, e % D, o, sh.split.l[r]);
  }
}

// Tensor-core kernel. Lane i has row i of 32 (the partials' layout [column][128
// rows] keeps its loads whole), each warp columns of its own; pieces are added in
// CTA order.
template <int D>
struct TilePart {
  static constexpr int kM = D == 256 ? 1 : 2;
  static constexpr size_t size = (size_t)(D + 2) * 128;
  const float* base;
  // The item's first piece, CTA c0's, is that CTA's second partial result, the
  // others first ones. r: row of the tile's 128-row part m.
  __device__ __forceinline__ TilePart(const Args& p, int c0, int m, int r)
      : base(p.tile_partials + ((size_t)c0 * 2 * kM + m) * size + r) {}
  __device__ __forceinline__ const float* operator()(int c) const {
    return base + (size_t)(2 * c + (c == 0)) * kM * size;
  }
};
template <int N>
__device__ __forceinline__ void put_cols(__nv_bfloat16* at, const float (&v)[N], float il) {
  uint32_t w[N / 2];
#pragma unroll
  for (int k = 0; k < N / 2; ++k) w[k] = pack_bf16x2(put_one(v[2 * k], il), put_one(v[2 * k + 1], il));
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int k = 0; k < N / 2; k += 4)
      *reinterpret_cast<uint4*>(at + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t*>(at) = w[0];
  }
}

// Few tiles, of many pieces each: CTA (k, y) takes the k-th cut one and of it 32
// rows and a quarter of the columns, with 32 loads of a thread in flight.
template <int D>
__device__ __forceinline__ void join_tile_few(const Args& p, JoinShared& sh, int k0, int y) {
  constexpr int kCols = D / 32, kBatch = 32 / kCols;
  if (!find_cut(sh, p.tile_starts, p.tile_grid, k0)) return;
  const Start& next = sh.next;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int m = y >> 4, r = ((y >> 2) & 3) * 32 + lane, col0 = ((y & 3) * 8 + w) * kCols;
  const int G = p.Hq / p.Hk, n = next.pieces;
  const int row = next.it.row0 + m * 128 + r, tok = row / G;
  if (row - lane >= next.len * G) return;                // none of the CTA's rows
  const TilePart<D> part(p, sh.c0, m, r);
  for (int c = w; c < n; c += kJoinThreads / 32)
    sh.ml[c * 32 + lane] = make_float2(__ldcg(part(c)), __ldcg(part(c) + 128));
  float v[kBatch][kCols];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (c0 + i < n) v[i][k] = __ldcg(part(c0 + i) + (size_t)(2 + col0 + k) * 128);
  };
  fetch(0);
  __syncthreads();
  float top = -INFINITY, l = 0.f, o[kCols];
  for (int c = 0; c < n; ++c) top = fmaxf(top, sh.ml[c * 32 + lane].x);
#pragma unroll
  for (int k = 0; k < kCols; ++k) o[k] = 0.f;
#pragma unroll 1
  for (int c = 0; c < n; c += kBatch) {
    if (c > 0) fetch(c);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i < n) {
        const float2 ml = sh.ml[(c + i) * 32 + lane];
        // NaN sums pass on: a NaN row has m = -inf and its l as it is.
        const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
        l = add_scaled(l, ml.y, f, ml.x - top);
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[k] = fmaf(v[i][k], f, o[k]);
      }
  }
  if (row < next.len * G)
    put_cols(p.o + ((int64_t)(next.first + tok) * p.Hq + next.head * G + row - tok * G) * D + col0, o,
             over_sum(l));
}

// Many tiles, of two or three pieces: CTA (c0, y) takes the one, if any, that CTA c0
// began and did not end, and of it 32 rows.
template <int D>
__device__ __forceinline__ void join_tile_many(const Args& p, int c0, int y) {
  constexpr int kCols = D / 8;
  const Start next = read_start(p.tile_starts + c0 + 1);
  if (next.count == 0 || next.c0 != c0 || next.u == (long long)next.head * next.units + next.it.cum)
    return;
  const int lane = threadIdx.x & 31, m = y >> 2, r = (y & 3) * 32 + lane, col0 = (threadIdx.x >> 5) * kCols;
  const int G = p.Hq / p.Hk, n = next.pieces;
  const int row = next.it.row0 + m * 128 + r, tok = row / G;
  if (row >= next.len * G) return;
  const TilePart<D> part(p, c0, m, r);
  float top = -INFINITY, l = 0.f, o[kCols];
#pragma unroll 4
  for (int c = 0; c < n; ++c) top = fmaxf(top, __ldcg(part(c)));
#pragma unroll
  for (int k = 0; k < kCols; ++k) o[k] = 0.f;
#pragma unroll 2
  for (int c = 0; c < n; ++c) {
    const float* q = part(c);
    const float mc = __ldcg(q);
    const float f = mc == -INFINITY ? 1.f : ex2_approx(mc - top);
    l = add_scaled(l, __ldcg(q + 128), f, mc - top);
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[k] = fmaf(__ldcg(q + (size_t)(2 + col0 + k) * 128), f, o[k]);
  }
  put_cols(p.o + ((int64_t)(next.first + tok) * p.Hq + next.head * G + row - tok * G) * D + col0, o,
           over_sum(l));
}

// CTAs [0, split_ctas): the split kernel's items, `cuts` of them at most; the
// others: the tensor-core kernel's, tile_cuts at most.
template <int D, int QM, int COLS>
__global__ void __launch_bounds__(kJoinThreads)
attn_join_kernel(const Args p, const int split_ctas, const int cuts, const int tile_cuts) {
  __shared__ JoinShared sh;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x - split_ctas;
  if (b < 0) join_split<D, QM, COLS>(p, sh, blockIdx.x % cuts, blockIdx.x / cuts);
  else if (tile_cuts <= kFewTiles) join_tile_few<D>(p, sh, b % tile_cuts, b / tile_cuts);
  else join_tile_many<D>(p, b % tile_cuts, b / tile_cuts);
}

// Many tiles alone: without the other forms' shared memory and registers more CTAs
// are resident (4,096 tokens of 16,384: the step 743 -> 739 us).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_tiles_kernel(const Args p, const int tile_cuts) {
  pdl_wait();
  pdl_trigger();
  join_tile_many<D>(p, blockIdx.x % tile_cuts, blockIdx.x / tile_cuts);
}

template <int D, int QM>
gdn_status_t launch_join(const Args& a, bool split, bool tile, cudaStream_t st) {
  // At most one cut item per piece, and no more than there are items.
  const int64_t rows = (int64_t)a.T * (a.Hq / a.Hk);
  auto most = [&](int grid, int tile_rows) {
    return (int)std::min<int64_t>(grid - 1, (rows / tile_rows + a.N) * a.Hk);
  };
  const int cuts = split ? most(a.split_grid, 8 * QM) : 0;
  int tile_cuts = tile ? most(a.tile_grid, 128 * TilePart<D>::kM) : 0;
  if (tile_cuts > kFewTiles) tile_cuts = a.tile_grid - 1;
  // Long items (many partials each) are few: more CTAs share one.
  const int cols = cuts <= 16 ? 8 : 2, shares = TilePart<D>::kM * 4 * (tile_cuts <= kFewTiles ? 4 : 1);
  const int grid = cuts * cols + tile_cuts * shares;
  if (grid <= 0) return GDN_OK;
  if (cuts == 0 && tile_cuts > kFewTiles)
    return check_launch(launch_pdl(attn_join_tiles_kernel<D>, dim3(grid), dim3(kJoinThreads), 0, st, a, tile_cuts));
  const auto kernel = cols == 8 ? attn_join_kernel<D, QM, 8> : attn_join_kernel<D, QM, 2>;
  return check_launch(launch_pdl(kernel, dim3(grid), dim3(kJoinThreads), 0, st, a, cuts * cols,
                                 std::max(cuts, 1), std::max(tile_cuts, 1)));
}

}  // namespace

gdn_status_t launch_attn_join(const Args& a, bool split, bool tile, cudaStream_t st) {
  const bool two = a.split_rows == 16;
  if (a.d == 64) return two ? launch_join<64, 2>(a, split, tile, st) : launch_join<64, 1>(a, split, tile, st);
  if (a.d == 128) return two ? launch_join<128, 2>(a, split, tile, st) : launch_join<128, 1>(a, split, tile, st);
  return two ? launch_join<256, 2>(a, split, tile, st) : launch_join<256, 1>(a, split, tile, st);
}

}  // namespace gdn
