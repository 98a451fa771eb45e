// Shared by the paged-attention units: the plan that one launch builds from
// the step's lengths and the others read, and its layout in the workspace.
#pragma once

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

// A CTA's piece [u, u_end) of the work line (units of all heads), with all that
// its first segment needs: one 64-byte line instead of a chain of loads.
struct alignas(64) Start {
  int item, head, num_items, units;   // of unit u; of the list: tiles, one head's units
  Item it;
  int first, len, kv, per_cta;        // the item's sequence; units per CTA
  long long u, u_end;
};

struct Layout {
  size_t starts, tile_starts, items, counters, partials, tiles, tile_partials, total;
  int item_cap, tile_cap, split_rows, tile_rows;
};

// Rows of a tile of the tensor-core kernel.
inline int tile_rows(int d) { return d == 256 ? 128 : 256; }
inline int tile_grid() { return num_sms() < 160 ? num_sms() : 160; }

// Sequences of at most this many rows (new tokens x G) go to the split kernel.
inline int split_limit(int G) { return 64; }

// Rows of a split tile: 16 where the query heads of a token need more than 8.
inline int split_rows(int G) { return G > 8 ? 16 : 8; }

// CTAs of the split kernel: one wave, by the shared memory of its rings.
constexpr int kSplitGridMax = 320;
inline int split_grid(int d) {
  const int n = num_sms() * (d == 256 ? 1 : 2);
  return n < kSplitGridMax ? n : kSplitGridMax;
}

Layout layout(int T, int N, int Hq, int Hk, int d);

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
  int* counters;                       // arrivals, see the split kernel
  float* partials;
  Item* tiles;
  int split_rows, split_grid, tile_grid;
  const Start *starts, *tile_starts;
  float* tile_partials;
};

// Lengths of sequence n, malformed ones as an empty sequence.
struct Seq {
  int first, len, kv;
};
__device__ __forceinline__ Seq seq_of(const int32_t* cu, const int32_t* kv, int n, int T,
                                      int64_t kv_max) {
  Seq s;
  s.first = __ldg(cu + n);
  s.len = __ldg(cu + n + 1) - s.first;
  if (s.first < 0 || s.len < 0 || s.first > T - s.len) s.first = s.len = 0;
  const int64_t k = __ldg(kv + n);
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

}  // namespace attn

gdn_status_t launch_attn_plan(const int32_t* cu, const int32_t* kv, int N, int T, int Hq, int Hk,
                              int d, int64_t kv_max, void* workspace, cudaStream_t st);
gdn_status_t launch_attn_split(const attn::Args& a, cudaStream_t st);
gdn_status_t launch_attn_tile(const attn::Args& a, cudaStream_t st);

}  // namespace gdn
