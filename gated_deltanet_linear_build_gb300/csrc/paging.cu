// Paged-cache maps of one engine step: block tables, positions, slots and page
// pieces from the requests' lengths.
//
// With c_n cached and l_n new tokens of sequence n and B tokens per block:
//   need_n  = ceil((c_n + l_n) / B) - ceil(c_n / B)       blocks to take,
//   first_n = sum over m < n of need_m                    where they lie in the free list,
//   table[n, ceil(c_n / B) + j] = free[first_n + j],      j < need_n.
// A token at position p of sequence n goes to slot table[n, p / B] * B + p % B,
// and every (sequence, block) that receives tokens is one piece.
//
// The work is a prefix sum over the sequences and 12 bytes written per token:
// a few megabytes at most, so launches and dependent loads bound it, not
// bandwidth. One launch: every CTA owns a contiguous slice of tokens and forms
// the prefix sums it needs itself (one block-wide reduction over all earlier
// sequences, which also gives the totals that decide whether the step fits),
// instead of a scan kernel followed by a fill kernel. Every CTA then reads every
// sequence's lengths, which is most of the time where they are many. 4,000
// sequences, 125,000 tokens: 6.2 us alone, 7.2 to 8.0 in a stream of other calls
// (10.2 us alone with the sums of a slice formed in two passes).
#include <algorithm>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabSeqs = 512;          // sequences per tile of a slice

struct SeqLens {
  int first, len, ctx;
};

// Lengths of sequence n; bad is set where the inputs are malformed.
__device__ __forceinline__ SeqLens seq_lens(const int32_t* cu, const int32_t* ctx, int n, int T,
                                            int& bad) {
  SeqLens s;
  s.first = __ldg(cu + n);
  const int end = __ldg(cu + n + 1);
  s.len = end - s.first;
  s.ctx = __ldg(ctx + n);
  if (s.first < 0 || s.len < 0 || end > T || s.ctx < 0 || s.ctx > 0x7fffffff - 128 - s.len) {
    bad = 1;
    s.first = s.len = s.ctx = 0;
  }
  return s;
}

// Inclusive scan of a pair over the block (kTabThreads threads); total in tot.
__device__ __forceinline__ int2 block_scan2(int2 v, int2* warp_sums, int2& tot) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  constexpr int kWarps = kTabThreads / 32;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v.x, d), b = __shfl_up_sync(0xffffffffu, v.y, d);
    if (lane >= d) { v.x += a; v.y += b; }
  }
  __syncthreads();                     // earlier readers of warp_sums are done
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  int2 before = make_int2(0, 0);
  tot = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int2 s = warp_sums[i];
    if (i < w) { before.x += s.x; before.y += s.y; }
    tot.x += s.x;
    tot.y += s.y;
  }
  return make_int2(v.x + before.x, v.y + before.y);
}

struct TabArgs {
  const int32_t *cu, *ctx, *free_blocks;
  int num_free, N, T, log_b, max_blocks;
  int64_t table_stride;
  int32_t *table, *kv, *positions;
  int64_t* slots;
  gdn_page_piece_t* pieces;
  int piece_cap;
  int32_t *counts, *status;
};

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TabArgs p) {
  __shared__ int2 warp_sums[kTabThreads / 32];
  __shared__ int s_cu[kTabSeqs + 1], s_ctx[kTabSeqs], s_need[kTabSeqs], s_piece[kTabSeqs];
  __shared__ int s_sum[6];             // first sequence, needs and pieces before it, of all, errors
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int B = 1 << p.log_b;
  const int per = (p.T + gridDim.x - 1) / gridDim.x;
  const int t0 = min(p.T, (int)blockIdx.x * per), t1 = min(p.T, t0 + per);

  if (tid < 6) s_sum[tid] = 0;
  __syncthreads();
  // Needs and pieces of the sequences that end at or before t0, and of all; the
  // former are those before the slice's first sequence.
  int first = 0, need_b = 0, pcs_b = 0, need_a = 0, pcs_a = 0, bad = 0;
#pragma unroll 4
  for (int n = tid; n < p.N; n += kTabThreads) {
    const SeqLens s = seq_lens(p.cu, p.ctx, n, p.T, bad);
    const int have = (s.ctx + B - 1) >> p.log_b, want = (s.ctx + s.len + B - 1) >> p.log_b;
    const int need = want - have, pcs = s.len > 0 ? want - (s.ctx >> p.log_b) : 0;
    if (want > p.max_blocks && s.len > 0) bad |= 2;
    need_a += need;
    pcs_a += pcs;
    if (s.first + s.len <= t0) {
      ++first;
      need_b += need;
      pcs_b += pcs;
    }
  }
  if (tid == 0 && (__ldg(p.cu) != 0 || __ldg(p.cu + p.N) != p.T)) bad |= 1;
  const int sums[6] = {first, need_b, pcs_b, need_a, pcs_a, bad};
#pragma unroll
  for (int k = 0; k < 6; ++k) {
    const int v = k < 5 ? __reduce_add_sync(0xffffffffu, sums[k]) : __reduce_or_sync(0xffffffffu, sums[k]);
    if ((tid & 31) == k) {
      if (k < 5) atomicAdd(s_sum + k, v);
      else atomicOr(s_sum + k, v);
    }
  }
  __syncthreads();
  const int n0 = s_sum[0];
  const int2 tot_before = make_int2(s_sum[1], s_sum[2]), tot_all = make_int2(s_sum[3], s_sum[4]);
  int err = s_sum[5];
  if (tot_all.x > p.num_free || tot_all.y > p.piece_cap) err |= 2;
  const int status = (err & 1) ? GDN_ERR_INVALID_ARG : err ? GDN_ERR_WORKSPACE : GDN_OK;
  if (blockIdx.x == 0 && tid == 0) {
    p.counts[0] = err ? 0 : tot_all.y;
    p.counts[1] = err ? 0 : tot_all.x;
    if (p.status) *p.status = status;
  }
  if (err) {                            // nothing but the slots is written
    for (int t = t0 + tid; t < t1; t += kTabThreads) p.slots[t] = -1;
    return;
  }
  for (int n = blockIdx.x * kTabThreads + tid; n < p.N; n += gridDim.x * kTabThreads)
    p.kv[n] = __ldg(p.ctx + n) + __ldg(p.cu + n + 1) - __ldg(p.cu + n);

  int2 base = tot_before;
  for (int tile = n0; tile < p.N; tile += kTabSeqs) {
    const int cnt = min(kTabSeqs, p.N - tile);
    int2 mine = make_int2(0, 0);
    __syncthreads();                    // the previous tile's readers are done
    if (tid < cnt) {
      const int first = __ldg(p.cu + tile + tid), end = __ldg(p.cu + tile + tid + 1);
      const int c = __ldg(p.ctx + tile + tid), len = end - first;
      const int have = (c + B - 1) >> p.log_b, want = (c + len + B - 1) >> p.log_b;
      mine = make_int2(want - have, len > 0 ? want - (c >> p.log_b) : 0);
      s_cu[tid] = first;
      s_ctx[tid] = c;
      if (tid == cnt - 1) s_cu[cnt] = end;
    }
    int2 tot;
    const int2 inc = block_scan2(mine, warp_sums, tot);
    if (tid < cnt) {
      s_need[tid] = base.x + inc.x - mine.x;
      s_piece[tid] = base.y + inc.y - mine.y;
    }
    __syncthreads();
    const int from = max(t0, s_cu[0]), to = min(t1, s_cu[cnt]);
    for (int t = from + tid; t < to; t += kTabThreads) {
      int lo = 0, hi = cnt - 1;         // last sequence that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int c = s_ctx[lo], first = s_cu[lo], len = s_cu[lo + 1] - first;
      const int pos = c + (t - first);
      const int idx = pos >> p.log_b, off = pos & (B - 1);
      const int have = (c + B - 1) >> p.log_b;
      int32_t* row = p.table + (int64_t)(tile + lo) * p.table_stride;
      int block;
      if (idx >= have) {
        block = __ldg(p.free_blocks + s_need[lo] + (idx - have));
        if (off == 0) row[idx] = block;  // a taken block's first token enters it in the table
      } else {
        block = row[idx];                // below ceil(c / B): no CTA writes it
      }
      p.positions[t] = pos;
      p.slots[t] = (int64_t)block * B + off;
      if (off == 0 || t == first) {
        const int k = s_piece[lo] + idx - (c >> p.log_b);
        *reinterpret_cast<int4*>(p.pieces + k) =
            make_int4(block, t, min(B - off, first + len - t), off);
      }
    }
    base.x += tot.x;
    base.y += tot.y;
    if (s_cu[cnt] >= t1) break;          // uniform: shared
  }
}

}  // namespace

gdn_status_t launch_block_tables(const int32_t* cu, const int32_t* ctx, const int32_t* free_blocks,
                                 int32_t num_free, int32_t N, int32_t T, int32_t block_tokens,
                                 int32_t* table, int64_t table_stride, int32_t max_blocks,
                                 int32_t* kv, int32_t* positions, int64_t* slots,
                                 gdn_page_piece_t* pieces, int32_t piece_cap, int32_t* counts,
                                 int32_t* status, cudaStream_t st) {
  TabArgs p;
  p.cu = cu;
  p.ctx = ctx;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.N = N;
  p.T = T;
  p.log_b = __builtin_ctz((unsigned)block_tokens);
  p.max_blocks = max_blocks;
  p.table_stride = table_stride;
  p.table = table;
  p.kv = kv;
  p.positions = positions;
  p.slots = slots;
  p.pieces = pieces;
  p.piece_cap = piece_cap;
  p.counts = counts;
  p.status = status;
  // One CTA per kTabThreads tokens until every SM has two.
  const int grid = std::max(1, std::min(2 * num_sms(), (T + kTabThreads - 1) / kTabThreads));
  return check_launch(launch_pdl(block_tables_kernel, dim3(grid), dim3(kTabThreads), 0, st, p));
}

}  // namespace gdn
