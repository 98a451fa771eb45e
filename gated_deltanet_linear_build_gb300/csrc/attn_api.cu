// C ABI of the attention-side operators: host-side argument validation, then
// the kernel launchers. Nothing here allocates device memory or synchronises.
#include <cmath>

#include "paged_attn.cuh"

using namespace gdn;

namespace {

bool block_tokens_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }
bool cache_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool rotary_dim_ok(int d) { return d == 16 || d == 32 || cache_dim_ok(d); }
// Loops over sequences or tokens in strides of a block or a grid end below 2^31.
constexpr int32_t kMaxCount = 0x7fff0000;
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A BF16 tensor of T tokens x H heads x d values, read or written by rows.
gdn_status_t check_rows(const void* x, int64_t stride, int32_t H, int32_t d) {
  if (!x) return GDN_ERR_INVALID_ARG;
  if (stride < (int64_t)H * d) return GDN_ERR_INVALID_ARG;
  if (stride % 8 != 0 || !aligned16(x)) return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

gdn_status_t check_rotation(const int32_t* positions, const int64_t* phases, int32_t d,
                            int32_t rot_dim, int32_t interleaved, int32_t inverse, float scale) {
  if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0) return GDN_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return GDN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 1024.f)) return GDN_ERR_INVALID_ARG;
  if (rot_dim > 0) {
    if (!positions || !phases) return GDN_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned16(phases)) return GDN_ERR_ALIGNMENT;
  }
  return GDN_OK;
}

gdn_status_t check_plan(const int32_t* cu, const int32_t* kv, int32_t N, int32_t T, int32_t Hq,
                        int32_t Hk, int32_t d, int32_t block_tokens, int32_t max_blocks,
                        int32_t max_new_tokens, const void* workspace, size_t bytes,
                        bool* nothing) {
  *nothing = false;
  if (N < 0 || T < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0) return GDN_ERR_INVALID_ARG;
  if (max_blocks < 0 || max_new_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (!cache_dim_ok(d) || !block_tokens_ok(block_tokens) || Hq / Hk > 16 || N > kMaxCount)
    return GDN_ERR_UNSUPPORTED;
  // Keys are counted in 32 bits, up to a few units past a sequence's end.
  if ((int64_t)max_blocks * block_tokens > 0x7fffffff - 1023) return GDN_ERR_UNSUPPORTED;
  if (N == 0 || T == 0) {
    *nothing = true;
    return GDN_OK;
  }
  if (!cu || !kv) return GDN_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || !aligned(kv, 4)) return GDN_ERR_ALIGNMENT;
  if ((int64_t)T * (Hq / Hk) > 0x3fffffff || (int64_t)N * Hk > 0x7fffffff)
    return GDN_ERR_UNSUPPORTED;
  if (!workspace || bytes < attn::layout(T, N, Hq, Hk, d).total) return GDN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_build_block_tables(const int32_t* cu_seqlens, const int32_t* context_lens,
                                    const int32_t* free_blocks, int32_t num_free, int32_t N,
                                    int32_t T, int32_t block_tokens, int32_t* block_table,
                                    int64_t table_stride, int32_t max_blocks, int32_t* kv_lens,
                                    int32_t* positions, int64_t* slots, gdn_page_piece_t* pieces,
                                    int32_t piece_capacity, int32_t* counts,
                                    int32_t* device_status, void* stream) {
  if (N < 0 || T < 0 || num_free < 0 || max_blocks < 0 || piece_capacity < 0 ||
      table_stride < max_blocks)
    return GDN_ERR_INVALID_ARG;
  if (!block_tokens_ok(block_tokens) || N > kMaxCount || T > kMaxCount) return GDN_ERR_UNSUPPORTED;
  if (N == 0) return T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !context_lens || !kv_lens || !counts) return GDN_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_blocks) || (max_blocks > 0 && !block_table) ||
      (T > 0 && (!positions || !slots)) || (piece_capacity > 0 && !pieces))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(context_lens, 4) || !aligned(free_blocks, 4) ||
      !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(positions, 4) ||
      !aligned(slots, 8) || !aligned16(pieces) || !aligned(counts, 4) ||
      !aligned(device_status, 4))
    return GDN_ERR_ALIGNMENT;
  return launch_block_tables(cu_seqlens, context_lens, free_blocks, num_free, N, T, block_tokens,
                             block_table, table_stride, max_blocks, kv_lens, positions, slots,
                             pieces, piece_capacity, counts, device_status,
                             static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_rotary_phases(int32_t rot_dim, double base, int32_t scaling, double factor,
                               double original_length, double fast, double slow,
                               int64_t* phases) {
  if (!phases || rot_dim <= 0) return GDN_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > 256) return GDN_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !(factor >= 1.0) || std::isinf(base) || std::isinf(factor))
    return GDN_ERR_INVALID_ARG;
  if (scaling < GDN_ROTARY_PLAIN || scaling > GDN_ROTARY_BY_PARTS) return GDN_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double lo = 0.0, hi = 0.0;
  if (scaling == GDN_ROTARY_BY_PARTS) {
    if (!(original_length > 0.0) || !(slow > 0.0) || !(fast > slow) || std::isinf(fast) ||
        std::isinf(original_length))
      return GDN_ERR_INVALID_ARG;
    // The pair that turns b times over the original length:
    // base^(-2 i / r) * length = 2 pi b.
    auto pair_of = [&](double b) {
      return rot_dim * std::log(original_length / (kTwoPi * b)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(slow)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == GDN_ROTARY_LINEAR) f /= factor;
    if (scaling == GDN_ROTARY_BY_PARTS) {
      const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    phases[i] = static_cast<int64_t>(static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64)));
  }
  return GDN_OK;
}

gdn_status_t gdn_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const int32_t* positions, const int64_t* phases, void* q_out,
                        int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t T,
                        int32_t Hq, int32_t Hk, int32_t d, int32_t rot_dim, int32_t interleaved,
                        int32_t inverse, float scale, void* stream) {
  if (T < 0 || Hq < 0 || Hk < 0) return GDN_ERR_INVALID_ARG;
  if (!rotary_dim_ok(d)) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)Hq + Hk > 65536) return GDN_ERR_UNSUPPORTED;
  if (T == 0 || Hq + Hk == 0) return GDN_OK;
  gdn_status_t rc =
      check_rotation(positions, phases, d, rot_dim, interleaved, inverse, scale);
  if (rc == GDN_OK && Hq > 0) rc = check_rows(q, q_stride, Hq, d);
  if (rc == GDN_OK && Hq > 0) rc = check_rows(q_out, q_out_stride, Hq, d);
  if (rc == GDN_OK && Hk > 0) rc = check_rows(k, k_stride, Hk, d);
  if (rc == GDN_OK && Hk > 0) rc = check_rows(k_out, k_out_stride, Hk, d);
  if (rc != GDN_OK) return rc;
  if ((Hq > 0 && q == q_out && q_stride != q_out_stride) ||
      (Hk > 0 && k == k_out && k_stride != k_out_stride))
    return GDN_ERR_INVALID_ARG;
  return launch_rotary(q, q_stride, k, k_stride, positions, phases, q_out, q_out_stride, k_out,
                       k_out_stride, T, Hq, Hk, d, rot_dim, scale, interleaved, inverse,
                       static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_rotary_kv_append(const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride,
                                  const int32_t* positions, const int64_t* phases,
                                  const gdn_page_piece_t* pieces, const int32_t* num_pieces,
                                  int32_t piece_capacity, void* q_out, int64_t q_out_stride,
                                  void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                  int32_t num_blocks, int32_t block_tokens, int32_t T, int32_t Hq,
                                  int32_t Hk, int32_t d, int32_t rot_dim, int32_t interleaved,
                                  float scale, void* stream) {
  if (T < 0 || Hq < 0 || Hk <= 0 || num_blocks < 0 || piece_capacity < 0)
    return GDN_ERR_INVALID_ARG;
  if (!cache_dim_ok(d) || !block_tokens_ok(block_tokens)) return GDN_ERR_UNSUPPORTED;
  if (Hq > 65536 || Hk > 65536) return GDN_ERR_UNSUPPORTED;
  if (T == 0) return GDN_OK;
  gdn_status_t rc = check_rotation(positions, phases, d, rot_dim, interleaved, 0, scale);
  if (rc != GDN_OK) return rc;
  const bool with_q = q != nullptr || q_out != nullptr;
  if (with_q != (rot_dim > 0) && rot_dim > 0) return GDN_ERR_INVALID_ARG;
  if (with_q && Hq > 0) {
    if ((rc = check_rows(q, q_stride, Hq, d)) != GDN_OK) return rc;
    if ((rc = check_rows(q_out, q_out_stride, Hq, d)) != GDN_OK) return rc;
    if (q == q_out && q_stride != q_out_stride) return GDN_ERR_INVALID_ARG;
  }
  if ((rc = check_rows(k, k_stride, Hk, d)) != GDN_OK) return rc;
  if ((rc = check_rows(v, v_stride, Hk, d)) != GDN_OK) return rc;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !num_pieces ||
      (piece_capacity > 0 && !pieces))
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned16(pieces) || !aligned(num_pieces, 4))
    return GDN_ERR_ALIGNMENT;
  // Without q: k and v alone. Without rotation q is copied.
  const bool turn_q = with_q && Hq > 0;
  return launch_rotary_kv_append(turn_q ? q : nullptr, q_stride, k, k_stride, v, v_stride,
                                 positions, phases, pieces, num_pieces, piece_capacity, q_out,
                                 q_out_stride, k_cache, v_cache, k_scale, v_scale, num_blocks,
                                 block_tokens, T, Hq, Hk, d, rot_dim, scale, interleaved,
                                 static_cast<cudaStream_t>(stream));
}

size_t gdn_paged_attention_workspace_size(int32_t T, int32_t N, int32_t Hq, int32_t Hk,
                                          int32_t d) {
  if (T < 0 || N < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0 || Hq / Hk > 16 || !cache_dim_ok(d) ||
      N > kMaxCount)
    return 0;
  if ((int64_t)T * (Hq / Hk) > 0x3fffffff || (int64_t)N * Hk > 0x7fffffff) return 0;
  return attn::layout(T, N, Hq, Hk, d).total;
}

gdn_status_t gdn_paged_attention_plan(const int32_t* cu_seqlens, const int32_t* kv_lens,
                                      int32_t N, int32_t T, int32_t Hq, int32_t Hk, int32_t d,
                                      int32_t block_tokens, int32_t max_blocks,
                                      int32_t max_new_tokens, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  bool nothing = false;
  const gdn_status_t rc = check_plan(cu_seqlens, kv_lens, N, T, Hq, Hk, d, block_tokens,
                                     max_blocks, max_new_tokens, workspace, workspace_bytes,
                                     &nothing);
  if (rc != GDN_OK || nothing) return rc;
  return launch_attn_plan(cu_seqlens, kv_lens, N, T, Hq, Hk, d,
                          (int64_t)max_blocks * block_tokens, max_new_tokens, workspace,
                          static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_paged_attention(const void* q, int64_t q_stride, const void* k_cache,
                                 const void* v_cache, const float* k_scale, const float* v_scale,
                                 int32_t num_blocks, int32_t block_tokens,
                                 const int32_t* block_table, int64_t table_stride,
                                 int32_t max_blocks, const int32_t* cu_seqlens,
                                 const int32_t* kv_lens, int32_t N, int32_t T,
                                 int32_t max_new_tokens, void* o, int32_t Hq, int32_t Hk,
                                 int32_t d, float softmax_scale, int32_t flags, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  bool nothing = false;
  if ((flags & ~GDN_FLAG_PLANNED) != 0 || table_stride < max_blocks || num_blocks < 0)
    return GDN_ERR_INVALID_ARG;
  if (!(std::fabs(softmax_scale) <= 3.0e38f)) return GDN_ERR_INVALID_ARG;
  if (Hk > 0 && (int64_t)num_blocks * Hk >= 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  gdn_status_t rc = check_plan(cu_seqlens, kv_lens, N, T, Hq, Hk, d, block_tokens, max_blocks,
                               max_new_tokens, workspace, workspace_bytes, &nothing);
  if (rc != GDN_OK || nothing) return rc;
  if ((rc = check_rows(q, q_stride, Hq, d)) != GDN_OK) return rc;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !o || (max_blocks > 0 && !block_table))
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(block_table, 4))
    return GDN_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool self_plan = (flags & GDN_FLAG_PLANNED) == 0 && attn::self_planned(
                                                              N, T, Hq / Hk, Hk, max_new_tokens,
                                                              (int64_t)max_blocks * block_tokens);
  if ((flags & GDN_FLAG_PLANNED) == 0 && !self_plan) {
    rc = launch_attn_plan(cu_seqlens, kv_lens, N, T, Hq, Hk, d,
                          (int64_t)max_blocks * block_tokens, max_new_tokens, workspace, st);
    if (rc != GDN_OK) return rc;
  }
  const attn::Layout l = attn::layout(T, N, Hq, Hk, d);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  attn::Args a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = k_scale;
  a.vs = v_scale;
  a.table = block_table;
  a.table_stride = table_stride;
  a.cu = cu_seqlens;
  a.kv = kv_lens;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.N = N;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.d = d;
  a.log_b = __builtin_ctz((unsigned)block_tokens);
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.items = reinterpret_cast<attn::Item*>(ws + l.items);
  a.partials = reinterpret_cast<float*>(ws + l.partials);
  a.tiles = reinterpret_cast<attn::Item*>(ws + l.tiles);
  a.sorted_tiles = reinterpret_cast<attn::Item*>(ws + l.sorted_tiles);
  a.self_plan = self_plan ? 1 : 0;
  // A plan in the workspace stays as it is.
  a.starts = reinterpret_cast<attn::Start*>(ws + (self_plan ? l.self_starts : l.starts));
  a.tile_starts = reinterpret_cast<const attn::Start*>(ws + l.tile_starts);
  a.split_rows = l.split_rows;
  a.split_grid = attn::split_grid(d, l.split_rows);
  a.tile_grid = attn::tile_grid();
  a.tile_partials = reinterpret_cast<float*>(ws + l.tile_partials);
  // The two kernels share a step's sequences by their rows; a step whose
  // lengths rule one of them out launches the other alone.
  const attn::Kernels use =
      attn::kernels_of(N, T, Hq / Hk, Hk, max_new_tokens, (int64_t)max_blocks * block_tokens);
  a.after_split = use.split ? 1 : 0;
  if (use.split) rc = launch_attn_split(a, st);
  if (rc == GDN_OK && use.tile) rc = launch_attn_tile(a, st);
  return rc == GDN_OK ? launch_attn_join(a, use.split, use.tile, st) : rc;
}

}  // extern "C"
