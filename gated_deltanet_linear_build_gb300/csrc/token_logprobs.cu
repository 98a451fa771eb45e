// Log probabilities of given tokens, entropy, ranks and the best tokens, from logits.
//
// With z = logit / temperature, m = max z and R = the sum of e^(z - m) over all tokens
// but one of the largest:
//   log p(i) = (z_i - m) - log1p(R),   H = log1p(R) - sum (z - m) e^(z - m) / (1 + R).
// The largest one is left out of the sum, so that a probability next to 1 keeps its
// distance from it. The order is by logit, then by index: a key of 64 bits.
//
// Bound: each logit is read once, for seven instructions or so (an exponential, a sum, a
// weighted sum, a maximum, a comparison), so HBM bounds it where there are many rows, FP32
// logits more than BF16 ones, and latency where there are few. One pass: a warp keeps a
// maximum, a thread the sum of what is below it, how many are equal to it and the weighted
// sum, rescaled when the maximum grows; only rounds with a new maximum or one equal to it
// look at equality. A row is one CTA's, or shared by a cluster of up to eight whose results
// meet in the first one's shared memory; four CTAs are resident.
//   2,048 x 131,072 FP32, eight best 184 us (5.8 TB/s; none: 164), BF16, twenty best 124
//   (4.3 TB/s; none: 102); 32 x 131,072 12.2; 333 x 50,001 BF16 15.8; 1 x 200,003 BF16,
//   twenty best 11.2; 32 x 4,096 6.4.
//
// The best k: a thread notes but the largest logit of each round (16 or 32 logits of its
// own), or of a few, in shared memory. At the end the k-th largest of the maxima of 64
// groups of lanes is a threshold that k tokens reach. The notes that reach it name what is
// read again, some tens of vectors, and what reaches it of that goes to a list, of which
// the best k stay. Where the list runs over (many equal logits, or all large ones in a few
// lanes), the threshold is raised by a closer look and the vectors are read once more.
//
// Rows with a NaN or +inf, which have no probabilities, get their order by keys alone.
#include <algorithm>
#include <type_traits>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kResident = 4;             // CTAs of an SM
constexpr int kMaxTop = 32;
constexpr int kList = 1024;            // candidates
constexpr int kGroups = 64;            // of lanes
constexpr int kNotes = 16;             // a thread
constexpr int kLanes = kThreads / kGroups;
constexpr int kMaxCluster = 8;

// 32 bits in the order of the values; -0 is 0, NaN below all.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (isnan(v)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, int i) { return ((uint64_t)ordered(v) << 32) | (uint32_t)~i; }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }

// What has been seen of a row: with d = x - m (logits), r the sum of e^d over d < 0 and
// n the number of d = 0, w the sum of d e^d.
struct Sums {
  float m, r, w;
  int n;
};
// a as seen from a larger maximum m. (c: log2 e / temperature.)
__device__ __forceinline__ Sums seen_from(const Sums& a, float m, float c) {
  if (a.m == m) return a;
  const float s = a.r + (float)a.n;
  if (s == 0.f) return {m, a.r, a.w, 0};                       // nothing yet (or NaN: kept)
  const float d = fmaxf(a.m - m, -1e30f), f = ex2_approx(d * c);
  return {m, s * f, f == 0.f ? a.w * 0.f : f * fmaf(d, s, a.w), 0};   // (NaN stays)
}
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const Sums x = seen_from(a, m, c), y = seen_from(b, m, c);
  return {m, x.r + y.r, x.w + y.w, x.n + y.n};
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename In>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4, per_round = 4;    // per_round: vectors a thread and round
  __device__ static void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  // Largest of `count` vectors (NaN left out).
  template <int count>
  __device__ static float top(const uint4 (&v)[count]) {
    float m = __uint_as_float(v[0].x);
#pragma unroll
    for (int i = 0; i < count; ++i) {
      float x[4];
      unpack(v[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, x[j]);
    }
    return m;
  }
  // Not below the type's lowest number (NaN stays).
  __device__ static uint4 finite(uint4 v) {
    auto one = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), -3.402823466e38f)); };
    return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
  }
  // How many are larger than `mark` (a value of the type), or smaller.
  template <bool larger, int count>
  __device__ static float passing(const uint4 (&v)[count], float mark) {
    float2 n = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < count; ++i) {
      float x[4], one[4];
      unpack(v[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (larger) asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(one[j]) : "f"(x[j]), "f"(mark));
        else asm("set.lt.f32.f32 %0, %1, %2;" : "=f"(one[j]) : "f"(x[j]), "f"(mark));
      }
      n = add2(n, add2(make_float2(one[0], one[1]), make_float2(one[2], one[3])));
    }
    return n.x + n.y;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8, per_round = 4;
  __device__ static void unpack(const uint4& v, float* x) { unpack8(v, x); }
  template <int count>
  __device__ static float top(const uint4 (&v)[count]) {
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m = two(v[0].x);
#pragma unroll
    for (int i = 0; i < count; ++i)
      m = __hmax2(__hmax2(__hmax2(m, two(v[i].x)), __hmax2(two(v[i].y), two(v[i].z))), two(v[i].w));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ static uint4 finite(uint4 v) {
    auto two = [](uint32_t& w) {
      __nv_bfloat162& x = *reinterpret_cast<__nv_bfloat162*>(&w);
      x = __hmax2_nan(x, __float2bfloat162_rn(-3.38953139e38f));
    };
    two(v.x), two(v.y), two(v.z), two(v.w);
    return v;
  }
  template <bool larger, int count>
  __device__ static float passing(const uint4 (&v)[count], float mark) {
    const __nv_bfloat162 m = __float2bfloat162_rn(mark);
    auto two = [&](uint32_t w) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
      return larger ? __hgt2(x, m) : __hlt2(x, m);
    };
    __nv_bfloat162 n = __float2bfloat162_rn(0.f);            // (some tens at most)
#pragma unroll
    for (int i = 0; i < count; ++i)
      n = __hadd2(n, __hadd2(__hadd2(two(v[i].x), two(v[i].y)), __hadd2(two(v[i].z), two(v[i].w))));
    return __low2float(n) + __high2float(n);
  }
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// What a row's sums say. (none: a NaN or +inf in it; masked: -inf all over.)
struct Row {
  float m, lse, temperature, entropy;
  bool none, masked;
  __device__ __forceinline__ Row(const Sums& s, float temperature)
      : m(s.m), temperature(temperature), none(isnan(s.w)), masked(s.n == 0 && s.r == 0.f) {
    const float R = s.r + (float)(s.n - 1);                  // m is the row's largest, once left out
    lse = masked ? 0.f : log1pf(R);
    entropy = none ? NAN : masked ? 0.f : lse - s.w / temperature / (1.f + R);
  }
  __device__ __forceinline__ float logprob(float v) const {
    return none ? NAN : masked || v == -INFINITY ? -INFINITY : (v - m) / temperature - lse;
  }
};

struct Args {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float *logprobs, *entropy;
  int32_t *ranks, *top_ids;
  float* top_logprobs;
  int V, k;
  float temperature;
};

// What a CTA hands to the first of its cluster.
struct Part {
  Sums s;
  int before;                          // tokens that stand before the given one
  uint64_t top[kMaxTop];
};

// Shared memory of the search for the best.
struct Search {
  uint64_t list[kList];
  uint64_t group[kGroups];
  uint64_t threshold;
  int count;                             // entries of the list
  uint32_t notes[kWarps][kNotes][32];    // the largest logits (as floats); what passed
};

// How many of the n <= 2 kGroups keys at `list` stand above key i (equal ones by their
// place), by neighbouring lanes together; i is the thread's, -1 for none.
__device__ __forceinline__ int count_above(const uint64_t* list, int n, int* i) {
  const int lanes = n > kGroups ? kThreads / kGroups / 2 : kThreads / kGroups;
  const int mine = threadIdx.x / lanes, part = threadIdx.x % lanes;
  const uint64_t key = mine < n ? list[mine] : ~0ull;
  int above = 0;
#pragma unroll 8
  for (int j = part; j < n; j += lanes) {
    const uint64_t other = list[j];
    above += other > key || (other == key && j < mine);
  }
  for (int d = 1; d < lanes; d <<= 1) above += __shfl_xor_sync(0xffffffffu, above, d);
  *i = part == 0 && mine < n ? mine : -1;
  return above;
}

// The k-th largest of the groups' maxima (0: less than k are not 0). All threads. (kUser:
// rows without probabilities have copies of their own. With one for both the kernel's calls
// became longer: 1 x 200,003, twenty best, 11.2 -> 11.7 us.)
template <int kUser>
__device__ __noinline__ uint64_t group_threshold(Search& s, uint64_t mine, int k) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, d));
  if (tid % kLanes == 0) s.group[tid / kLanes] = mine;
  __syncthreads();
  int i;
  const int above = count_above(s.group, kGroups, &i);
  if (i >= 0 && above == k - 1) s.threshold = s.group[i];
  __syncthreads();
  return s.threshold;
}

// The k largest of the first n entries of the list, to its front in their order; the
// rest of the first k places is 0. All threads; n is cut off at the list's length.
template <int kUser>
__device__ __noinline__ void keep_best(Search& s, int n, int k) {
  const int tid = threadIdx.x;
  constexpr int kEach = kList / kThreads;
  n = min(n, kList);
  __syncthreads();
  // Fewer first: what reaches the k-th of the groups' maxima. (Entries are dealt to the
  // groups in turn, two each at least; those of the other groups fall out.)
  while (n > 2 * kGroups) {
    uint64_t mine[kEach], most = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = tid / kLanes + kGroups * (tid % kLanes + kLanes * j);
      mine[j] = i < n ? s.list[i] : 0;
      most = max(most, mine[j]);
    }
    const uint64_t t = group_threshold<kUser>(s, most, k);
    if (tid == 0) s.count = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (mine[j] > 0 && mine[j] >= t) s.list[atomicAdd(&s.count, 1)] = mine[j];
    __syncthreads();
    n = s.count;
    __syncthreads();
  }
  int i;
  const int above = count_above(s.list, n, &i);
  const uint64_t mine = i >= 0 ? s.list[i] : 0;
  __syncthreads();
  if (tid < k) s.list[tid] = 0;
  __syncthreads();
  if (i >= 0 && above < k) s.list[above] = mine;
  __syncthreads();
}

// A CTA's part of a row: vectors v0 to v1, of 16 bytes from the boundary before the row.
template <typename In>
struct RowPart {
  static constexpr int n = Vec<In>::n;
  const In* row;
  int V, first, v0, v1;                  // first: element of vector 0
  // Vector v, what is outside the row as -inf.
  __device__ __forceinline__ uint4 load(int v) const {
    const int e = v * n + first;
    if (e >= 0 && e + n <= V) return load_stream(row + e);
    union {
      uint4 u;
      In x[n];
    } a;
#pragma unroll
    for (int j = 0; j < n; ++j) a.x[j] = e + j >= 0 && e + j < V ? row[e + j] : (In)-INFINITY;
    return a.u;
  }
};

// The part's candidates to the list: its best k are among them. All threads; a note is of
// 2^shift rounds.
template <typename In>
__device__ __forceinline__ void find_candidates(Search& s, const RowPart<In>& part, int rounds, int shift, int k) {
  constexpr int VE = Vec<In>::n, kVecs = Vec<In>::per_round, kVecsLog = kVecs == 4 ? 2 : 1;
  static_assert(kVecs == 1 << kVecsLog, "vectors of a round");
  const int tid = threadIdx.x, lane = tid & 31, slots = (rounds + (1 << shift) - 1) >> shift;
  uint32_t* const notes = &s.notes[tid / 32][0][0];
  float most = -INFINITY;
  for (int r = 0; r < slots; ++r) most = fmaxf(most, __uint_as_float(notes[r * 32 + lane]));
  uint64_t threshold = group_threshold<0>(s, (uint64_t)ordered(most) << 32, k);
  // The warp's own notes that pass: slot * 32 + lane, from the notes' front.
  int n = 0;
  for (int r = 0; r < slots; ++r) {
    const bool again = ordered(__uint_as_float(notes[r * 32 + lane])) >= (uint32_t)(threshold >> 32);
    const uint32_t mask = __ballot_sync(0xffffffffu, again);
    if (again) notes[n + __popc(mask & ((1u << lane) - 1))] = r * 32 + lane;
    n += __popc(mask);
    __syncwarp();
  }
  // f(key) for the logits that reach the threshold.
  const int log = kVecsLog + shift;                          // vectors of a note
  const int64_t vectors = (int64_t)n << log;
  auto each = [&](auto f) {
    const float least = value_of((uint32_t)(threshold >> 32));     // (NaN: all do)
#pragma unroll 1
    for (int64_t i = lane; i < vectors; i += 4 * 32) {
      int v[4];
      uint4 of[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = i + j * 32;
        v[j] = part.v1;
        if (at < vectors) {
          const uint32_t note = notes[at >> log];
          const int64_t u = part.v0 + ((((int64_t)(note / 32) << log) + (at & ((1 << log) - 1))) * kThreads) +
                            (tid & ~31) + (int)(note % 32);
          v[j] = (int)min(u, (int64_t)part.v1);
        }
        if (v[j] < part.v1) of[j] = part.load(v[j]);
      }
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        if (v[0] < part.v1) {
          float x[VE];
          Vec<In>::unpack(of[0], x);
#pragma unroll
          for (int h = 0; h < VE; ++h) {
            const int e = v[0] * VE + part.first + h;
            if (!(x[h] < least) && e >= 0 && e < part.V) {
              const uint64_t key = key_of(x[h], e);
              if (key >= threshold) f(key);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 3; ++h) v[h] = v[h + 1], of[h] = of[h + 1];
      }
    }
  };
  for (int time = 0;; ++time) {
    if (tid == 0) s.count = 0;
    __syncthreads();
    each([&](uint64_t key) {
      const int at = atomicAdd(&s.count, 1);
      if (at < kList) s.list[at] = key;
    });
    __syncthreads();
    if (s.count <= kList) break;
    // It has run over. What k of these vectors' logits reach is a better threshold, and
    // the next time what k of the list's do, which leaves out half of it at least.
    uint64_t best = 0;
    if (time == 0) {
      each([&](uint64_t key) { best = max(best, key); });
    } else {
      for (int i = tid; i < kList; i += kThreads) best = max(best, s.list[i]);
    }
    threshold = max(threshold, group_threshold<0>(s, best, k));
  }
}

// f(key) for all of a row's logits, by one CTA: four vectors of a thread on their way.
template <typename In, typename F>
__device__ __forceinline__ void each_key(const RowPart<In>& row, F f) {
  constexpr int VE = Vec<In>::n;
#pragma unroll 1
  for (int v = row.v0 + threadIdx.x; v < row.v1; v += 4 * kThreads) {
    uint4 of[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v + j * kThreads < row.v1) of[j] = row.load(v + j * kThreads);
#pragma unroll 1
    for (int j = 0; j < 4 && v + j * kThreads < row.v1; ++j) {
      float x[VE];
      Vec<In>::unpack(of[0], x);
#pragma unroll
      for (int h = 0; h < VE; ++h) {
        const int e = (v + j * kThreads) * VE + row.first + h;
        if (e >= 0 && e < row.V) f(key_of(x[h], e));
      }
#pragma unroll
      for (int h = 0; h < 3; ++h) of[h] = of[h + 1];
    }
  }
}

// The order of a row by keys alone, for one CTA: the best k to the list's front, the rank
// of the given token. Two passes: the threads' largest keys and what stands before the
// token, then what reaches the k-th of the groups' largest. (A call with such a row of
// 200,003, twenty best: 118 us, without it 12; of 2^26, 32 best: 38 ms. By a pass for each
// of the best 772 us and 564 ms.)
template <typename In>
__device__ __noinline__ void by_keys(const In* logits, int V, int k, Search& s, int token, int* rank) {
  const int tid = threadIdx.x;
  const int off = (int)((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(In));
  const RowPart<In> row = {logits, V, -off, 0, (int)(((int64_t)V + off + Vec<In>::n - 1) / Vec<In>::n)};
  const uint64_t mine = token >= 0 ? key_of((float)logits[token], token) : ~0ull;
  uint64_t best = 0;
  int before = 0;
  each_key(row, [&](uint64_t key) {
    best = max(best, key);
    before += key > mine;
  });
  before = __reduce_add_sync(0xffffffffu, before);
  __syncthreads();
  if (tid == 0) *rank = 0;
  __syncthreads();
  if (tid % 32 == 0) atomicAdd(rank, before);
  uint64_t threshold = 0;
  while (k > 0) {
    threshold = max(threshold, group_threshold<1>(s, best, k));
    if (tid == 0) s.count = 0;
    __syncthreads();
    each_key(row, [&](uint64_t key) {
      if (key < threshold) return;
      const int at = atomicAdd(&s.count, 1);
      if (at < kList) s.list[at] = key;
    });
    __syncthreads();
    if (s.count <= kList) break;
    // It has run over: what k of the list's keys reach leaves out half of it at least.
    best = 0;
    for (int i = tid; i < kList; i += kThreads) best = max(best, s.list[i]);
  }
  if (k > 0) keep_best<1>(s, s.count, k);
  __syncthreads();
}

template <typename In, bool kTop>
__global__ void __launch_bounds__(kThreads, kResident) token_logprobs_kernel(const __grid_constant__ Args p) {
  constexpr int VE = Vec<In>::n, kVecs = Vec<In>::per_round, kRound = kThreads * kVecs;
  __shared__ Search s_search;
  __shared__ Part s_part[kMaxCluster];
  __shared__ Sums s_sums[kWarps];
  __shared__ int s_before[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, C;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int t = blockIdx.x / C;
  const In* row = static_cast<const In*>(p.logits) + (int64_t)t * p.stride;
  // 16-byte vectors from the boundary before the row; elements outside count as -inf.
  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(In));
  const int vecs = (int)(((int64_t)p.V + off + VE - 1) / VE);
  const int v0 = (int)((int64_t)vecs * rank / C), v1 = (int)((int64_t)vecs * (rank + 1) / C);
  const int first = -off;                // element of vector 0
  const RowPart<In> in = {row, p.V, first, v0, v1};
  const float c = 1.4426950408889634f / p.temperature;
  // (That all CTAs of the cluster have begun is asked for where one writes to another.)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  const int rounds = (v1 - v0 + kRound - 1) / kRound;
  int shift = 0;                         // a note is of 2^shift rounds
  while (kTop && kNotes << shift < rounds) ++shift;
  // Rounds begun to full hold neither the row's first vector nor the part's last.
  const int begun = v0 == 0, full = (v1 - 1 - v0) / kRound;
  const uint4* const mine = reinterpret_cast<const uint4*>(row + first) + (v0 + tid);
  const uint32_t minus = sizeof(In) == 4 ? 0xff800000u : 0xff80ff80u;
  auto fetch = [&](int round, uint4 (&to)[kVecs]) {
    if (round >= begun && round < full) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) to[j] = load_stream(mine + (round * kRound + j * kThreads));
      return;
    }
    const int v = v0 + round * kRound + tid;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      to[j] = make_uint4(minus, minus, minus, minus);
      const int w = v + j * kThreads;
      if (w > 0 && w < v1 - 1) to[j] = load_stream(mine + (round * kRound + j * kThreads));
    }
    const int last = v1 - 1 - v;
    if (v == 0 || (last >= 0 && last < kRound && last % kThreads == 0)) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (v + j * kThreads == 0 || last == j * kThreads) to[j] = in.load(v + j * kThreads);
    }
  };
  uint4 next[kVecs];
  fetch(0, next);
  const int token = p.tokens ? __ldg(p.tokens + t) : -1;
  const bool given = token >= 0 && token < p.V;
  const float mark = given ? (float)row[token] : 0.f;
  // Rounds up to `upto` lie before the given token, from `after` on behind it.
  const int held = (token - first) / VE - v0;                // its vector
  const int upto = min(held < 0 ? 0 : held / kRound, full), after = held < 0 ? 0 : held / kRound + 1;
  // The warp's maximum and the thread's sums; how many stand before the given token (below
  // 2^24; those before it in the row that are smaller count less one); what the warp's
  // logits stay below where nothing needs a closer look.
  Sums s = {-3.402823466e38f, 0.f, 0.f, 0};
  float before = 0.f, below = -INFINITY, noted = 0.f;
#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    uint4 cur[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) cur[j] = next[j];
    if (round + 1 < rounds) fetch(round + 1, next);
    const float top = Vec<In>::top(cur);
    if constexpr (kTop) {
      noted = (round & ((1 << shift) - 1)) == 0 ? top : fmaxf(noted, top);
      s_search.notes[warp][round >> shift][lane] = __float_as_uint(noted);
    }
    const bool closer = __any_sync(0xffffffffu, !(top < below));
    if (closer) {
      // The warp's maximum. (By its order as a whole number: one instruction.)
      const float m = fmaxf(s.m, value_of(__reduce_max_sync(0xffffffffu, ordered(top))));
      if (m > s.m) s = seen_from(s, m, c);
      below = fabsf(m) < 1e30f ? m : -INFINITY;
    }
    // Two at a time. Where the maximum itself is among the warp's, what equals it is counted
    // instead of summed. (-inf acts as the lowest number, or as a distance of 1e30 where
    // that could be near the maximum.)
    auto add = [&](auto closely) {
      float2 r = make_float2(0.f, 0.f), w = r;
      const float2 minus_m = make_float2(-s.m, -s.m), cc = make_float2(c, c);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float x[VE];
        Vec<In>::unpack(closely.value ? cur[j] : Vec<In>::finite(cur[j]), x);
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          float2 d = add2(make_float2(x[i], x[i + 1]), minus_m);
          if (closely.value) d = make_float2(max_nan(d.x, -1e30f), max_nan(d.y, -1e30f));
          const float2 z = mul2(d, cc);
          float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
          if (closely.value) {
            if (d.x == 0.f) ++s.n, e.x = 0.f;
            if (d.y == 0.f) ++s.n, e.y = 0.f;
          }
          r = add2(r, e);
          w = fma2(d, e, w);
        }
      }
      s.r += r.x + r.y;
      s.w += w.x + w.y;
    };
    if (closer)
      add(std::true_type());
    else
      add(std::false_type());
    // Before the given token those count that are not smaller, behind it the larger ones.
    if (given) {
      if (round >= after) {                                  // (-inf behind the part's end)
        before += Vec<In>::template passing<true>(cur, mark);
      } else if (round < upto) {
        before -= Vec<In>::template passing<false>(cur, mark);
      } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const int v = v0 + (round * kVecs + j) * kThreads + tid, e = v * VE + first;
          float x[VE];
          Vec<In>::unpack(cur[j], x);
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (v < v1) before += e + i < token ? -(float)(x[i] < mark) : (float)(x[i] > mark);
        }
      }
    }
  }
  // The warps' sums, by the first.
  bool bad = !(s.w <= 0.f);              // NaN
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    // (One maximum for all lanes.)
    s.r += __shfl_xor_sync(0xffffffffu, s.r, d);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, d);
  }
  s.n = __reduce_add_sync(0xffffffffu, s.n);
  const int n = __reduce_add_sync(0xffffffffu, (int)before);
  if (lane == 0) s_sums[warp] = s, s_before[warp] = n;
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  bad = __syncthreads_or(bad);
  Part* part = &s_part[0];
  if constexpr (kTop) {
    find_candidates(s_search, in, rounds, shift, p.k);
    keep_best<0>(s_search, s_search.count, p.k);
  }
  if (warp == 0) {
    Sums all = lane < kWarps ? s_sums[lane] : s_sums[0];
    if (lane >= kWarps) all.r = all.w = 0.f, all.n = 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const Sums o = {__shfl_xor_sync(0xffffffffu, all.m, d), __shfl_xor_sync(0xffffffffu, all.r, d),
                      __shfl_xor_sync(0xffffffffu, all.w, d), __shfl_xor_sync(0xffffffffu, all.n, d)};
      all = joined(all, o, c);
    }
    if (bad) all.w = NAN;
    const int stand = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_before[lane] : 0);
    // To the first CTA of the cluster.
    if (C > 1) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(&s_part[rank])), "r"(0));
      auto put = [&](uint32_t o, uint32_t v) {
        asm volatile("st.shared::cluster.b32 [%0], %1;" :: "r"(at + o), "r"(v) : "memory");
      };
      if (lane == 0) {
        put(0, __float_as_uint(all.m));
        put(4, __float_as_uint(all.r));
        put(8, __float_as_uint(all.w));
        put(12, (uint32_t)all.n);
        put(16, (uint32_t)stand);
      }
      if (kTop && lane < p.k) {
        put(24 + lane * 8, (uint32_t)s_search.list[lane]);
        put(28 + lane * 8, (uint32_t)(s_search.list[lane] >> 32));
      }
    } else if (lane == 0) {
      part->s = all;
      part->before = stand;
    }
  }
  __syncwarp();
  if (C > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    if (kTop) {
      for (int i = tid; i < (int)C * p.k; i += kThreads) s_search.list[i] = s_part[i / p.k].top[i % p.k];
      int n = 0;                         // (A part with less than k tokens has zeros behind them.)
      __syncthreads();
      n = (int)C * p.k;
      keep_best<0>(s_search, n, p.k);
    }
    if (tid == 0)
      for (int q = 1; q < (int)C; ++q) {
        const bool nan = isnan(part->s.w) || isnan(s_part[q].s.w);
        part->s = joined(part->s, s_part[q].s, c);
        if (nan) part->s.w = NAN;
        part->before += s_part[q].before;
      }
  }
  __syncthreads();
  const Sums all = part->s;
  const bool none = isnan(all.w);
  int place = given ? part->before + token + (mark == -INFINITY ? 0 : off) : -1;
  if (none && (kTop || given)) {
    by_keys(row, p.V, p.k, s_search, given ? token : -1, s_before);
    if (given) place = s_before[0];
  }
  const Row of(all, p.temperature);
  if (tid == 0) {
    if (p.logprobs) p.logprobs[t] = given ? of.logprob(mark) : NAN;
    if (p.ranks) p.ranks[t] = place;
    if (p.entropy) p.entropy[t] = of.entropy;
  }
  if (kTop && tid < p.k) {
    const uint64_t key = s_search.list[tid];
    p.top_ids[(int64_t)t * p.k + tid] = index_of(key);
    p.top_logprobs[(int64_t)t * p.k + tid] = of.logprob(value_of((uint32_t)(key >> 32)));
  }
}

// ---------------------------------------------------------------------------
// Short rows (up to 1,024): a warp each, all of it in registers. The best k are taken one
// by one, the largest of the lanes' largest; all orders are by keys, in rows with a NaN too.
// (3,284 x 182, 32 best: 12.3 us, by a CTA a row 80.)
// ---------------------------------------------------------------------------
constexpr int kShortWarps = 4;
template <typename In, int kPer>
__global__ void __launch_bounds__(kShortWarps * 32) short_logprobs_kernel(const __grid_constant__ Args p, int T) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kShortWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const In* row = static_cast<const In*>(p.logits) + t * p.stride;
  float x[kPer];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) x[j] = j * 32 + lane < p.V ? (float)row[j * 32 + lane] : -INFINITY;
  const int token = p.tokens ? __ldg(p.tokens + t) : -1;
  const bool given = token >= 0 && token < p.V;
  const float mark = given ? (float)row[token] : 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) top = fmaxf(top, x[j]);
  const float c = 1.4426950408889634f / p.temperature;
  Sums s = {fmaxf(-3.402823466e38f, value_of(__reduce_max_sync(0xffffffffu, ordered(top)))), 0.f, 0.f, 0};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float d = max_nan(x[j] - s.m, -1e30f), e = ex2_approx(d * c);
    s.w = fmaf(d, e, s.w);
    if (d == 0.f) ++s.n;
    else s.r += e;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s.r += __shfl_xor_sync(0xffffffffu, s.r, d);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, d);
  }
  s.n = __reduce_add_sync(0xffffffffu, s.n);
  const Row of(s, p.temperature);
  // From here on in the order of the keys: 0 behind the row's end.
  uint32_t o[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = j * 32 + lane < p.V ? ordered(x[j]) + 1 : 0;
  if (given) {
    const uint32_t m = ordered(mark) + 1;
    int before = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) before += o[j] > m || (o[j] == m && j * 32 + lane < token);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0 && p.ranks) p.ranks[t] = before;
  } else if (lane == 0 && p.ranks) {
    p.ranks[t] = -1;
  }
  if (lane == 0) {
    if (p.logprobs) p.logprobs[t] = given ? of.logprob(mark) : NAN;
    if (p.entropy) p.entropy[t] = of.entropy;
  }
  int id = 0;
  float value = 0.f;
#pragma unroll 1
  for (int k = 0; k < p.k; ++k) {
    uint32_t most = o[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < kPer; ++j)
      if (o[j] > most) most = o[j], at = j;
    const uint32_t best = __reduce_max_sync(0xffffffffu, most);
    const uint32_t who = __reduce_min_sync(0xffffffffu, most == best ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
    if (lane == k) id = (int)who, value = value_of(best - 1);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (who == (uint32_t)(j * 32 + lane)) o[j] = 0;
  }
  if (lane < p.k) {
    p.top_ids[t * p.k + lane] = id;
    p.top_logprobs[t * p.k + lane] = of.logprob(value);
  }
}

template <typename In, int kPer>
gdn_status_t launch_short(const Args& a, int T, cudaStream_t st) {
  return check_launch(launch_pdl(short_logprobs_kernel<In, kPer>, dim3((unsigned)(((int64_t)T + kShortWarps - 1) / kShortWarps)),
                                 dim3(kShortWarps * 32), 0, st, a, T));
}

// Shared memory with which `each` CTAs go to an SM and one more does not. (28 KB: the
// kernel's own, about.)
constexpr int apart(int each) { return (228 * 1024 / (each + 1) + 228 * 1024 / each) / 2 - 28 * 1024; }

template <typename In>
gdn_status_t launch(const Args& a, int T, cudaStream_t st) {
  if (a.V <= 256) return launch_short<In, 8>(a, T, st);
  if (a.V <= 1024) return launch_short<In, 32>(a, T, st);
  auto kernel = a.k > 0 ? token_logprobs_kernel<In, true> : token_logprobs_kernel<In, false>;
  // CTAs a row: as many as are resident at a time, with a round each at least. (Twice as
  // many: 400 x 131,072 45 -> 53 us.)
  const int64_t round = (int64_t)kThreads * Vec<In>::per_round * Vec<In>::n;
  const int sms = num_sms();
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)T * cluster * 2 <= kResident * sms && a.V >= 2 * cluster * round) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(T * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  // Where fewer fit them all, no more go to one SM: shared memory that nobody uses keeps
  // them apart. (333 x 50,001 in BF16: 18.2 -> 15.8 us; clusters are spread as it is, and lose
  // by it: 32 x 131,072 12.2 -> 16.1.)
  const int64_t each = ((int64_t)T + sms - 1) / sms;
  if (cluster == 1 && each < kResident) {
    static DeviceOnce once[2];
    const cudaError_t set = allow_smem(once[a.k > 0], kernel, apart(1));
    if (set != cudaSuccess) return check_launch(set);
    cfg.dynamicSmemBytes = apart((int)each);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return check_launch(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace

gdn_status_t launch_token_logprobs(const void* logits, int64_t stride, int32_t type, const int32_t* tokens,
                                   float* logprobs, float* entropy, int32_t* ranks, int32_t* top_ids,
                                   float* top_logprobs, int32_t T, int32_t V, int32_t k, float temperature,
                                   cudaStream_t st) {
  const Args a = {logits, stride, tokens, logprobs, entropy, ranks, top_ids, top_logprobs, V, k, temperature};
  return type == GDN_TYPE_F32 ? launch<float>(a, T, st) : launch<__nv_bfloat16>(a, T, st);
}

}  // namespace gdn
