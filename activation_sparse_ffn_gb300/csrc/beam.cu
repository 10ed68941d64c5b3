// The best continuations over beams and vocabulary.
//
// k_beam_rows reads every logit once: a block takes a part of one row, a chunk
// at a time with the next on its way, sums the exponentials and keeps the n_out
// best so far. k_beam_merge, a block for each search, joins the sums of a row,
// turns the kept logits into totals and picks the n_out best of those.
//
// Sums of exponentials. exp(z) = 2^(z log2 e); the reference that a thread takes
// off is a whole number R near its largest z log2 e, so that sums are brought
// together by powers of two, exactly. log2 e rounded to a float is off by 2^-26
// of itself, which a logit of 20 makes 2^-21; what the rounding left is put right
// for the part's largest z at the end, by one product. Above |z| = 2^22 a
// whole number no longer lies near enough: such a part is summed again, its
// largest z the reference. A thread adds up a chunk's terms in a tree and the chunks
// with what each addition rounds off (one running sum of a vocabulary of 2^20 was off
// by 2^-16), so that a sum has at most 17 roundings: 5 + 2 of a thread, 2 of its
// pair, 8 of the block.
//
// The n_out best. A bound that at least n_out elements of the first chunk reach,
// and few others: the ceil(n_out / 8)-th largest of the lanes' own maxima, in
// each of eight warps, and the least of those over the warps. What reaches it
// goes to a list, of every chunk, with no barrier between them. At the end the
// same is done with the list, and each of the few that are left counts those
// ahead of it. (Keeping the n_out best in order after every chunk took 40 us of
// 32 x 8 rows of 131072 bf16 logits, most of it at barriers.) Where too many
// reach the bound for the list, a search over all bits and then over indices,
// which reads the logits again, takes exactly the first of them.
//
// Measured: 32 x 8 rows of 131072 bf16 logits 28 us and the merge, 29 us of a graph back to back;
// 14 instructions a logit, 55% of the issue slots busy, the exponentials' unit a quarter of
// the time. Four rows of 32000, one alive, 11 us: two launches and their dependent reads.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "rows_io.cuh"
#include "step.h"

namespace sffn {

namespace {

constexpr int kThreads = 256;
constexpr int kMergeThreads = 512;
constexpr int kMaxOut = 64;
constexpr int kMaxBeams = 64;
constexpr int kList = 2048;
constexpr int kRuns = 4;      // times 16 bytes of a chunk that a thread holds, and as many on their way
constexpr int kRowBlocks = 4; // of an SM
constexpr int kSteps = 256;   // of 1/16 below the largest total
constexpr int kKept = 4;      // candidates that a thread of k_beam_merge holds
constexpr int kTighten = 512; // entries of the list that raise the bound: four chunks add some 500 at most, of random logits
constexpr int kMerged = 4096; // candidates of a search for which parts of a row are cut
constexpr int kRanked = 256;  // entries that are put in order by counting

struct BeamArgs {
  sffn_rows logits;
  const float* scores;
  const uint8_t* done;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  uint32_t* err;
  // workspace: sums of each row's chunks, and their candidates
  float4* sums;    // [rows][parts]: reference, sum, mode, largest logit
  int2* found;     // [rows][parts][n_out]: logit, token; token -1: none
  int vocab, beams, n_out, batch, end_token, dtype, parts, chunks;   // parts of a row, chunks of one
  bool vec;
};

// Patterns that order like the numbers (NaN aside).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// The number of a pattern.
__device__ __forceinline__ double number(unsigned long long o) {
  return __longlong_as_double(o >> 63 ? o ^ 1ull << 63 : ~o);
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  const unsigned long long u = __double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// The number of a pattern.
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
template <typename T>
__device__ __forceinline__ float lowest() {   // finite
  return sizeof(T) == 4 ? -3.402823466e38f : std::is_same<T, __half>::value ? -65504.f : -3.3895313892515355e38f;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^d of a whole number d up to 0; 0 far below it.
__device__ __forceinline__ float power_of_two(float d) {
  return d < -126.f ? 0.f : __int_as_float((127 + (int)fminf(d, 0.f)) << 23);
}

constexpr float kLog2eHi = 1.44269502f;           // log2(e) rounded
constexpr double kLeftOver = 1.33497581575e-8;     // (log2(e) - kLog2eHi) * ln 2
constexpr double kLn2 = 0.6931471805599453;
constexpr float kWholeLimit = 0x1p22f;
constexpr float kAbove = 8.f;   // how far above its reference a thread's logits go, times log2 e: arguments are rounded to 2^-21 there

enum PartMode { kNothing = 0, kWhole = 1, kOwnMax = 2, kBad = 3 };

template <typename V>
__device__ __forceinline__ V block_sum(V v, V* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(SFFN_FULL_MASK, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  V t = lane < warps ? red[lane] : V(0);
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(SFFN_FULL_MASK, t, o);
  return t;
}

// The want-th largest pattern among the lanes of a warp (want of 1 to 32; 0 counts as none).
__device__ __forceinline__ uint32_t nth_largest(uint32_t best, int want) {
  uint32_t t = 0;
  for (int i = 0; i < want; ++i) {
    t = __reduce_max_sync(SFFN_FULL_MASK, best);
    const unsigned who = __ballot_sync(SFFN_FULL_MASK, best == t);
    if ((threadIdx.x & 31) == __ffs(who) - 1) best = 0;
  }
  return t;
}

// Elements of a row by their index, for the rare paths.
struct Range {
  const void* p;
  size_t row;
  int from, to, dtype;
  __device__ __forceinline__ float at(int token) const { return ld_elem(p, row + token, dtype); }
};

// The first n_out of a range by (value, index), to the list; all threads of the block.
__device__ __noinline__ void exact_best(const Range c, int n_out, float* value, int* token, int* count, int* red) {
  const int tid = threadIdx.x;
  auto reach = [&](uint32_t t, int last) {   // elements above t, or at t up to index `last`
    int n = 0;
    for (int i = c.from + tid; i < c.to; i += kThreads) {
      const float z = c.at(i);
      const uint32_t o = ordered(z);
      n += z > -INFINITY && (o > t || (o == t && i <= last));
    }
    return block_sum(n, red);
  };
  uint32_t t = 0;
  for (int b = 31; b >= 0; --b)
    if (reach(t | 1u << b, INT_MAX) >= n_out) t |= 1u << b;
  int last = 0;   // the smallest index with which there are enough
  for (int b = 30; b >= 0; --b)
    if (reach(t, last + (1 << b) - 1) < n_out) last += 1 << b;
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int i = c.from + tid; i < c.to; i += kThreads) {
    const float z = c.at(i);
    const uint32_t o = ordered(z);
    if (z > -INFINITY && (o > t || (o == t && i <= last))) {
      const int k = atomicAdd(count, 1);
      if (k < kList) value[k] = z, token[k] = i;
    }
  }
  __syncthreads();
}

template <typename T>
constexpr int type_of() {
  return sizeof(T) == 4 ? SFFN_F32 : std::is_same<T, __half>::value ? SFFN_F16 : SFFN_BF16;
}

// Element j of 16 bytes.
template <typename T>
__device__ __forceinline__ float element(const uint4& v, int j) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (sizeof(T) == 4) return __uint_as_float(w[j & 3]);
  const uint32_t u = w[(j >> 1) & 3];
  if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)(j & 1 ? u >> 16 : u)));
  return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
}

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Adds p to s, what the rounding left to `rest`, which goes into the next addition.
__device__ __forceinline__ void add_with_rest(float& s, float& rest, float p) {
  const float y = __fadd_rn(p, rest), t = __fadd_rn(s, y);
  rest = __fadd_rn(__fsub_rn(s, t), y), s = t;
}
__device__ __forceinline__ void add_with_rest(float2& s, float2& rest, float2 p) {
  const float2 y = __fadd2_rn(p, rest), t = __fadd2_rn(s, y);
  rest = __fadd2_rn(__ffma2_rn(t, make_float2(-1.f, -1.f), s), y), s = t;
}

// Largest logit of a range and, relative to it, the sum of exponentials: for logits that are far from 0, or none.
__device__ __noinline__ float2 far_sum(const Range c, float* red) {
  float m = -INFINITY, sum = 0.f, rest = 0.f;
  for (int i = c.from + threadIdx.x; i < c.to; i += kThreads) m = fmaxf(m, c.at(i));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(SFFN_FULL_MASK, m, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);
  for (int i = c.from + threadIdx.x; i < c.to; i += kThreads) add_with_rest(sum, rest, exp2_fast((c.at(i) - m) * kLog2eHi));
  __syncthreads();
  return make_float2(m, block_sum(sum + rest, red));
}

// Largest element of 16 bytes; NaN aside.
template <typename T>
__device__ __forceinline__ float largest(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    using P = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    const P m = __hmax2(__hmax2(*reinterpret_cast<const P*>(&v.x), *reinterpret_cast<const P*>(&v.y)),
                        __hmax2(*reinterpret_cast<const P*>(&v.z), *reinterpret_cast<const P*>(&v.w)));
    return fmaxf(to_float(m.x), to_float(m.y));
  }
}

// Which elements of 16 bytes reach `bound`, a value of their type: bit p for element 2 p and bit 16 + p for 2 p + 1, or bit
// j for element j of fp32, shifted up by `at`.
template <typename T>
__device__ __forceinline__ uint32_t which_reach(const uint4& v, float bound, int at) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (sizeof(T) == 4) {
      if (__uint_as_float(w[p]) >= bound) m |= 1u << (at + p);
    } else {
      using P = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
      P b;
      if constexpr (std::is_same<T, __half>::value) b = __float2half2_rn(bound); else b = __float2bfloat162_rn(bound);
      m |= __hge2_mask(*reinterpret_cast<const P*>(&w[p]), b) & (0x10001u << (at + p));
    }
  }
  return m;
}

// Raises the bound by the list of n > kThreads places and takes out what does not reach it; all threads of the block.
__device__ __noinline__ void tighten(const BeamArgs& a, size_t base, int n, float* value, int* token, uint32_t* bounds,
                                     int* count, uint32_t& bound) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x;
  uint32_t best = 0;
  for (int i = tid; i < n; i += kThreads) {
    value[i] = ld_elem(a.logits.ptr, base + token[i], a.dtype);
    best = max(best, ordered(value[i]));
  }
  const uint32_t own = nth_largest(best, (a.n_out + kWarps - 1) / kWarps);
  if ((tid & 31) == 0) bounds[tid >> 5] = own;
  int kept[kList / kThreads];
#pragma unroll
  for (int k = 0; k < kList / kThreads; ++k) kept[k] = tid + k * kThreads < n ? token[tid + k * kThreads] : -1;
  __syncthreads();
  uint32_t least = ~0u;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) least = min(least, bounds[w]);
  bound = max(bound, least);
  if (tid == 0) *count = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kList / kThreads; ++k)
    if (kept[k] >= 0 && ordered(value[tid + k * kThreads]) >= bound) token[atomicAdd(count, 1)] = kept[k];
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kRowBlocks) k_beam_rows(const BeamArgs a) {
  constexpr int N = 16 / sizeof(T), kWarps = kThreads / 32, kChunk = kThreads * kRuns * N;
  __shared__ float s_red[32], s_value[kList], s_best[kRanked];
  __shared__ int s_token[kList], s_at[kRanked], s_int[32], s_count, s_left;
  __shared__ uint32_t s_bound[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t slot = (size_t)row * a.parts + part;
  int2* found = a.found + slot * a.n_out;
  const float score = __ldcg(a.scores + row);
  if (!(fabsf(score) < INFINITY) || (a.done && __ldcg(a.done + row))) {   // its logits are not looked at
    if (tid == 0) a.sums[slot] = make_float4(0.f, 0.f, (float)kNothing, 0.f);
    for (int i = tid; i < a.n_out; i += kThreads) found[i] = make_int2(0, -1);
    return;
  }
  const int c0 = (int)((long long)a.chunks * part / a.parts), c1 = (int)((long long)a.chunks * (part + 1) / a.parts);
  const size_t base = row * a.logits.row_stride;
  auto load = [&](int c, uint4* v) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int at = c * kChunk + (r * kThreads + tid) * N, left = a.vocab - at;
      if (a.vec && left >= N) {
        v[r] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.logits.ptr) + base + at));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (sizeof(T) == 4) {
            w[k] = k < left ? __ldcg(static_cast<const uint32_t*>(a.logits.ptr) + base + at + k) : 0xff800000u;
          } else {
            const unsigned short* p = static_cast<const unsigned short*>(a.logits.ptr) + base + at + 2 * k;
            const uint32_t none = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
            w[k] = (2 * k < left ? __ldcg(p) : none) | (2 * k + 1 < left ? __ldcg(p + 1) : none) << 16;
          }
        }
        v[r] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  if (tid == 0) s_count = s_left = 0;
  uint4 v[kRuns];
  load(c0, v);
  // of this thread; until something is above -2^22 the reference is there, and nothing adds to the sum
  float ref = -kWholeLimit, most = -INFINITY;
  float2 sum2 = make_float2(0.f, 0.f), rest2 = sum2;
  uint32_t bound = 0;   // what an element has to reach
  for (int c = c0; c < c1; ++c) {
    uint4 nv[kRuns];
    if (c + 1 < c1) load(c + 1, nv);
    float top = largest<T>(v[0]);
#pragma unroll
    for (int r = 1; r < kRuns; ++r) top = fmaxf(top, largest<T>(v[r]));
    // -- sum of exponentials; a masked logit's is 0, that of no number is none
    if (top > most) {
      const float near = rintf(top * kLog2eHi);
      if (top >= -kWholeLimit && (most < -kWholeLimit || near > ref + kAbove)) {
        const float down = power_of_two(ref - near);
        sum2.x *= down, sum2.y *= down, rest2.x *= down, rest2.y *= down, ref = near;
      }
      most = top;
    }
    const float2 hi = make_float2(kLog2eHi, kLog2eHi), off = make_float2(-ref, -ref);
    auto term = [&](int r, int j) {
      const float2 x = __ffma2_rn(make_float2(element<T>(v[r], j), element<T>(v[r], j + 1)), hi, off);
      return make_float2(exp2_fast(x.x), exp2_fast(x.y));
    };
    float2 chunk = make_float2(0.f, 0.f), pair = chunk;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      float2 run = term(r, 0);
#pragma unroll
      for (int j = 2; j < N; j += 2) run = __fadd2_rn(run, term(r, j));
      pair = r & 1 ? __fadd2_rn(pair, run) : run;
      if (r & 1) chunk = r == 1 ? pair : __fadd2_rn(chunk, pair);
    }
    add_with_rest(sum2, rest2, chunk);
    // -- what may be among the best
    const uint32_t best = top > -INFINITY ? ordered(top) : 0u;
    if (bound == 0) {   // at the first chunk, and until one has enough elements; before that, everything goes
      const uint32_t wbound = nth_largest(best, (a.n_out + kWarps - 1) / kWarps);
      __syncthreads();
      if (lane == 0) s_bound[warp] = wbound;
      __syncthreads();
      bound = ~0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) bound = min(bound, s_bound[w]);
    }
    // the places of what reaches it; values are fetched again at the end. With no bound yet, of all that is not masked.
    uint32_t hits = 0;
    if (best >= bound && best) {
      const float from = bound ? value_of(bound) : lowest<T>();
#pragma unroll
      for (int r = 0; r < kRuns; ++r) hits |= which_reach<T>(v[r], from, 4 * r);
    }
    int n = 0;
    if (bound == 0) {   // many: one addition a warp
      const int own = __popc(hits);
      int upto = own;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int p = __shfl_up_sync(SFFN_FULL_MASK, upto, o);
        if (lane >= o) upto += p;
      }
      if (lane == 31) n = atomicAdd(&s_count, upto);
      n = __shfl_sync(SFFN_FULL_MASK, n, 31) + upto - own;
    }
    while (hits) {
      const int bit = __ffs(hits) - 1, p = bit & 15;
      hits &= hits - 1;
      const int j = sizeof(T) == 4 ? p & 3 : 2 * (p & 3) + (bit >> 4);
      if (bound) n = atomicAdd(&s_count, 1);
      if (n < kList) s_token[n] = c * kChunk + ((p >> 2) * kThreads + tid) * N + j;
      ++n;
    }
    if (((c - c0) & 3) == 3) {   // a long list raises the bound: what reaches it of eight warps' entries, as above
      __syncthreads();
      const int listed = s_count;
      __syncthreads();   // read by all before anything is added
      if (listed > kTighten && listed <= kList) tighten(a, base, listed, s_value, s_token, s_bound, &s_count, bound);
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r) v[r] = nv[r];
  }
  __syncthreads();
  int n = s_count;
  if (n > kList) {
    const Range all = {a.logits.ptr, base, c0 * kChunk, min(c1 * kChunk, a.vocab), a.dtype};
    exact_best(all, a.n_out, s_value, s_token, &s_count, s_int);
    n = min(s_count, kList);
  } else {
    for (int i = tid; i < n; i += kThreads) s_value[i] = ld_elem(a.logits.ptr, base + s_token[i], a.dtype);
    __syncthreads();
  }
  // -- a bound for the list: of the warps whose lanes all have an entry of it
  const int warps = min(kWarps, n / 32), want = warps ? (a.n_out + warps - 1) / warps : 33;
  uint32_t best = 0, least = 0;
  for (int i = tid; i < n; i += kThreads) best = max(best, ordered(s_value[i]));
  if (want <= 32 && n > 48) {
    const uint32_t wbound = nth_largest(best, want);
    if (lane == 0) s_bound[warp] = wbound;
    __syncthreads();
    least = ~0u;
    for (int w = 0; w < warps; ++w) least = min(least, s_bound[w]);
  }
  for (int i = tid; i < n; i += kThreads)
    if (ordered(s_value[i]) >= least) {
      const int k = atomicAdd(&s_left, 1);
      if (k < kRanked) s_best[k] = s_value[i], s_at[k] = s_token[i];
    }
  __syncthreads();
  const bool few = s_left <= kRanked;   // else the list itself is put in order
  const float* value = few ? s_best : s_value;
  const int* token = few ? s_at : s_token;
  n = few ? s_left : n;
  for (int i = tid; i < n; i += kThreads) {
    const float z = value[i];
    const int t = token[i];
    int ahead = 0;
    for (int k = 0; k < n; ++k) ahead += value[k] > z || (value[k] == z && token[k] < t);
    if (ahead < a.n_out) found[ahead] = make_int2(__float_as_int(z), t);
  }
  for (int i = n + tid; i < a.n_out; i += kThreads) found[i] = make_int2(0, -1);
  // -- the block's sum, relative to the largest reference
  float bref = most >= -kWholeLimit ? ref : -INFINITY, bmost = most;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    bref = fmaxf(bref, __shfl_xor_sync(SFFN_FULL_MASK, bref, o));
    bmost = fmaxf(bmost, __shfl_xor_sync(SFFN_FULL_MASK, bmost, o));
  }
  if (lane == 0) s_red[warp] = bref, s_red[kWarps + warp] = bmost;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) bref = fmaxf(bref, s_red[w]), bmost = fmaxf(bmost, s_red[kWarps + w]);
  __syncthreads();
  float sum = block_sum(((sum2.x + sum2.y) + (rest2.x + rest2.y)) * power_of_two(ref - bref), s_red);
  int mode = bmost == -INFINITY ? kNothing : kWhole;
  // below -2^22 a thread has no reference, so that its logits count for nothing: 256 above it they do
  if ((bmost > kWholeLimit || bmost < 256.f - kWholeLimit) && mode == kWhole) {
    const Range all = {a.logits.ptr, base, c0 * kChunk, min(c1 * kChunk, a.vocab), a.dtype};
    const float2 f = far_sum(all, s_red);
    bref = bmost = f.x, sum = f.y, mode = kOwnMax;
  }
  if (sum != sum || bmost == INFINITY) mode = kBad;
  if (tid == 0) a.sums[slot] = make_float4(bref, sum, (float)mode, bmost);
}

// What decides between equal totals, the smallest first: beam, logit (the largest first, where a large score swallows what
// sets totals apart), token.
__device__ __forceinline__ unsigned long long place_of(int j, int logit, int token) {
  return (unsigned long long)j << 56 | (unsigned long long)~ordered(__int_as_float(logit)) << 24 | (unsigned)token;
}

__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamArgs a) {
  constexpr int kWarps = kMergeThreads / 32;
  __shared__ double s_lse[kMaxBeams];      // log of the row's sum
  __shared__ double s_sum[kMaxBeams], s_ref[kMaxBeams];
  __shared__ float s_score[kMaxBeams];     // -infinity: no candidates
  __shared__ int s_done[kMaxBeams];
  __shared__ int s_int[32], s_count;
  __shared__ float s_top[kWarps];
  __shared__ int s_steps[kSteps], s_step;
  __shared__ unsigned long long s_key[kList], s_place[kList];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the first candidates of a thread are on their way while the rows' sums are joined
  int2 kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int e = tid + i * kMergeThreads, all = a.beams * a.parts * a.n_out;
    kept[i] = e < all ? __ldcg(a.found + (size_t)b * all + e) : make_int2(0, -1);
  }
  // -- a warp for each row: its sum, as a power of two or a logarithm times a number
  for (int j = warp; j < a.beams; j += kWarps) {
    const int row = b * a.beams + j;
    const float score = __ldcg(a.scores + row);
    const bool ended = a.done && __ldcg(a.done + row);
    bool bad = !(score < INFINITY);
    double sum = 0.0, ref = 0.0;
    if (!ended && fabsf(score) < INFINITY) {
      const float4* sums = a.sums + (size_t)row * a.parts;
      const float4 first = lane < a.parts ? __ldcg(sums + lane) : make_float4(0.f, 0.f, (float)kNothing, 0.f);
      float top = -INFINITY, peak = -INFINITY;
      bool own = false;
      for (int c = lane; c < a.parts; c += 32) {
        const float4 s = c < 32 ? first : __ldcg(sums + c);
        bad |= s.z == (float)kBad, own |= s.z == (float)kOwnMax;
        if (s.z == (float)kWhole) top = fmaxf(top, s.x), peak = fmaxf(peak, s.w);
      }
      own = __any_sync(SFFN_FULL_MASK, own), bad = __any_sync(SFFN_FULL_MASK, bad);
      if (!own) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          top = fmaxf(top, __shfl_xor_sync(SFFN_FULL_MASK, top, o));
          peak = fmaxf(peak, __shfl_xor_sync(SFFN_FULL_MASK, peak, o));
        }
        for (int c = lane; c < a.parts; c += 32) {
          const float4 s = c < 32 ? first : __ldcg(sums + c);
          if (s.z == (float)kWhole)
            sum += (double)(s.y * power_of_two(s.x - top)) * (1.0 + (s.w - peak) * kLeftOver);
        }
        ref = top * kLn2 + peak * kLeftOver;
      } else {
        // some part's own largest is its reference: all in the measure of logits, with what rounding log2 e left
        auto reference = [](const float4& s) { return s.z == (float)kWhole ? s.x * kLn2 + s.w * kLeftOver : (double)s.x; };
        double most = -INFINITY;
        for (int c = lane; c < a.parts; c += 32) {
          const float4 s = c < 32 ? first : __ldcg(sums + c);
          if (s.z != (float)kNothing) most = fmax(most, reference(s));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmax(most, __shfl_xor_sync(SFFN_FULL_MASK, most, o));
        for (int c = lane; c < a.parts; c += 32) {
          const float4 s = c < 32 ? first : __ldcg(sums + c);
          if (s.z != (float)kNothing) sum += s.y * exp(reference(s) - most);
        }
        ref = most;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(SFFN_FULL_MASK, sum, o);
    }
    if (lane == 0) {
      s_sum[j] = sum, s_ref[j] = ref, s_done[j] = ended;
      s_score[j] = bad || (!ended && !(sum > 0.0)) ? -INFINITY : score;
      if (bad) set_device_error(a.err, SFFN_ERR_DEVICE);
    }
  }
  if (tid == 0) s_count = 0;
  if (tid < kSteps) s_steps[tid] = 0;
  __syncthreads();
  // logarithms in 64 bits, a lane each: every warp that does one takes a microsecond of the SM
  for (int j = tid; j < a.beams; j += kMergeThreads) s_lse[j] = s_ref[j] + log(s_sum[j]);
  __syncthreads();
  // -- candidates: those found in parts, and the last places of sequences that have ended
  const int per_row = a.parts * a.n_out, entries = a.beams * per_row;
  const int2* found = a.found + (size_t)b * entries;
  auto fetch = [&](int e) { return e < entries ? __ldcg(found + e) : make_int2(0, -1); };
  // the candidate at place e: its pattern (0: none), beam and token
  auto candidate = [&](int e, const int2& f, int& j, int& token) -> unsigned long long {
    if (e >= entries) return 0;
    j = e / per_row, token = s_done[j] ? a.end_token : f.y;
    if (s_score[j] == -INFINITY || (s_done[j] ? e != j * per_row : token < 0)) return 0;
    return ordered(s_done[j] ? (double)s_score[j] : (__int_as_float(f.x) - s_lse[j]) + s_score[j]);
  };
  // those that a thread holds are worked out once: 64-bit arithmetic is slow
  unsigned long long keys[kKept];
  float values[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    int j, token;
    keys[i] = candidate(tid + i * kMergeThreads, kept[i], j, token);
    values[i] = keys[i] ? (float)number(keys[i]) : -INFINITY;
  }
  auto each = [&](auto&& take) {   // take(pattern, value, place())
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (keys[i]) {
        const int j = (tid + i * kMergeThreads) / per_row;
        take(keys[i], values[i], [&] { return s_done[j] ? place_of(j, 0, a.end_token) : place_of(j, kept[i].x, kept[i].y); });
      }
    for (int e = tid + kKept * kMergeThreads; e < entries; e += kMergeThreads) {
      int j, token;
      const int2 f = fetch(e);
      const unsigned long long o = candidate(e, f, j, token);
      if (o) take(o, (float)number(o), [&] { return place_of(j, s_done[j] ? 0 : f.x, token); });
    }
  };
  // a bound that n_out totals reach and few others: how many lie how far below the largest, in steps of 1/16
  float best = -INFINITY;
  each([&](unsigned long long, float v, auto) { best = fmaxf(best, v); });
#pragma unroll
  for (int o = 16; o; o >>= 1) best = fmaxf(best, __shfl_xor_sync(SFFN_FULL_MASK, best, o));
  if (lane == 0) s_top[warp] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) best = fmaxf(best, s_top[w]);
  auto step_of = [&](float v) { return (int)fminf((best - v) * 16.f, kSteps - 1.f); };
  each([&](unsigned long long, float v, auto) { atomicAdd(&s_steps[step_of(v)], 1); });
  __syncthreads();
  if (warp == 0) {
    int n = 0, at = kSteps - 1;
#pragma unroll
    for (int i = 0; i < kSteps / 32; ++i) n += s_steps[lane * (kSteps / 32) + i];
    int upto = n;   // in the steps of this lane and those before
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int p = __shfl_up_sync(SFFN_FULL_MASK, upto, o);
      if (lane >= o) upto += p;
    }
#pragma unroll
    for (int i = kSteps / 32 - 1; i >= 0; --i) {
      if (upto >= a.n_out) at = lane * (kSteps / 32) + i;
      upto -= s_steps[lane * (kSteps / 32) + i];
    }
    at = __reduce_min_sync(SFFN_FULL_MASK, at);
    if (lane == 0) s_step = at;
  }
  __syncthreads();
  const int last_step = s_step;   // the last of all has no end
  each([&](unsigned long long o, float v, auto place) {
    if (step_of(v) <= last_step) {
      const int n = atomicAdd(&s_count, 1);
      if (n < kList) s_key[n] = o, s_place[n] = place();
    }
  });
  __syncthreads();
  int n = s_count;
  if (n > kList) {
    auto reach = [&](unsigned long long t, unsigned long long last) {
      int c = 0;
      each([&](unsigned long long o, float, auto place) { c += o > t || (o == t && place() <= last); });
      return block_sum(c, s_int);
    };
    unsigned long long t = 0;
    for (int i = 63; i >= 0; --i)
      if (reach(t | 1ull << i, ~0ull) >= a.n_out) t |= 1ull << i;
    unsigned long long last = 0;   // the smallest place with which there are enough
    for (int i = 61; i >= 0; --i)
      if (reach(t, last + (1ull << i) - 1) < a.n_out) last += 1ull << i;
    if (tid == 0) s_count = 0;
    __syncthreads();
    each([&](unsigned long long o, float, auto place) {
      const unsigned long long p = place();
      if (o > t || (o == t && p <= last)) {
        const int k = atomicAdd(&s_count, 1);
        if (k < kList) s_key[k] = o, s_place[k] = p;
      }
    });
    __syncthreads();
    n = min(s_count, kList);
  }
  const size_t out = (size_t)b * a.n_out;
  for (int i = tid; i < n; i += kMergeThreads) {
    const unsigned long long v = s_key[i], p = s_place[i];
    int ahead = 0;
    for (int k = 0; k < n; ++k) {
      const unsigned long long o = s_key[k];
      ahead += o > v || (o == v && s_place[k] < p);
    }
    if (ahead < a.n_out) {
      a.out_scores[out + ahead] = (float)number(v);
      a.out_parents[out + ahead] = (int)(p >> 56), a.out_tokens[out + ahead] = (int)(p & 0xffffff);
    }
  }
  for (int i = n + tid; i < a.n_out; i += kMergeThreads)
    a.out_scores[out + i] = -INFINITY, a.out_parents[out + i] = 0, a.out_tokens[out + i] = 0;
}

// Parts of a row: as many as give every SM its blocks in one wave, a chunk at least each, and no more than one block merges
// (16 beams over 254727 for 32 places: 120 us with 62 parts a row).
struct Split {
  int chunks, parts;
};
Split split_of(const sffn_beam& H, int batch, int elem) {
  Split s;
  s.chunks = (H.desc.vocab + kThreads * kRuns * 16 / elem - 1) / (kThreads * kRuns * 16 / elem);
  s.parts = std::min({s.chunks, std::max(1, H.num_sms * kRowBlocks / (batch * H.desc.beams)),
                      std::max(1, kMerged / (H.desc.beams * H.desc.n_out))});
  return s;
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_rows(const BeamArgs& a, cudaStream_t st) {
  return launch_ex(k_beam_rows<T>, dim3(a.parts, a.batch * a.beams), dim3(kThreads), 0, st, true, 1, a);
}

}  // namespace

// Enough for every smaller batch too, whose rows are cut into more parts: rows times parts is at most what fills the SMs
// once, or the rows.
size_t beam_ws_bytes(const sffn_beam& H, int batch) {
  const size_t rows = (size_t)batch * H.desc.beams;
  size_t most = std::max(rows, std::min((size_t)H.num_sms * kRowBlocks, rows * split_of(H, 1, 4).chunks));
  return up256(most * sizeof(float4)) + up256(most * H.desc.n_out * sizeof(int2));
}

cudaError_t launch_beam(const sffn_beam& H, const sffn_rows& logits, const float* scores, const uint8_t* done,
                        int end_token, int batch, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                        int dtype, void* ws, cudaStream_t st) {
  BeamArgs a = {};
  const int elem = dtype == SFFN_F32 ? 4 : 2;
  const Split s = split_of(H, batch, elem);
  a.logits = logits, a.scores = scores, a.done = done, a.out_scores = out_scores, a.out_parents = out_parents;
  a.out_tokens = out_tokens, a.err = H.err;
  a.vocab = H.desc.vocab, a.beams = H.desc.beams, a.n_out = H.desc.n_out, a.batch = batch, a.end_token = end_token;
  a.dtype = dtype, a.chunks = s.chunks, a.parts = s.parts;
  const size_t slots = (size_t)batch * a.beams * a.parts;
  a.sums = static_cast<float4*>(ws);
  a.found = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + up256(slots * sizeof(float4)));
  a.vec = reinterpret_cast<uintptr_t>(logits.ptr) % 16 == 0 &&
          ((long long)batch * a.beams <= 1 || logits.row_stride * elem % 16 == 0);
  cudaError_t e = dtype == SFFN_F32   ? launch_rows<float>(a, st)
                  : dtype == SFFN_F16 ? launch_rows<__half>(a, st)
                                      : launch_rows<__nv_bfloat16>(a, st);
  if (e != cudaSuccess) return e;
  return launch_ex(k_beam_merge, dim3(batch), dim3(kMergeThreads), 0, st, true, 1, a);
}

}  // namespace sffn
