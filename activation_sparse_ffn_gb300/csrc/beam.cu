// The best continuations over beams and vocabulary.
//
// k_beam_rows reads every logit once: a block takes a chunk of one row into
// registers, sums its exponentials and keeps its n_out best. k_beam_merge, a
// block for each search, joins the sums of a row, turns the kept logits into
// totals and picks the n_out best of those.
//
// Sums of exponentials. exp(z) = 2^(z log2 e); the reference that a chunk takes
// off is a whole number R near the largest z log2 e, so that sums of different
// chunks are brought together by a power of two, exactly. log2 e is carried by
// two floats: one alone is off by 2^-26 of itself, which a logit of 20 makes
// 2^-21. Above |z| = 2^22 a whole number no longer lies near enough; the
// chunk's largest z is the reference there.
//
// The n_out best of a chunk. The n_out-th largest of the threads' own maxima
// bounds the n_out-th largest element from below; a binary search over the upper
// bits of their ordered patterns finds it nearly, and the few elements that
// reach it go to a list, where each counts those ahead of it. Where too many are
// equal for the list, a search over all bits and then over indices takes exactly
// the first of them.
#include <algorithm>

#include "rows_io.cuh"
#include "step.h"

namespace sffn {

namespace {

constexpr int kThreads = 256;
constexpr int kMergeThreads = 512;
constexpr int kMaxOut = 64;
constexpr int kMaxBeams = 64;
constexpr int kList = 2048;   // (kMaxOut - 1) * 32 elements of fewer than kMaxOut threads always fit

struct BeamArgs {
  sffn_rows logits;
  const float* scores;
  const uint8_t* done;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  uint32_t* err;
  // workspace: sums of each row's chunks, and their candidates
  float4* sums;    // [rows][chunks]: reference, sum, mode, -
  int2* found;     // [rows][chunks][n_out]: logit, token; token -1: none
  int vocab, beams, n_out, batch, end_token, dtype, chunks;
  bool vec;
};

// Patterns that order like the numbers (NaN aside).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  const unsigned long long u = __double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2eHi = 1.44269502f;        // log2(e) rounded
constexpr float kLog2eLo = 1.92596303e-8f;     // and what that left
constexpr float kWholeLimit = 0x1p22f;

enum ChunkMode { kNothing = 0, kWhole = 1, kOwnMax = 2, kBad = 3 };

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

// Largest pattern t (of its upper bits) that at least `want` threads' `best` reach; 0 if fewer have anything.
template <int BITS>
__device__ __forceinline__ uint32_t reached(uint32_t best, int want) {
  uint32_t t = 0;
  for (int b = 31; b > 31 - BITS; --b) {
    const uint32_t up = t | 1u << b;
    if (__syncthreads_count(best >= up) >= want) t = up;
  }
  return t;
}

template <typename T, int EPT>
__global__ void __launch_bounds__(kThreads) k_beam_rows(const BeamArgs a) {
  constexpr int N = 16 / sizeof(T), RUNS = EPT / N;
  __shared__ float red[32];
  __shared__ int s_count, s_int[32];
  __shared__ float s_value[kList];
  __shared__ int s_token[kList];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x;
  const size_t slot = (size_t)row * a.chunks + chunk;
  int2* found = a.found + slot * a.n_out;
  const float score = __ldcg(a.scores + row);
  if (!(fabsf(score) < INFINITY) || (a.done && __ldcg(a.done + row))) {   // its logits are not looked at
    if (tid == 0) a.sums[slot] = make_float4(0.f, 0.f, (float)kNothing, 0.f);
    for (int i = tid; i < a.n_out; i += kThreads) found[i] = make_int2(0, -1);
    return;
  }
  const int at0 = chunk * (kThreads * EPT) + tid * N;
  float z[EPT];
#pragma unroll
  for (int r = 0; r < RUNS; ++r) {
    const int at = at0 + r * kThreads * N, left = a.vocab - at;
    const size_t i = row * a.logits.row_stride + at;
    if (a.vec && left >= N) {
      ld_run<N>(a.logits.ptr, i, sizeof(T) == 4 ? SFFN_F32 : std::is_same<T, __half>::value ? SFFN_F16 : SFFN_BF16,
                z + r * N);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) z[r * N + j] = j < left ? ld_elem(a.logits.ptr, i + j, a.dtype) : -INFINITY;
    }
  }
  // -- largest, and whether anything is no number
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPT; ++j) top = fmaxf(top, z[j]), bad |= !(z[j] < INFINITY);
  const uint32_t best = ordered(top);
  const uint32_t wtop = __reduce_max_sync(SFFN_FULL_MASK, best);
  if (tid == 0) s_count = 0;
  if ((tid & 31) == 0) s_int[tid >> 5] = (int)wtop;
  bad = __syncthreads_or(bad);
  const int lane = tid & 31;
  const uint32_t btop = __reduce_max_sync(SFFN_FULL_MASK, lane < kThreads / 32 ? (uint32_t)s_int[lane] : 0u);
  const float m = __uint_as_float(btop & 0x80000000u ? btop ^ 0x80000000u : ~btop);
  if (bad || m == -INFINITY) {
    if (tid == 0) a.sums[slot] = make_float4(0.f, 0.f, (float)(bad ? kBad : kNothing), 0.f);
    for (int i = tid; i < a.n_out; i += kThreads) found[i] = make_int2(0, -1);
    return;
  }
  // -- sum of exponentials
  const bool whole = fabsf(m) <= kWholeLimit;
  const float ref = whole ? rintf(m * kLog2eHi) : m;
  float sum = 0.f;
  if (whole) {
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      // a masked logit: -infinity in the first product, nothing in the sum
      const float x = fmaf(z[j], kLog2eHi, -ref);
      sum += exp2_fast(z[j] == -INFINITY ? -INFINITY : fmaf(z[j], kLog2eLo, x));
    }
  } else {
    for (int j = 0; j < EPT; ++j) sum += exp2_fast((z[j] - m) * kLog2eHi);
  }
  sum = block_sum(sum, red);
  if (tid == 0) a.sums[slot] = make_float4(ref, sum, (float)(whole ? kWhole : kOwnMax), 0.f);
  // -- the n_out best
  uint32_t bound = reached<16>(best, a.n_out);
#pragma unroll
  for (int j = 0; j < EPT; ++j)
    if (ordered(z[j]) >= bound && z[j] > -INFINITY) {
      const int n = atomicAdd(&s_count, 1);
      if (n < kList) s_value[n] = z[j], s_token[n] = at0 + (j / N) * kThreads * N + j % N;
    }
  __syncthreads();
  int n = s_count;
  if (n > kList) {
    // too many equal ones: the first of them by index
    auto count = [&](uint32_t t, int last) {   // elements above t, or at t up to index `last`
      int c = 0;
      for (int j = 0; j < EPT; ++j) {
        const uint32_t o = ordered(z[j]);
        c += z[j] > -INFINITY && (o > t || (o == t && at0 + (j / N) * kThreads * N + j % N <= last));
      }
      return block_sum(c, s_int);
    };
    uint32_t t = 0;
    for (int b = 31; b >= 0; --b)
      if (count(t | 1u << b, INT_MAX) >= a.n_out) t |= 1u << b;
    int last = 0;   // the smallest index with which there are enough
    for (int b = 30; b >= 0; --b)
      if (count(t, last + (1 << b) - 1) < a.n_out) last += 1 << b;
    if (tid == 0) s_count = 0;
    __syncthreads();
    for (int j = 0; j < EPT; ++j) {
      const uint32_t o = ordered(z[j]);
      const int token = at0 + (j / N) * kThreads * N + j % N;
      if (z[j] > -INFINITY && (o > t || (o == t && token <= last))) {
        const int k = atomicAdd(&s_count, 1);
        if (k < kList) s_value[k] = z[j], s_token[k] = token;
      }
    }
    __syncthreads();
    n = min(s_count, kList);
  }
  for (int i = tid; i < n; i += kThreads) {
    const float v = s_value[i];
    const int token = s_token[i];
    int ahead = 0;
    for (int k = 0; k < n; ++k) ahead += s_value[k] > v || (s_value[k] == v && s_token[k] < token);
    if (ahead < a.n_out) found[ahead] = make_int2(__float_as_int(v), token);
  }
  for (int i = n + tid; i < a.n_out; i += kThreads) found[i] = make_int2(0, -1);
}

__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(const BeamArgs a) {
  __shared__ double s_lse[kMaxBeams];   // log of the row's sum
  __shared__ double s_score[kMaxBeams];    // -infinity: no candidates
  __shared__ bool s_done[kMaxBeams];
  __shared__ int s_int[32], s_count;
  __shared__ double s_total[kList];
  __shared__ int s_place[kList][2];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // -- a warp for each row
  for (int j = warp; j < a.beams; j += kMergeThreads / 32) {
    const int row = b * a.beams + j;
    const float score = __ldcg(a.scores + row);
    const bool ended = a.done && __ldcg(a.done + row);
    double lse = -INFINITY;
    bool bad = !(score < INFINITY);
    if (!ended && fabsf(score) < INFINITY) {
      const float4* sums = a.sums + (size_t)row * a.chunks;
      float ref = -INFINITY;
      bool own = false;
      for (int c = lane; c < a.chunks; c += 32) {
        const float4 s = __ldcg(sums + c);
        bad |= s.z == (float)kBad, own |= s.z == (float)kOwnMax;
      }
      own = __any_sync(SFFN_FULL_MASK, own), bad = __any_sync(SFFN_FULL_MASK, bad);
      // references in the same measure: whole powers of two, or logits where some chunk has its own largest
      for (int c = lane; c < a.chunks; c += 32) {
        const float4 s = __ldcg(sums + c);
        if (s.z != (float)kNothing) ref = fmaxf(ref, own && s.z == (float)kWhole ? s.x * 0.693147181f : s.x);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(SFFN_FULL_MASK, ref, o));
      double sum = 0.0;
      for (int c = lane; c < a.chunks; c += 32) {
        const float4 s = __ldcg(sums + c);
        if (s.z == (float)kNothing || bad) continue;
        if (!own)
          sum += scalbn((double)s.y, max((int)(s.x - ref), -1000));
        else
          sum += s.y * exp((s.z == (float)kWhole ? s.x * 0.6931471805599453 : (double)s.x) - ref);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(SFFN_FULL_MASK, sum, o);
      if (!bad && sum > 0.0) lse = (own ? (double)ref : ref * 0.6931471805599453) + log(sum);
    }
    if (lane == 0) {
      s_lse[j] = lse, s_score[j] = bad || (!ended && lse == -INFINITY) ? -INFINITY : score, s_done[j] = ended;
      if (bad) set_device_error(a.err, SFFN_ERR_DEVICE);
    }
  }
  if (tid == 0) s_count = 0;
  __syncthreads();
  // -- candidates: those found in chunks, and the last places of sequences that have ended
  const int per_row = a.chunks * a.n_out, entries = a.beams * per_row;
  const int2* found = a.found + (size_t)b * entries;
  auto total = [&](int e, int& j, int& token) {   // NaN: none
    j = e / per_row;
    if (s_done[j]) {
      token = a.end_token;
      return e == j * per_row && s_score[j] > -INFINITY ? s_score[j] : nan("");
    }
    const int2 f = __ldcg(found + e);
    token = f.y;
    return token < 0 || s_score[j] == -INFINITY ? nan("") : (__int_as_float(f.x) - s_lse[j]) + s_score[j];
  };
  int j, token;
  uint32_t best = 0;
  for (int e = tid; e < entries; e += kMergeThreads) {
    const double v = total(e, j, token);
    if (v == v) best = max(best, ordered((float)v));
  }
  const uint32_t bound = reached<24>(best, a.n_out);
  for (int e = tid; e < entries; e += kMergeThreads) {
    const double v = total(e, j, token);
    if (v == v && ordered((float)v) >= bound) {
      const int n = atomicAdd(&s_count, 1);
      if (n < kList) s_total[n] = v, s_place[n][0] = j, s_place[n][1] = token;
    }
  }
  __syncthreads();
  int n = s_count;
  if (n > kList) {
    auto count = [&](unsigned long long t, long long last) {
      int c = 0;
      for (int e = tid; e < entries; e += kMergeThreads) {
        const double v = total(e, j, token);
        if (v == v) c += ordered(v) > t || (ordered(v) == t && (long long)j * a.vocab + token <= last);
      }
      return block_sum(c, s_int);
    };
    unsigned long long t = 0;
    for (int i = 63; i >= 0; --i)
      if (count(t | 1ull << i, LLONG_MAX) >= a.n_out) t |= 1ull << i;
    long long last = 0;
    for (int i = 32; i >= 0; --i)
      if (count(t, last + (1ll << i) - 1) < a.n_out) last += 1ll << i;
    if (tid == 0) s_count = 0;
    __syncthreads();
    for (int e = tid; e < entries; e += kMergeThreads) {
      const double v = total(e, j, token);
      if (v == v && (ordered(v) > t || (ordered(v) == t && (long long)j * a.vocab + token <= last))) {
        const int k = atomicAdd(&s_count, 1);
        if (k < kList) s_total[k] = v, s_place[k][0] = j, s_place[k][1] = token;
      }
    }
    __syncthreads();
    n = min(s_count, kList);
  }
  const size_t out = (size_t)b * a.n_out;
  for (int i = tid; i < n; i += kMergeThreads) {
    const double v = s_total[i];
    const int pj = s_place[i][0], pt = s_place[i][1];
    int ahead = 0;
    for (int k = 0; k < n; ++k) {
      const double o = s_total[k];
      ahead += o > v || (o == v && (s_place[k][0] < pj || (s_place[k][0] == pj && s_place[k][1] < pt)));
    }
    if (ahead < a.n_out) a.out_scores[out + ahead] = (float)v, a.out_parents[out + ahead] = pj, a.out_tokens[out + ahead] = pt;
  }
  for (int i = n + tid; i < a.n_out; i += kMergeThreads)
    a.out_scores[out + i] = -INFINITY, a.out_parents[out + i] = 0, a.out_tokens[out + i] = 0;
}

// Elements of a thread: few, so that a small call has blocks for every SM; more where there are rows enough.
int elements(const sffn_beam& H, int batch) {
  const long long cells = (long long)batch * H.desc.beams * H.desc.vocab;
  int ept = 8;
  while (ept < 32 && cells > (long long)H.num_sms * 8 * kThreads * ept) ept *= 2;
  return ept;
}
int chunks_of(const sffn_beam& H, int ept) { return (H.desc.vocab + kThreads * ept - 1) / (kThreads * ept); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_rows(const BeamArgs& a, int ept, cudaStream_t st) {
  auto kern = ept == 8 ? k_beam_rows<T, 8> : ept == 16 ? k_beam_rows<T, 16> : k_beam_rows<T, 32>;
  return launch_ex(kern, dim3(a.chunks, a.batch * a.beams), dim3(kThreads), 0, st, true, 1, a);
}

}  // namespace

// Enough for every smaller batch too, whose rows may be cut into more chunks.
size_t beam_ws_bytes(const sffn_beam& H, int batch) {
  size_t most = 0;
  for (int ept = 8; ept <= 32; ept *= 2) {
    const long long cells = (long long)H.desc.beams * H.desc.vocab, limit = (long long)H.num_sms * 8 * kThreads * ept;
    const long long b = ept == 32 ? batch : std::min((long long)batch, std::max(1ll, limit / cells));
    most = std::max(most, (size_t)b * H.desc.beams * chunks_of(H, ept));
  }
  return up256(most * sizeof(float4)) + up256(most * H.desc.n_out * sizeof(int2));
}

cudaError_t launch_beam(const sffn_beam& H, const sffn_rows& logits, const float* scores, const uint8_t* done,
                        int end_token, int batch, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                        int dtype, void* ws, cudaStream_t st) {
  BeamArgs a = {};
  const int ept = elements(H, batch);
  a.logits = logits, a.scores = scores, a.done = done, a.out_scores = out_scores, a.out_parents = out_parents;
  a.out_tokens = out_tokens, a.err = H.err;
  a.vocab = H.desc.vocab, a.beams = H.desc.beams, a.n_out = H.desc.n_out, a.batch = batch, a.end_token = end_token;
  a.dtype = dtype, a.chunks = chunks_of(H, ept);
  const size_t slots = (size_t)batch * a.beams * a.chunks;
  a.sums = static_cast<float4*>(ws);
  a.found = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + up256(slots * sizeof(float4)));
  const int elem = dtype == SFFN_F32 ? 4 : 2;
  a.vec = reinterpret_cast<uintptr_t>(logits.ptr) % 16 == 0 &&
          ((long long)batch * a.beams <= 1 || logits.row_stride * elem % 16 == 0);
  cudaError_t e = dtype == SFFN_F32   ? launch_rows<float>(a, ept, st)
                  : dtype == SFFN_F16 ? launch_rows<__half>(a, ept, st)
                                      : launch_rows<__nv_bfloat16>(a, ept, st);
  if (e != cudaSuccess) return e;
  return launch_ex(k_beam_merge, dim3(batch), dim3(kMergeThreads), 0, st, true, 1, a);
}

}  // namespace sffn
