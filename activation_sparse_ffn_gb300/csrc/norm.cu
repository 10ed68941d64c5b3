// Root-mean-square norm with the residual's addition, and rows of 8-bit codes.
//
// One block per row, which stays in registers from the one read to the one
// write. The codes have to be defined, so every step but the mean is one fp32
// rounding, and the mean, whose order of summation differs from block to
// block, is carried far enough that its rounding to f hardly ever depends on it:
// squares and sums as two floats each (the second has what the first's
// rounding left, by fma(t, t, -t^2) and by Knuth's two-sum), 2^-44 or better
// after all additions, and the root in 64 bits. One row in some 2^20 lies so near
// a rounding's border that f may be its other neighbour.
//
// Measured: 8192 rows of 8192 bf16 elements with a residual 106 us, 5.1 TB/s; 34 instructions an element, ten of them the
// sums', keep 55% of the issue slots busy, and two blocks an SM wait for each other's barriers. 4096 rows of 8192 to codes
// alone 82 us (45 instructions an element), their codes without a norm 40 (22). One fp32 row of 8192 5.0 us, a block's way
// through it: load, sum, root, store.
#include <algorithm>

#include "rows_io.cuh"
#include "step.h"

namespace sffn {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kSms = 152;                 // of a GB300
constexpr int kManyRows = 2 * kSms;

template <typename T>
constexpr int kRun = 16 / sizeof(T);   // elements of one 16-byte access

// s + p into s, what the rounding left into c.
__device__ __forceinline__ void two_sum(float& s, float& c, float p) {
  const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
  s = t;
}

// Sum of two-float numbers and largest of bit patterns over the block; every thread gets the result.
__device__ __forceinline__ void block_reduce(float& s, float& c, uint32_t& top, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float ps = __shfl_xor_sync(SFFN_FULL_MASK, s, o), pc = __shfl_xor_sync(SFFN_FULL_MASK, c, o);
    two_sum(s, c, ps);
    c = __fadd_rn(c, pc);
  }
  // lanes may differ in the last bits of c: the block goes by the first's
  s = __shfl_sync(SFFN_FULL_MASK, s, 0), c = __shfl_sync(SFFN_FULL_MASK, c, 0);
  top = __reduce_max_sync(SFFN_FULL_MASK, top);
  if (warps == 1) return __syncwarp();   // red may still be read from an earlier row, here and below
  __syncthreads();
  if (lane == 0) red[warp] = s, red[32 + warp] = c, red[64 + warp] = __uint_as_float(top);
  __syncthreads();
  s = lane < warps ? red[lane] : 0.f;
  c = lane < warps ? red[32 + lane] : 0.f;
  top = lane < warps ? __float_as_uint(red[64 + lane]) : 0u;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float ps = __shfl_xor_sync(SFFN_FULL_MASK, s, o), pc = __shfl_xor_sync(SFFN_FULL_MASK, c, o);
    two_sum(s, c, ps);
    c = __fadd_rn(c, pc);
  }
  s = __shfl_sync(SFFN_FULL_MASK, s, 0), c = __shfl_sync(SFFN_FULL_MASK, c, 0);
  top = __reduce_max_sync(SFFN_FULL_MASK, top);
}

__device__ __forceinline__ uint32_t block_max(uint32_t top, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  top = __reduce_max_sync(SFFN_FULL_MASK, top);
  if (warps == 1) return top;
  __syncthreads();
  if (lane == 0) red[warp] = __uint_as_float(top);
  __syncthreads();
  return __reduce_max_sync(SFFN_FULL_MASK, lane < warps ? __float_as_uint(red[lane]) : 0u);
}

// f32(1 / sqrt(sum / width + eps)), by one warp for the block: 64-bit arithmetic issues at a sixteenth of a warp a cycle, and
// all warps of a row of 8192 together took 9 us for it. Newton's iteration from the fp32 estimate doubles its 22
// bits twice.
__device__ __forceinline__ float factor(double sum, double inv_width, double eps, float* red) {
  if (threadIdx.x < 32) {
    const double v = fma(sum, inv_width, eps);
    double r = rsqrtf((float)v);
    if (v > 1e-30 && v < 1e30) {
#pragma unroll
      for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-v * r, r, 1.0), r);
    } else {
      r = 1.0 / sqrt(v);   // past what the estimate holds, 0, infinity or no number
    }
    if (threadIdx.x == 0) red[96] = (float)r;
  }
  __syncthreads();
  return red[96];
}

// |v| as bits: ordered like the values, infinity and then NaN above them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ float scale_of(uint32_t top) {
  return top >= kInfBits ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(top), 127.f);
}

// N codes: y / scale rounded to the nearest whole number, ties to even, as the quotient rounded to fp32 gives it, four in a
// word. The product with 1 / scale is off by less than 2^-15 where the quotient is at most 128, so only near a tie is the
// quotient itself looked at, which takes the division. Added to 3 2^22 a quotient is rounded and its code stands in the
// low byte, without a conversion (those issue at an eighth of the additions' rate).
template <int N>
__device__ __forceinline__ void codes_of(const float* y, float scale, float inv, uint32_t* w) {
  constexpr float kShift = 12582912.f;
  bool slow = !(scale >= 0x1p-120f);   // 0, no number, or too small for its reciprocal
  uint32_t c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float q = __fmul_rn(y[j], inv), m = __fadd_rn(q, kShift), off = __fsub_rn(q, __fsub_rn(m, kShift));
    slow |= !(fabsf(__fsub_rn(fabsf(off), 0.5f)) > 0x1p-14f);
    c[j] = __float_as_uint(m);
  }
  if (slow) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      c[j] = scale > 0.f ? (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(y[j], scale)), -127.f), 127.f) : 0u;
  }
#pragma unroll
  for (int j = 0; j < N; j += 4)
    w[j / 4] = __byte_perm(__byte_perm(c[j], c[j + 1], 0x0040), __byte_perm(c[j + 2], c[j + 3], 0x0040), 0x5410);
}

// Where rows may be read and written 16 bytes (codes: one run) at a time.
struct NormVec {
  bool x, residual, sum, y, codes, weight;
};

template <int N>
__device__ __forceinline__ void load_some(const void* p, size_t i, int left, int dtype, bool vec, float* o) {
  if (vec && left >= N) {
    ld_run<N>(p, i, dtype, o);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = j < left ? ld_elem(p, i + j, dtype) : 0.f;
  }
}

template <int N>
__device__ __forceinline__ void store_some(void* p, size_t i, int left, int dtype, bool vec, const float* v) {
  if (vec && left >= N) {
    st_run<N>(p, i, dtype, v);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < left) st_elem(p, i + j, v[j], dtype);
  }
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, int left, bool vec, const float* y, float scale, float inv) {
  uint32_t w[N / 4];
  codes_of<N>(y, scale, inv, w);
  if (vec && left >= N) {
    if (N == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[N / 4 - 1]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < left) p[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}

template <typename T>
constexpr int dtype_of() {
  return sizeof(T) == 4 ? SFFN_F32 : std::is_same<T, __half>::value ? SFFN_F16 : SFFN_BF16;
}

// f of the block's row, of which each thread has EPT elements.
template <int EPT>
__device__ __forceinline__ float row_factor(const float* t, int width, double eps, double inv_width, float* red) {
  // four sums, so that one addition need not wait for the one before
  float part[4] = {0.f, 0.f, 0.f, 0.f}, rest[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const float p = __fmul_rn(t[j], t[j]);
    two_sum(part[j & 3], rest[j & 3], p);
    rest[j & 3] = __fadd_rn(rest[j & 3], __fmaf_rn(t[j], t[j], -p));
    top = max(top, abs_bits(t[j]));
  }
  float s = part[0], c = __fadd_rn(__fadd_rn(rest[0], rest[1]), __fadd_rn(rest[2], rest[3]));
#pragma unroll
  for (int i = 1; i < 4; ++i) two_sum(s, c, part[i]);
  block_reduce(s, c, top, red);
  double sum = (double)s + (double)c;
  if (top >= kInfBits) {
    sum = top > kInfBits ? nan("") : (double)INFINITY;
  } else if (top && (top > __float_as_uint(0x1p56f) || top < __float_as_uint(0x1p-39f))) {
    // squares or what they leave would pass fp32's range: the row times a power of two
    const int e = 127 - (int)(top >> 23);   // of a subnormal row: 127
    const float up = scalbnf(1.f, e / 2), up2 = scalbnf(1.f, e - e / 2);
    s = c = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const float v = __fmul_rn(__fmul_rn(t[j], up), up2), p = __fmul_rn(v, v);
      two_sum(s, c, p);
      c = __fadd_rn(c, __fmaf_rn(v, v, -p));
    }
    block_reduce(s, c, top, red);
    sum = scalbn((double)s + (double)c, -2 * e);
  }
  return factor(sum, inv_width, eps, red);
}

// EPT elements a thread: in runs of 16 bytes, run r of thread t from (r * threads + t) * kRun on, or, where some array is not
// aligned to that (SPREAD), element k of thread t at k * threads + t, so that a warp reads what lies together (1671 rows of
// 4839 halves with a residual: 58 us with runs).
template <typename T, int EPT, bool SPREAD>
__global__ void __launch_bounds__(kMaxThreads) k_norm(const NormArgs a, double inv_width) {
  constexpr int N = kRun<T>, D = dtype_of<T>();
  __shared__ float red[97];
  pdl_launch_dependents();
  pdl_wait();
  const size_t row = blockIdx.x;
  const int step = blockDim.x;
  constexpr int G = 8;   // elements that are loaded together
  auto load = [&](const void* p, size_t from, int dtype, int k0, float* o) {
    if constexpr (SPREAD) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int at = (k0 + k) * step + threadIdx.x;
        o[k] = at < a.width ? ld_elem(p, from + at, dtype) : 0.f;
      }
    } else {
#pragma unroll
      for (int k = 0; k < G; k += N) {
        const int at = (k0 + k) * step + threadIdx.x * N;
        load_some<N>(p, from + at, a.width - at, dtype, true, o + k);
      }
    }
  };
  auto store = [&](void* p, size_t from, int dtype, const float* v) {
    if constexpr (SPREAD) {
#pragma unroll
      for (int k = 0; k < EPT; ++k) {
        const int at = k * step + threadIdx.x;
        if (at < a.width) st_elem(p, from + at, v[k], dtype);
      }
    } else {
#pragma unroll
      for (int k = 0; k < EPT; k += N) {
        const int at = (k * step) + threadIdx.x * N;
        store_some<N>(p, from + at, a.width - at, dtype, true, v + k);
      }
    }
  };
  auto inside = [&](int k) { return (SPREAD ? k * step + (int)threadIdx.x : k / N * N * step + (int)threadIdx.x * N + k % N) < a.width; };
  float t[EPT];
#pragma unroll
  for (int k0 = 0; k0 < EPT; k0 += G) load(a.x.ptr, row * a.x.row_stride, D, k0, t + k0);
  if (a.residual.ptr) {
#pragma unroll
    for (int k0 = 0; k0 < EPT; k0 += G) {
      float o[G];
      load(a.residual.ptr, row * a.residual.row_stride, D, k0, o);
#pragma unroll
      for (int k = 0; k < G; ++k) t[k0 + k] = __fadd_rn(t[k0 + k], o[k]);
    }
  }
  if (a.sum.ptr) store(a.sum.ptr, row * a.sum.row_stride, D, t);
  if (a.norm) {
    const float f = row_factor<EPT>(t, a.width, a.eps, inv_width, red);
    if (a.weight) {
#pragma unroll
      for (int k0 = 0; k0 < EPT; k0 += G) {
        float w[G];
        load(a.weight, 0, SFFN_F32, k0, w);
#pragma unroll
        for (int k = 0; k < G; ++k) t[k0 + k] = __fmul_rn(__fmul_rn(t[k0 + k], f), w[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < EPT; ++k) t[k] = __fmul_rn(t[k], f);
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) t[k] = inside(k) ? t[k] : 0.f;   // of no element, whatever f is
    if (a.y.ptr) store(a.y.ptr, row * a.y.row_stride, a.y_dtype, t);
  }
  if (a.codes.ptr) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < EPT; ++k) top = max(top, abs_bits(t[k]));
    top = block_max(top, red);
    const float scale = scale_of(top), inv = __fdiv_rn(1.f, scale);
    if (threadIdx.x == 0) a.scales[row] = scale;
    int8_t* out = static_cast<int8_t*>(a.codes.ptr) + row * a.codes.row_stride;
    if constexpr (SPREAD) {
#pragma unroll
      for (int k = 0; k < EPT; k += 4) {
        uint32_t w;
        codes_of<4>(t + k, scale, inv, &w);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (inside(k + e)) out[(k + e) * step + threadIdx.x] = (int8_t)(w >> (8 * e));
      }
    } else {
#pragma unroll
      for (int k = 0; k < EPT; k += N) {
        const int at = k * step + threadIdx.x * N;
        if (at < a.width) store_codes<N>(out + at, a.width - at, true, t + k, scale, inv);
      }
    }
  }
}

// Elements of 16 bytes.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& v, float* o) {
  WType<T>::unpack(v, o);
}

// The same for many rows that are aligned throughout: a block takes row after row, the next one on its way while one is
// reduced and written, and keeps the weights in shared memory. 8192 rows of 8192 bf16 elements with a residual: 143 us with
// a block for each row, where an SM waits for the loads, barriers and 64-bit arithmetic of the four it holds.
template <typename T, int EPT>
__global__ void __launch_bounds__(256, EPT == 32 ? 2 : 4) k_norm_many(const NormArgs a, double inv_width) {
  constexpr int N = kRun<T>, RUNS = EPT / N;
  extern __shared__ __align__(16) float weights[];
  __shared__ float red[97];
  pdl_launch_dependents();
  pdl_wait();
  if (a.weight)
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) weights[i] = __ldcg(a.weight + i);
  const int step = blockDim.x * N, at0 = threadIdx.x * N;
  uint4 x[RUNS], o[RUNS];
  auto fetch = [&](size_t row) {
    const T* px = static_cast<const T*>(a.x.ptr) + row * a.x.row_stride;
    const T* po = static_cast<const T*>(a.residual.ptr) + row * a.residual.row_stride;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const int at = at0 + r * step;
      x[r] = o[r] = make_uint4(0, 0, 0, 0);
      if (at < a.width) {
        x[r] = __ldcg(reinterpret_cast<const uint4*>(px + at));
        if (a.residual.ptr) o[r] = __ldcg(reinterpret_cast<const uint4*>(po + at));
      }
    }
  };
  fetch(blockIdx.x);
  __syncthreads();
  for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
    float t[EPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      unpack16<T>(x[r], t + r * N);
      if (a.residual.ptr) {
        float u[N];
        unpack16<T>(o[r], u);
#pragma unroll
        for (int j = 0; j < N; ++j) t[r * N + j] = __fadd_rn(t[r * N + j], u[j]);
      }
    }
    if (row + gridDim.x < (size_t)a.rows) fetch(row + gridDim.x);
    if (a.sum.ptr) {
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
        if (at0 + r * step < a.width) st_run<N>(a.sum.ptr, row * a.sum.row_stride + at0 + r * step, dtype_of<T>(), t + r * N);
    }
    if (a.norm) {
      const float f = row_factor<EPT>(t, a.width, a.eps, inv_width, red);
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        const int at = at0 + r * step;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
          if (a.weight && at < a.width) w = *reinterpret_cast<const float4*>(weights + at + j);
          float* v = t + r * N + j;
          v[0] = __fmul_rn(__fmul_rn(v[0], f), w.x), v[1] = __fmul_rn(__fmul_rn(v[1], f), w.y);
          v[2] = __fmul_rn(__fmul_rn(v[2], f), w.z), v[3] = __fmul_rn(__fmul_rn(v[3], f), w.w);
        }
        if (at >= a.width)
#pragma unroll
          for (int j = 0; j < N; ++j) t[r * N + j] = 0.f;   // of no element, whatever f is
      }
      if (a.y.ptr) {
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
          if (at0 + r * step < a.width) st_run<N>(a.y.ptr, row * a.y.row_stride + at0 + r * step, a.y_dtype, t + r * N);
      }
    }
    if (a.codes.ptr) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < EPT; ++j) top = max(top, abs_bits(t[j]));
      top = block_max(top, red);
      const float scale = scale_of(top), inv = __fdiv_rn(1.f, scale);
      if (threadIdx.x == 0) a.scales[row] = scale;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        const int at = at0 + r * step;
        if (at < a.width)
          store_codes<N>(static_cast<int8_t*>(a.codes.ptr) + row * a.codes.row_stride + at, N, true, t + r * N, scale, inv);
      }
    }
  }
}

// Rows too wide for a block's registers, as they are: read twice.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) k_quantize_wide(const NormArgs a, const NormVec vec) {
  constexpr int N = kRun<T>, D = dtype_of<T>();
  __shared__ float red[97];
  pdl_launch_dependents();
  pdl_wait();
  const size_t row = blockIdx.x;
  uint32_t top = 0;
  float t[N];
  for (int at = threadIdx.x * N; at < a.width; at += blockDim.x * N) {
    load_some<N>(a.x.ptr, row * a.x.row_stride + at, a.width - at, D, vec.x, t);
#pragma unroll
    for (int j = 0; j < N; ++j) top = max(top, abs_bits(t[j]));
  }
  top = block_max(top, red);
  const float scale = scale_of(top), inv = __fdiv_rn(1.f, scale);
  if (threadIdx.x == 0) a.scales[row] = scale;
  for (int at = threadIdx.x * N; at < a.width; at += blockDim.x * N) {
    load_some<N>(a.x.ptr, row * a.x.row_stride + at, a.width - at, D, vec.x, t);
    store_codes<N>(static_cast<int8_t*>(a.codes.ptr) + row * a.codes.row_stride + at, a.width - at, vec.codes, t, scale,
                   inv);
  }
}

bool on(const sffn_rows& r, int64_t rows, int elem, int run_bytes) {
  return reinterpret_cast<uintptr_t>(r.ptr) % run_bytes == 0 && (rows <= 1 || r.row_stride * elem % run_bytes == 0);
}

template <typename T>
cudaError_t launch_typed(const NormArgs& a, cudaStream_t st) {
  constexpr int N = kRun<T>;
  const int ye = a.y_dtype == SFFN_F32 ? 4 : 2;
  NormVec vec;
  vec.x = on(a.x, a.rows, sizeof(T), 16), vec.residual = on(a.residual, a.rows, sizeof(T), 16);
  vec.sum = on(a.sum, a.rows, sizeof(T), 16), vec.y = on(a.y, a.rows, ye, 16);
  vec.codes = on(a.codes, a.rows, 1, N), vec.weight = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  if (a.width > kMaxThreads * 32)
    return launch_ex(k_quantize_wide<T>, dim3(a.rows), dim3(kMaxThreads), 0, st, true, 1, a, vec);
  const bool aligned = vec.x && (!a.residual.ptr || vec.residual) && (!a.sum.ptr || vec.sum) && (!a.y.ptr || vec.y) &&
                       (!a.codes.ptr || vec.codes) && a.width % N == 0;
  if (a.rows > kManyRows && a.width <= 256 * 32 && aligned) {
    // as many blocks as the SMs hold
    const int ept = a.width <= 256 * 8 ? 8 : a.width <= 256 * 16 ? 16 : 32;
    const int threads = ((a.width + ept - 1) / ept + 31) / 32 * 32;
    const int per_sm = ept == 32 ? 2 : std::min(16, 4 * 256 / threads);
    auto kern = ept == 8 ? k_norm_many<T, 8> : ept == 16 ? k_norm_many<T, 16> : k_norm_many<T, 32>;
    return launch_ex(kern, dim3(std::min(a.rows, kSms * per_sm)), dim3(threads), a.weight ? a.width * sizeof(float) : 0, st,
                     true, 1, a, 1.0 / a.width);
  }
  // Few rows: as many threads as there are, for the shortest way through one row. Many: blocks of 256, so that an SM
  // holds several and one loads while another waits at its barriers.
  // Not aligned: 16 elements a thread while they reach, since 32 spill.
  const bool spread = !(vec.x && (!a.residual.ptr || vec.residual) && (!a.sum.ptr || vec.sum) && (!a.y.ptr || vec.y) &&
                        (!a.codes.ptr || vec.codes) && vec.weight);
  int ept = 8;
  while (ept < 32 && (a.width > kMaxThreads * ept || (a.rows > kManyRows && a.width > (!spread ? 256 : ept == 8 ? 512 : kMaxThreads) * ept))) ept *= 2;
  const int threads = std::min(kMaxThreads, ((a.width + ept - 1) / ept + 31) / 32 * 32);
  auto kern = spread ? ept == 8 ? k_norm<T, 8, true> : ept == 16 ? k_norm<T, 16, true> : k_norm<T, 32, true>
                     : ept == 8 ? k_norm<T, 8, false> : ept == 16 ? k_norm<T, 16, false> : k_norm<T, 32, false>;
  return launch_ex(kern, dim3(a.rows), dim3(threads), 0, st, true, 1, a, 1.0 / a.width);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  if (a.dtype == SFFN_F32) return launch_typed<float>(a, st);
  return a.dtype == SFFN_F16 ? launch_typed<__half>(a, st) : launch_typed<__nv_bfloat16>(a, st);
}

}  // namespace sffn
