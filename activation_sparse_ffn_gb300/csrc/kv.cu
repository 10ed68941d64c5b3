// Append to and read back from the paged 4-bit key/value cache.
#include <algorithm>
#include <type_traits>

#include "attn.h"
#include "kv_layout.cuh"
#include "rows_io.cuh"

namespace sffn {

namespace {

constexpr int kWarps = 4;
constexpr float kHalfMax = 65504.f;

struct CacheView {
  uint8_t* pages;
  size_t page_bytes, head_bytes;
  int n_pages, P, hkv, n_groups;
  uint32_t* err;
};

CacheView view_of(const sffn_kv& C) {
  return CacheView{C.pages,           C.page_bytes,      C.head_bytes, C.desc.n_pages, C.desc.page_size,
                   C.desc.n_kv_heads, C.desc.head_dim / C.desc.group, C.err};
}

// A warp handles rows (a head's channels) of one token, eight channels per
// lane: eight lanes are a row of 64, sixteen one of 128, so that four, two or
// one row are in hand at a time, the next ones' loads under way. Eight channels
// are a whole key word; value words take one channel of eight lanes each.
template <int D>
struct RowLanes {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;
};

// Eight consecutive elements as loaded, and as fp32.
template <typename T>
struct Raw {
  static constexpr int N = sizeof(T) / 2;   // 16-byte pieces
  uint4 v[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < N; ++i) WType<T>::unpack(v[i], x + i * WType<T>::kPerChunk);
  }
};

template <typename T>
constexpr int dtype_of() {
  return std::is_same<T, float>::value ? SFFN_F32 : std::is_same<T, __half>::value ? SFFN_F16 : SFFN_BF16;
}

struct AppendArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows q, k, v, q_out;
  int hq, dtype;
  int per, q_tasks, kv_tasks;   // rows of a task (one warp), tasks of a token's query rows, of its key rows and of its value rows
  sffn_rope rope;               // table null: no rotation
};

// The rotation of a lane's eight channels. Where pairs and halves fall on whole
// lanes, the (cos, sin) of the lane's channels stay in registers for all rows of
// the token and the other half comes by a shuffle; else channel by channel from
// memory.
template <int D>
struct Turn {
  float2 cs[8];
  int kind = 0;        // 0 none, 1 first half of pairs of lanes, 2 second half, 3 neighbouring channels, 4 by channel
  int partner = 0;     // lane of the other half
  bool shuffles = false;
  const float2* table = nullptr;

  __device__ __forceinline__ void set(const sffn_rope& r, int pos, int lane) {
    const int c0 = lane % RowLanes<D>::kLanes * 8, half = r.dim >> 1;
    table = reinterpret_cast<const float2*>(r.table) + (size_t)pos * half;
    partner = lane;
    if (r.style == 0 && half % 8 == 0) {
      shuffles = true;
      if (c0 < r.dim) {
        kind = c0 < half ? 1 : 2;
        partner = kind == 1 ? lane + half / 8 : lane - half / 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          cs[e] = __ldg(table + (kind == 1 ? c0 : c0 - half) + e);
          if (kind == 1) cs[e].y = -cs[e].y;   // a cos - b sin and b cos + a sin become one formula, the same bits
        }
      }
    } else if (r.style == 1 && r.dim % 8 == 0) {
      if (c0 < r.dim) {
        kind = 3;
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = __ldg(table + c0 / 2 + e);
      }
    } else {
      kind = 4;
    }
  }
  // x: the lane's channels of a row of elements of type dtype
  __device__ __forceinline__ void apply(const sffn_rope& r, float* x, const void* row, int dtype, int lane, bool on) const {
    if (shuffles) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(SFFN_FULL_MASK, x[e], partner);
      if (on && kind != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], cs[e].x), __fmul_rn(y[e], cs[e].y));
      }
    } else if (on && kind == 3) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = __fsub_rn(__fmul_rn(a, cs[e].x), __fmul_rn(b, cs[e].y));
        x[2 * e + 1] = __fadd_rn(__fmul_rn(b, cs[e].x), __fmul_rn(a, cs[e].y));
      }
    } else if (on && kind == 4) {
      const int c0 = lane % RowLanes<D>::kLanes * 8, half = r.dim >> 1;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        if (c >= r.dim) break;
        const bool first = r.style == 0 ? c < half : (c & 1) == 0;
        const int p = r.style == 0 ? (first ? c + half : c - half) : c ^ 1;
        const float2 t = __ldg(table + (r.style == 0 ? (first ? c : c - half) : c >> 1));
        const float u = __fmul_rn(ld_elem(row, c, dtype), t.x), w = __fmul_rn(ld_elem(row, p, dtype), t.y);
        const float v = first ? __fsub_rn(u, w) : __fadd_rn(u, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k == e) x[k] = v;
      }
    }
    __syncwarp();   // every partner is read before a row is written in place
  }
};

// Least and largest of three, NaN if one is NaN.
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Rows r0 .. r1 - 1 of one kind (0 queries, 1 keys, 2 values) of token i.
//
// A group's mid is the middle of its least and largest value and its step a
// fifteenth of the farther one's distance, each rounded to a half; code u = floor
// of (x - mid) / (2 step) + 8, limited to 0 .. 15, stands for mid + step (2u - 15).
// All of it in fp32 with one rounding per operation, in the order of the
// definition, so that the stored bits can be told beforehand.
//
// Bound: queries by memory; keys and values by about 250 instructions per lane
// and eight channels, which keep 77% of the issue slots of an active SM busy
// (DRAM 38% of its peak): no unit is at its limit, and the rest is waits for
// fixed latencies and loads. 7950 prompt tokens of 32 + 2 x 32 bf16 heads of 128 (297 MB) take 88
// us, 3.4 TB/s, of which keys and values alone 73; one token 3 us. Four channels
// a lane took 2.5 times as long, a loop that serves the three kinds 1.5 times;
// rows loaded 1 to 4 ahead make no difference, and neither do packed fp32
// operations.
template <int D, typename T, int KIND>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int i, const KvPlace* place, int r0, int r1, int lane) {
  constexpr int LR = RowLanes<D>::kLanes, RI = RowLanes<D>::kRows, dtype = dtype_of<T>();
  const int sub = lane / LR, lr = lane % LR, c0 = lr * 8;
  const sffn_rows& rows = KIND == 0 ? a.q : KIND == 1 ? a.k : a.v;
  const T* p = static_cast<const T*>(rows.ptr) + i * rows.row_stride + (r0 + sub) * rows.head_stride + c0;
  const int64_t hop = RI * rows.head_stride;
  Raw<T> next = {};   // the row after the one in hand
  if (r0 + sub < r1) next.load(p);
  const KvPlace at = kv_many(a.b) ? *place : kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  Turn<D> turn;
  if (KIND != 2 && a.rope.table) {
    const int pos = a.rope.positions ? ld_dep(a.rope.positions + i) : at.pos;
    if (pos >= 0 && pos < a.rope.length)
      turn.set(a.rope, pos, lane);
    else if (a.rope.positions || pos >= 0)
      set_device_error(a.c.err, SFFN_ERR_DEVICE);
  }
  const int glanes = LR / a.c.n_groups;
  uint8_t* word = nullptr;     // of the lane's codes, and of its group's params, in the block of head r0 + sub
  uint8_t* param = nullptr;
  T* out = nullptr;
  if (KIND == 0) {
    out = static_cast<T*>(a.q_out.ptr) + i * a.q_out.row_stride + (r0 + sub) * a.q_out.head_stride + c0;
  } else {
    if (at.pos < 0) return;
    const int page = kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err);
    if (page < 0) return;
    const int slot = at.pos % a.c.P;
    uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)(r0 + sub) * a.c.head_bytes;
    word = block + (KIND == 2 ? kv_value_off(a.c.P, D) : 0) + slot * (D / 2) +
           (KIND == 2 ? value_word_off<D>(slot, lr & 7, lr >> 3) : key_word_off<D>(slot, lr & 3, lr >> 2));
    param = block + kv_param_off(a.c.P, D) + param_off(slot, lr / glanes, a.c.n_groups, KIND == 2);
  }

  for (int left = r1 - r0 - sub; left + sub > 0; left -= RI) {   // rows from the lane's own on
    const bool in = left > 0;
    float x[8];
    next.get(x);
    if (left > RI) next.load(p + hop);
    if (KIND != 2) turn.apply(a.rope, x, p - c0, dtype, lane, in);
    p += hop;
    if (KIND == 0) {
      if (in) st_run<8>(out, 0, dtype, x);
      out += RI * a.q_out.head_stride;
      continue;
    }
    // least and largest value of the group, over the lanes that share it
    float lo = min3(min3(x[0], x[1], x[2]), min3(x[3], x[4], x[5]), min3(x[6], x[7], x[7]));
    float hi = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    for (int o = 1; o < glanes; o <<= 1) {
      const float a = __shfl_xor_sync(SFFN_FULL_MASK, lo, o), c = __shfl_xor_sync(SFFN_FULL_MASK, hi, o);
      lo = min3(lo, a, a);
      hi = max3(hi, c, c);
    }
    const bool bad = !(fabsf(lo) < __int_as_float(0x7f800000) && fabsf(hi) < __int_as_float(0x7f800000));
    const float m = __fadd_rn(__fmul_rn(lo, 0.5f), __fmul_rn(hi, 0.5f));
    __half mid = __float2half_rn(fminf(fmaxf(m, -kHalfMax), kHalfMax));
    const float midf = __half2float(mid);
    const float far = fmaxf(__fsub_rn(hi, midf), __fsub_rn(midf, lo));
    __half step = __float2half_rn(fminf(__fmul_rn(far, 1.f / 15.f), kHalfMax));
    if (bad) mid = __ushort_as_half(0), step = __ushort_as_half(0x7fff);
    const float stepf = __half2float(step), inv = __frcp_rn(__fmul_rn(2.f, stepf));
    // floor and limits of (x - mid) inv + 8: limits first, then 2^23 + t cut off at the units, whose bit pattern is
    // 0x4b000000 + floor(t); the eight of them are added up with their shifts and the constant taken off at the end.
    // A step that is a normal half and not the largest is within 2^-11 of a fifteenth of the farther end, so that t
    // stays in (0.49, 15.51): then there is nothing to limit.
    // of keys in the order of their word, before its rotation; of values by channel, for the exchange
    auto place = [](int e) { return KIND == 1 ? key_field(e) : 4 * e; };
    uint32_t codes = 0;
    if (__all_sync(SFFN_FULL_MASK, stepf >= 6.103515625e-5f && stepf < kHalfMax)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = __fadd_rn(__fmul_rn(__fsub_rn(x[e], midf), inv), 8.f);
        codes += __float_as_uint(__fadd_rz(t, 8388608.f)) << place(e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = __fadd_rn(__fmul_rn(__fsub_rn(x[e], midf), inv), 8.f);
        codes += __float_as_uint(__fadd_rz(fminf(fmaxf(t, 0.f), 15.f), 8388608.f)) << place(e);
      }
    }
    codes -= 0x4b000000u * 0x11111111u;
    if (stepf == 0.f || bad) codes = 0x88888888u;
    const uint32_t w = KIND == 2 ? value_word(transpose_codes(codes, lane)) : key_word(codes);
    if (in) {
      *reinterpret_cast<uint32_t*>(word) = w;
      if (lr % glanes == 0) *reinterpret_cast<__half2*>(param) = __halves2half2(step, mid);
    }
    word += RI * a.c.head_bytes;
    param += RI * a.c.head_bytes;
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32) k_kv_append(const AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, tasks = a.q_tasks + 2 * a.kv_tasks;
  // A block's warps take neighbouring tokens and run the same of the three loops (mixed within a block: 1.25 times as
  // long); blocks take turns, so that the queries' loads and stores are under way beside the others' arithmetic (7950
  // prompt tokens: 88 us; all queries, then keys, then values 92).
  const int part = blockIdx.x % tasks, i0 = blockIdx.x / tasks * kWarps, warp = threadIdx.x >> 5, i = i0 + warp;
  __shared__ KvPlace s_places[kWarps];
  if (kv_many(a.b)) kv_places<kWarps>(a.b, i0, kWarps * 32, a.c.P, a.c.err, s_places);
  if (i >= a.b.n_tokens) return;
  if (part < a.q_tasks) {
    append_rows<D, T, 0>(a, i, s_places + warp, part * a.per, min((part + 1) * a.per, a.hq), lane);
  } else {
    const int n = part - a.q_tasks, value = n >= a.kv_tasks, r0 = (n - value * a.kv_tasks) * a.per;
    const int r1 = min(r0 + a.per, a.c.hkv);
    if (value)
      append_rows<D, T, 2>(a, i, s_places + warp, r0, r1, lane);
    else
      append_rows<D, T, 1>(a, i, s_places + warp, r0, r1, lane);
  }
}

struct GatherArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows k, v;
  int dtype;
  int per, tasks;   // rows of a task, tasks of a token's key rows and of its value rows
};

// Rows r0 .. r1 - 1 of the keys or values of token i, read back: mid + step (2u - 15),
// rounded once in fp32 and once to the rows' type. Issue slots are 72% busy,
// DRAM 31%, the rest waits: 7950 tokens of 2 x 32 bf16 heads of 128 (167 MB) take
// 42 us, 4.0 TB/s.
template <int D, typename T, bool VALUE>
__device__ __forceinline__ void gather_rows(const GatherArgs& a, int i, const KvPlace* place, int r0, int r1, int lane) {
  constexpr int LR = RowLanes<D>::kLanes, RI = RowLanes<D>::kRows, kBatch = 4;
  const sffn_rows& rows = VALUE ? a.v : a.k;
  if (!rows.ptr) return;
  const int sub = lane / LR, lr = lane % LR;
  const KvPlace at = kv_many(a.b) ? *place : kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  const bool placed = at.pos >= 0;
  const int page = placed ? max(0, kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err)) : 0;
  const int slot = placed ? at.pos % a.c.P : 0;
  const uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)(r0 + sub) * a.c.head_bytes;
  const uint8_t* word = block + (VALUE ? kv_value_off(a.c.P, D) : 0) + slot * (D / 2) +
                        (VALUE ? value_word_off<D>(slot, lr & 7, lr >> 3) : key_word_off<D>(slot, lr & 3, lr >> 2));
  const uint8_t* param = block + kv_param_off(a.c.P, D) + param_off(slot, lr / (LR / a.c.n_groups), a.c.n_groups, VALUE);
  T* out = static_cast<T*>(rows.ptr) + i * rows.row_stride + (r0 + sub) * rows.head_stride + lr * 8;
  for (int rb = r0; rb < r1; rb += RI * kBatch) {
    uint32_t w[kBatch], pm[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      w[k] = pm[k] = 0u;
      if (placed && rb + sub + k * RI < r1) {
        w[k] = __ldcg(reinterpret_cast<const uint32_t*>(word));
        pm[k] = __ldcg(reinterpret_cast<const uint32_t*>(param));
      }
      word += RI * a.c.head_bytes;
      param += RI * a.c.head_bytes;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t codes = VALUE ? transpose_codes(value_codes(w[k]), lane) : key_fields(w[k]);
      const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pm[k]));
      float x[8];
      // 2u - 15 from the bit pattern of 2^23 + 2u; its product with step is exact in fp32 (a 4-bit by an 11-bit
      // number), so there is one rounding
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = VALUE ? 4 * e : key_field(e);
        const uint32_t u2 = at == 0 ? codes << 1 : codes >> (at - 1);
        x[e] = __fmaf_rn(__uint_as_float((u2 & 30u) | 0x4b000000u) - 8388623.f, sm.x, sm.y);
      }
      if (rb + sub + k * RI < r1) st_run<8>(out, 0, dtype_of<T>(), x);   // no place: step and mid are 0
      out += RI * rows.head_stride;
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32) k_kv_gather(const GatherArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, part = blockIdx.x % (2 * a.tasks), value = part >= a.tasks;
  const int i0 = blockIdx.x / (2 * a.tasks) * kWarps, warp = threadIdx.x >> 5, i = i0 + warp;
  __shared__ KvPlace s_places[kWarps];
  if (kv_many(a.b)) kv_places<kWarps>(a.b, i0, kWarps * 32, a.c.P, a.c.err, s_places);
  if (i >= a.b.n_tokens) return;
  const int r0 = (part - value * a.tasks) * a.per, r1 = min(r0 + a.per, a.c.hkv);
  if (value)
    gather_rows<D, T, true>(a, i, s_places + warp, r0, r1, lane);
  else
    gather_rows<D, T, false>(a, i, s_places + warp, r0, r1, lane);
}

// Rows that a task takes: all of a token's where there are tokens enough to fill
// the GPU, so that its place and rotation are found once; fewer, down to what a
// warp has in hand at a time, where there are not.
int rows_per_task(long long rows, int of_token, int at_once, int num_sms) {
  const long long warps = 32ll * num_sms;
  const long long per = rows / warps / at_once * at_once;
  return (int)std::min<long long>(std::max<long long>(per, at_once), (of_token + at_once - 1) / at_once * at_once);
}

template <typename F>
cudaError_t by_dim(int D, F&& f) {
  switch (D) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    default: return f(std::integral_constant<int, 256>());
  }
}

}  // namespace

cudaError_t launch_kv_append(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                             const sffn_rows& k, const sffn_rows& v, const sffn_rows& q_out, const sffn_rope& rope,
                             int dtype, cudaStream_t st) {
  AppendArgs a{view_of(C), b, q, k, v, q_out, q.ptr ? n_q_heads : 0, dtype, 0, 0, 0, rope};
  const int at_once = 32 / (C.desc.head_dim / 8);
  a.per = rows_per_task((long long)b.n_tokens * (a.hq + 2 * a.c.hkv), std::max(a.hq, a.c.hkv), at_once, C.num_sms);
  a.q_tasks = (a.hq + a.per - 1) / a.per;
  a.kv_tasks = (a.c.hkv + a.per - 1) / a.per;
  const dim3 grid((unsigned)((b.n_tokens + kWarps - 1) / kWarps * (a.q_tasks + 2 * a.kv_tasks)));
  return by_dim(C.desc.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto run = [&](auto* kern) { return launch_ex(kern, grid, dim3(kWarps * 32), 0, st, true, 1, a); };
    return dtype == SFFN_F32 ? run(k_kv_append<D, float>)
                             : dtype == SFFN_F16 ? run(k_kv_append<D, __half>) : run(k_kv_append<D, __nv_bfloat16>);
  });
}

cudaError_t launch_kv_gather(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& k_out, const sffn_rows& v_out,
                             int dtype, cudaStream_t st) {
  GatherArgs a{view_of(C), b, k_out, v_out, dtype, 0, 0};
  const int at_once = 32 / (C.desc.head_dim / 8);
  a.per = rows_per_task((long long)b.n_tokens * 2 * a.c.hkv, a.c.hkv, at_once, C.num_sms);
  a.tasks = (a.c.hkv + a.per - 1) / a.per;
  const dim3 grid((unsigned)((b.n_tokens + kWarps - 1) / kWarps * 2 * a.tasks));
  return by_dim(C.desc.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto run = [&](auto* kern) { return launch_ex(kern, grid, dim3(kWarps * 32), 0, st, true, 1, a); };
    return dtype == SFFN_F32 ? run(k_kv_gather<D, float>)
                             : dtype == SFFN_F16 ? run(k_kv_gather<D, __half>) : run(k_kv_gather<D, __nv_bfloat16>);
  });
}

}  // namespace sffn
