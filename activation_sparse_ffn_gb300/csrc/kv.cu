// Append to and read back from the paged 4-bit key/value cache.
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

struct AppendArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows q, k, v, q_out;
  int hq, dtype;
  sffn_rope rope;  // table null: no rotation
};

// One warp per (token, head) row: query heads are rotated and written out; key
// heads are rotated, rounded and stored; value heads are rounded and stored.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_append(const AppendArgs a) {
  constexpr int CPL = D / 32;  // consecutive channels of a lane
  __shared__ __align__(16) float s_row[kWarps][D];
  __shared__ __align__(16) uint8_t s_code[kWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.hq + 2 * a.c.hkv;
  const long long item = (long long)blockIdx.x * kWarps + warp;
  if (item >= (long long)a.b.n_tokens * heads) return;
  const int i = (int)(item / heads), h = (int)(item % heads);
  const int kind = h < a.hq ? 0 : h < a.hq + a.c.hkv ? 1 : 2;
  const int hh = kind == 0 ? h : kind == 1 ? h - a.hq : h - a.hq - a.c.hkv;
  const sffn_rows& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int c0 = lane * CPL;
  float x[CPL];
  ld_run<CPL>(src.ptr, (size_t)(i * src.row_stride + hh * src.head_stride) + c0, a.dtype, x);
  const KvPlace at = kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  if (kind != 2 && a.rope.table) {
    const int pos = a.rope.positions ? ld_dep(a.rope.positions + i) : at.pos;
    if (pos >= 0 && pos < a.rope.length) {
      const int half = a.rope.dim >> 1;
      float* row = s_row[warp];
#pragma unroll
      for (int e = 0; e < CPL; ++e) row[c0 + e] = x[e];
      __syncwarp();
      const float2* cs = reinterpret_cast<const float2*>(a.rope.table) + (size_t)pos * half;
#pragma unroll
      for (int e = 0; e < CPL; ++e) {
        const int c = c0 + e;
        if (c < a.rope.dim) {
          const int j = a.rope.style == 0 ? (c < half ? c : c - half) : c >> 1;
          const bool first = a.rope.style == 0 ? c < half : (c & 1) == 0;
          const int p = a.rope.style == 0 ? (first ? c + half : c - half) : c ^ 1;
          const float2 t = __ldg(cs + j);
          const float u = __fmul_rn(x[e], t.x), w = __fmul_rn(row[p], t.y);
          x[e] = first ? __fsub_rn(u, w) : __fadd_rn(u, w);
        }
      }
      __syncwarp();
    } else if (a.rope.positions || pos >= 0) {
      set_device_error(a.c.err, SFFN_ERR_DEVICE);
    }
  }
  if (kind == 0) {
    st_run<CPL>(a.q_out.ptr, (size_t)(i * a.q_out.row_stride + hh * a.q_out.head_stride) + c0, a.dtype, x);
    return;
  }
  if (at.pos < 0) return;
  const int page = kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err);
  if (page < 0) return;
  uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)hh * a.c.head_bytes;
  const int slot = at.pos % a.c.P, which = kind - 1;

  // least and largest value of the group, over the lanes that share it
  float lo = x[0], hi = x[0];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    bad |= !(fabsf(x[e]) < __int_as_float(0x7f800000));
  }
  const int lanes = 32 / a.c.n_groups;
  for (int o = lanes >> 1; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(SFFN_FULL_MASK, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(SFFN_FULL_MASK, hi, o));
    bad |= __shfl_xor_sync(SFFN_FULL_MASK, (int)bad, o) != 0;
  }
  const float m = __fadd_rn(__fmul_rn(lo, 0.5f), __fmul_rn(hi, 0.5f));
  __half mid = __float2half_rn(fminf(fmaxf(m, -kHalfMax), kHalfMax));
  const float midf = __half2float(mid);
  const float far = fmaxf(__fsub_rn(hi, midf), __fsub_rn(midf, lo));
  __half step = __float2half_rn(fminf(__fmul_rn(far, 1.f / 15.f), kHalfMax));
  if (bad) mid = __ushort_as_half(0), step = __ushort_as_half(0x7fff);
  const float stepf = __half2float(step), inv = __frcp_rn(__fmul_rn(2.f, stepf));
  uint8_t* code = s_code[warp];
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    const float t = floorf(__fadd_rn(__fmul_rn(__fsub_rn(x[e], midf), inv), 8.f));
    code[c0 + e] = stepf == 0.f || bad ? 8 : (uint8_t)fminf(fmaxf(t, 0.f), 15.f);
  }
  __syncwarp();
  if (lane % lanes == 0) {
    const int grp = lane / lanes;
    *reinterpret_cast<__half2*>(block + kv_param_off(a.c.P, D) + param_off(slot, grp, a.c.n_groups, which)) =
        __halves2half2(step, mid);
  }
  if (lane < D / 8) {
    uint8_t u[8];
    uint32_t* dst;
    if (which == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = code[8 * lane + e];
      dst = reinterpret_cast<uint32_t*>(block + slot * (D / 2) + key_word_off<D>(slot, lane & 3, lane >> 2));
      *dst = key_word(u);
    } else {
      const int g = lane & 7, w = lane >> 3;
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = code[64 * w + 8 * e + g];
      dst = reinterpret_cast<uint32_t*>(block + kv_value_off(a.c.P, D) + slot * (D / 2) + value_word_off<D>(slot, g, w));
      *dst = value_word(u);
    }
  }
}

struct GatherArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows k, v;
  int dtype;
};

// One warp per (token, key head, keys or values).
template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_gather(const GatherArgs a) {
  constexpr int CPL = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + warp;
  if (item >= 2ll * a.b.n_tokens * a.c.hkv) return;
  const int which = (int)(item & 1), h = (int)((item >> 1) % a.c.hkv), i = (int)((item >> 1) / a.c.hkv);
  const sffn_rows& dst = which ? a.v : a.k;
  if (!dst.ptr) return;
  const KvPlace at = kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  float x[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) x[e] = 0.f;
  if (at.pos >= 0) {
    const int page = max(0, kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err));
    const uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)h * a.c.head_bytes;
#pragma unroll
    for (int e = 0; e < CPL; ++e)
      x[e] = kv_value<D>(block, a.c.P, a.c.n_groups, at.pos % a.c.P, lane * CPL + e, which);
  }
  st_run<CPL>(dst.ptr, (size_t)(i * dst.row_stride + h * dst.head_stride) + lane * CPL, a.dtype, x);
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
  const AppendArgs a{view_of(C), b, q, k, v, q_out, q.ptr ? n_q_heads : 0, dtype, rope};
  const long long rows = (long long)b.n_tokens * (a.hq + 2 * a.c.hkv);
  return by_dim(C.desc.head_dim, [&](auto d) {
    return launch_ex(k_kv_append<decltype(d)::value>, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                     0, st, true, 1, a);
  });
}

cudaError_t launch_kv_gather(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& k_out, const sffn_rows& v_out,
                             int dtype, cudaStream_t st) {
  const GatherArgs a{view_of(C), b, k_out, v_out, dtype};
  const long long rows = 2ll * b.n_tokens * a.c.hkv;
  return by_dim(C.desc.head_dim, [&](auto d) {
    return launch_ex(k_kv_gather<decltype(d)::value>, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                     0, st, true, 1, a);
  });
}

}  // namespace sffn
