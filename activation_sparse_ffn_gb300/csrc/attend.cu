// Attention of decode tokens over the paged 4-bit cache.
#include "attn.h"
#include "kv_layout.cuh"
#include "rows_io.cuh"

namespace sffn {

namespace {

struct AttendArgs {
  const uint8_t* pages;
  size_t page_bytes, head_bytes;
  int n_pages, P, hkv, n_groups;
  uint32_t* err;
  sffn_kv_batch b;
  sffn_rows q, out;
  float* lse;
  int hq, dtype, window;
  float scale;
};

// One warp per (token, query head), one position at a time.
template <int D>
__global__ void __launch_bounds__(128) k_attend(const AttendArgs a) {
  constexpr int CPL = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (long long)a.b.n_tokens * a.hq) return;
  const int i = (int)(item / a.hq), h = (int)(item % a.hq), kh = h / (a.hq / a.hkv);
  const KvPlace at = kv_place(a.b, i, lane, a.P, a.err);
  if (at.seq < 0) return;
  float q[CPL], o[CPL];
  ld_run<CPL>(a.q.ptr, (size_t)(i * a.q.row_stride + h * a.q.head_stride) + lane * CPL, a.dtype, q);
#pragma unroll
  for (int e = 0; e < CPL; ++e) q[e] *= a.scale * 1.4426950408889634f, o[e] = 0.f;
  const float ninf = __int_as_float(0xff800000);
  float m = ninf, l = 0.f;
  const int first = a.window > 0 ? max(0, at.pos - a.window + 1) : 0;
  for (int j = first; j <= at.pos; ++j) {
    const int page = max(0, kv_page(a.b, at.seq, j / a.P, a.n_pages, a.err));
    const uint8_t* block = a.pages + (size_t)page * a.page_bytes + (size_t)kh * a.head_bytes;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) s = fmaf(q[e], kv_value<D>(block, a.P, a.n_groups, j % a.P, lane * CPL + e, 0), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), back = m == mn ? 1.f : exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * back + p;
#pragma unroll
    for (int e = 0; e < CPL; ++e)
      o[e] = o[e] * back + p * kv_value<D>(block, a.P, a.n_groups, j % a.P, lane * CPL + e, 1);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < CPL; ++e) o[e] *= inv;
  st_run<CPL>(a.out.ptr, (size_t)(i * a.out.row_stride + h * a.out.head_stride) + lane * CPL, a.dtype, o);
  if (a.lse && lane == 0) a.lse[(size_t)i * a.hq + h] = l == 0.f ? ninf : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t configure_attend_kernels(const sffn_kv&) { return cudaSuccess; }

size_t attend_ws_bytes(const sffn_kv&, int, int, int) { return 256; }

cudaError_t launch_attend(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                          const sffn_rows& out, float* lse, float scale, int window, int dtype, void* ws,
                          cudaStream_t st) {
  (void)ws;
  const AttendArgs a{C.pages, C.page_bytes, C.head_bytes, C.desc.n_pages, C.desc.page_size, C.desc.n_kv_heads,
                     C.desc.head_dim / C.desc.group, C.err, b, q, out, lse, n_q_heads, dtype, window, scale};
  const dim3 grid((unsigned)(((long long)b.n_tokens * n_q_heads + 3) / 4)), block(128);
  switch (C.desc.head_dim) {
    case 64: return launch_ex(k_attend<64>, grid, block, 0, st, true, 1, a);
    case 128: return launch_ex(k_attend<128>, grid, block, 0, st, true, 1, a);
    default: return launch_ex(k_attend<256>, grid, block, 0, st, true, 1, a);
  }
}

}  // namespace sffn
