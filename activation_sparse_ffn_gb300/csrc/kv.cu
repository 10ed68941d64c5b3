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

struct AppendArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows q, k, v, q_out;
  int hq, dtype;
  int per, q_tasks, kv_tasks;   // rows of a task (one warp), tasks of a token's query rows and of its key and value rows
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
  // x: the lane's channels of a row whose channel 0 is element `at` of src
  __device__ __forceinline__ void apply(const sffn_rope& r, float* x, const void* src, size_t at, int dtype, int lane,
                                        bool on) const {
    if (shuffles) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = __shfl_sync(SFFN_FULL_MASK, x[e], partner);
        if (on && kind != 0) x[e] = __fadd_rn(__fmul_rn(x[e], cs[e].x), __fmul_rn(y, cs[e].y));
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
        const float u = __fmul_rn(ld_elem(src, at + c, dtype), t.x), w = __fmul_rn(ld_elem(src, at + p, dtype), t.y);
        const float v = first ? __fsub_rn(u, w) : __fadd_rn(u, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k == e) x[k] = v;
      }
    }
    __syncwarp();   // every partner is read before a row is written in place
  }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 8) k_kv_append(const AppendArgs a) {
  constexpr int LR = RowLanes<D>::kLanes, RI = RowLanes<D>::kRows;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane / LR, lr = lane % LR, c0 = lr * 8;
  const int tasks = a.q_tasks + a.kv_tasks;
  const int task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (task >= a.b.n_tokens * tasks) return;
  const int i = task / tasks, part = task - i * tasks;
  const bool query = part < a.q_tasks;
  const int r0 = (query ? part : part - a.q_tasks) * a.per, rows = query ? a.hq : 2 * a.c.hkv;
  const int r1 = min(r0 + a.per, rows);
  auto where = [&](int r, const void*& src) {   // element of channel 0
    const bool key = r < a.c.hkv;
    const sffn_rows& s = query ? a.q : key ? a.k : a.v;
    src = s.ptr;
    return (size_t)(i * s.row_stride + (query ? r : key ? r : r - a.c.hkv) * s.head_stride);
  };
  float nx[8];
  const void* nsrc = nullptr;
  size_t nat = 0;
  auto fetch = [&](int r) {
    if (r < r1) {
      nat = where(r, nsrc);
      ld_run<8>(nsrc, nat + c0, a.dtype, nx);
    }
  };
#pragma unroll
  for (int e = 0; e < 8; ++e) nx[e] = 0.f;
  fetch(r0 + sub);
  const KvPlace at = kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  Turn<D> turn;
  if (a.rope.table && (query || r0 < a.c.hkv)) {
    const int pos = a.rope.positions ? ld_dep(a.rope.positions + i) : at.pos;
    if (pos >= 0 && pos < a.rope.length)
      turn.set(a.rope, pos, lane);
    else if (a.rope.positions || pos >= 0)
      set_device_error(a.c.err, SFFN_ERR_DEVICE);
  }
  int page = -1;
  if (!query) {
    if (at.pos < 0) return;
    page = kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err);
    if (page < 0) return;
  }
  const int slot = query ? 0 : at.pos % a.c.P;
  const int glanes = LR / a.c.n_groups, grp = lr / glanes;
  const unsigned group_mask = (glanes == 32 ? 0xffffffffu : (1u << glanes) - 1u) << (lane / glanes * glanes);

  for (int r = r0 + sub; r - sub < r1; r += RI) {
    float x[8];
    const void* src = nsrc;
    const size_t elem = nat;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = nx[e];
    fetch(r + RI);
    const bool in = r < r1;
    turn.apply(a.rope, x, src, elem, a.dtype, lane, in && (query || r < a.c.hkv));
    if (query) {
      if (in) st_run<8>(a.q_out.ptr, (size_t)(i * a.q_out.row_stride + r * a.q_out.head_stride) + c0, a.dtype, x);
      continue;
    }
    // least and largest value of the group, over the lanes that share it
    float lo = x[0], hi = x[0], nan = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      nan = fmaf(x[e], 0.f, nan);   // NaN if a value is not finite
    }
    for (int o = 1; o < glanes; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(SFFN_FULL_MASK, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(SFFN_FULL_MASK, hi, o));
    }
    const bool bad = (__ballot_sync(SFFN_FULL_MASK, nan != 0.f) & group_mask) != 0u;
    const float m = __fadd_rn(__fmul_rn(lo, 0.5f), __fmul_rn(hi, 0.5f));
    __half mid = __float2half_rn(fminf(fmaxf(m, -kHalfMax), kHalfMax));
    const float midf = __half2float(mid);
    const float far = fmaxf(__fsub_rn(hi, midf), __fsub_rn(midf, lo));
    __half step = __float2half_rn(fminf(__fmul_rn(far, 1.f / 15.f), kHalfMax));
    if (bad) mid = __ushort_as_half(0), step = __ushort_as_half(0x7fff);
    const float stepf = __half2float(step), inv = __frcp_rn(__fmul_rn(2.f, stepf));
    // floor and limits of (x - mid) inv + 8: limits first, then 2^23 + t cut off at the units, whose bit pattern is
    // 0x4b000000 + floor(t); the eight of them are added up with their shifts and the constant taken off at the end
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = __fadd_rn(__fmul_rn(__fsub_rn(x[e], midf), inv), 8.f);
      codes += __float_as_uint(__fadd_rz(fminf(fmaxf(t, 0.f), 15.f), 8388608.f)) << (4 * e);
    }
    codes -= 0x4b000000u * 0x11111111u;
    if (stepf == 0.f || bad) codes = 0x88888888u;
    const bool value = r >= a.c.hkv;
    const uint32_t turned = __any_sync(SFFN_FULL_MASK, value) ? transpose_codes(codes, lane) : 0u;
    if (in) {
      const int h = value ? r - a.c.hkv : r;
      uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)h * a.c.head_bytes;
      uint8_t* row = block + (value ? kv_value_off(a.c.P, D) : 0) + slot * (D / 2);
      const int off = value ? value_word_off<D>(slot, lr & 7, lr >> 3) : key_word_off<D>(slot, lr & 3, lr >> 2);
      *reinterpret_cast<uint32_t*>(row + off) = value ? value_word(turned) : key_word(codes);
      if (lr % glanes == 0)
        *reinterpret_cast<__half2*>(block + kv_param_off(a.c.P, D) + param_off(slot, grp, a.c.n_groups, value)) =
            __halves2half2(step, mid);
    }
  }
}

struct GatherArgs {
  CacheView c;
  sffn_kv_batch b;
  sffn_rows k, v;
  int dtype;
  int per, tasks;   // rows of a task, tasks of a token
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_gather(const GatherArgs a) {
  constexpr int LR = RowLanes<D>::kLanes, RI = RowLanes<D>::kRows, kBatch = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane / LR, lr = lane % LR;
  const int task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (task >= a.b.n_tokens * a.tasks) return;
  const int i = task / a.tasks, r0 = (task - i * a.tasks) * a.per, r1 = min(r0 + a.per, 2 * a.c.hkv);
  const KvPlace at = kv_place(a.b, i, lane, a.c.P, a.c.err);
  if (at.seq < 0) return;
  const int page = at.pos >= 0 ? max(0, kv_page(a.b, at.seq, at.pos / a.c.P, a.c.n_pages, a.c.err)) : 0;
  const int slot = at.pos >= 0 ? at.pos % a.c.P : 0, grp = lr / (LR / a.c.n_groups);
  for (int rb = r0; rb < r1; rb += RI * kBatch) {
    uint32_t w[kBatch], pm[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = rb + k * RI + sub;
      w[k] = pm[k] = 0u;
      if (r < r1 && at.pos >= 0) {
        const bool value = r >= a.c.hkv;
        const uint8_t* block = a.c.pages + (size_t)page * a.c.page_bytes + (size_t)(value ? r - a.c.hkv : r) * a.c.head_bytes;
        const uint8_t* row = block + (value ? kv_value_off(a.c.P, D) : 0) + slot * (D / 2);
        const int off = value ? value_word_off<D>(slot, lr & 7, lr >> 3) : key_word_off<D>(slot, lr & 3, lr >> 2);
        w[k] = __ldcg(reinterpret_cast<const uint32_t*>(row + off));
        pm[k] = __ldcg(reinterpret_cast<const uint32_t*>(block + kv_param_off(a.c.P, D) +
                                                         param_off(slot, grp, a.c.n_groups, value)));
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = rb + k * RI + sub;
      const bool value = r >= a.c.hkv;
      const uint32_t turned = __any_sync(SFFN_FULL_MASK, value) ? transpose_codes(value_codes(w[k]), lane) : 0u;
      const uint32_t codes = value ? turned : key_codes(w[k]);
      const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pm[k]));
      float x[8];
      // 2u - 15 from the bit pattern of 2^23 + 2u; its product with step is exact in fp32 (a 4-bit by an 11-bit
      // number), so there is one rounding
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u2 = e == 0 ? codes << 1 : codes >> (4 * e - 1);
        x[e] = __fmaf_rn(__uint_as_float((u2 & 30u) | 0x4b000000u) - 8388623.f, sm.x, sm.y);
        if (at.pos < 0) x[e] = 0.f;
      }
      const sffn_rows& dst = value ? a.v : a.k;
      if (r < r1 && dst.ptr)
        st_run<8>(dst.ptr, (size_t)(i * dst.row_stride + (value ? r - a.c.hkv : r) * dst.head_stride) + lr * 8, a.dtype, x);
    }
  }
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
  const int kv = 2 * a.c.hkv, at_once = 32 / (C.desc.head_dim / 8);
  a.per = rows_per_task((long long)b.n_tokens * (a.hq + kv), std::max(a.hq, kv), at_once, C.num_sms);
  a.q_tasks = (a.hq + a.per - 1) / a.per;
  a.kv_tasks = (kv + a.per - 1) / a.per;
  const long long tasks = (long long)b.n_tokens * (a.q_tasks + a.kv_tasks);
  return by_dim(C.desc.head_dim, [&](auto d) {
    return launch_ex(k_kv_append<decltype(d)::value>, dim3((unsigned)((tasks + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                     0, st, true, 1, a);
  });
}

cudaError_t launch_kv_gather(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& k_out, const sffn_rows& v_out,
                             int dtype, cudaStream_t st) {
  GatherArgs a{view_of(C), b, k_out, v_out, dtype, 0, 0};
  const int kv = 2 * a.c.hkv, at_once = 32 / (C.desc.head_dim / 8);
  a.per = rows_per_task((long long)b.n_tokens * kv, kv, at_once, C.num_sms);
  a.tasks = (kv + a.per - 1) / a.per;
  const long long tasks = (long long)b.n_tokens * a.tasks;
  return by_dim(C.desc.head_dim, [&](auto d) {
    return launch_ex(k_kv_gather<decltype(d)::value>, dim3((unsigned)((tasks + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                     0, st, true, 1, a);
  });
}

}  // namespace sffn
