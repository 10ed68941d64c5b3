// Element access of activation arrays whose type is known only at run time
// (sffn_dtype), always as fp32 in registers.
#pragma once

#include "common.cuh"

namespace sffn {

__device__ __forceinline__ float ld_elem(const void* p, size_t i, int dtype) {
  if (dtype == SFFN_F32) return __ldcg(static_cast<const float*>(p) + i);
  const unsigned short h = __ldcg(static_cast<const unsigned short*>(p) + i);
  return dtype == SFFN_F16 ? __half2float(__ushort_as_half(h)) : __uint_as_float((uint32_t)h << 16);
}

__device__ __forceinline__ void st_elem(void* p, size_t i, float v, int dtype) {
  if (dtype == SFFN_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == SFFN_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// N consecutive elements (N * element size a multiple of 4 bytes, aligned to
// the largest power of two up to 16 that divides it).
template <int N>
__device__ __forceinline__ void ld_run(const void* p, size_t i, int dtype, float* o) {
  if (dtype == SFFN_F32) {
    const float* q = static_cast<const float*>(p) + i;
    if (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + k));
        o[k] = v.x, o[k + 1] = v.y, o[k + 2] = v.z, o[k + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(q + k));
        o[k] = v.x, o[k + 1] = v.y;
      }
    }
  } else {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const unsigned short*>(p) + i);
    uint32_t w[N / 2];
    if (N % 8 == 0) {
#pragma unroll
      for (int k = 0; k < N / 2; k += 4) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(q + k));
        w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
      }
    } else if (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N / 2; k += 2) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(q + k));
        w[k] = v.x, w[k + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) w[k] = __ldcg(q + k);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      if (dtype == SFFN_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        o[2 * k] = f.x, o[2 * k + 1] = f.y;
      } else {
        o[2 * k] = __uint_as_float(w[k] << 16), o[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void st_run(void* p, size_t i, int dtype, const float* v) {
  if (dtype == SFFN_F32) {
    float* q = static_cast<float*>(p) + i;
    if (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(q + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 2) *reinterpret_cast<float2*>(q + k) = make_float2(v[k], v[k + 1]);
    }
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      if (dtype == SFFN_F16) {
        const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint32_t* q = reinterpret_cast<uint32_t*>(static_cast<unsigned short*>(p) + i);
    if (N % 8 == 0) {
#pragma unroll
      for (int k = 0; k < N / 2; k += 4) *reinterpret_cast<uint4*>(q + k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
    } else if (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N / 2; k += 2) *reinterpret_cast<uint2*>(q + k) = make_uint2(w[k], w[k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) q[k] = w[k];
    }
  }
}

}  // namespace sffn
