// Host-side internals of what stands around the halves of a decode step: the
// norm with 8-bit rows, the 8-bit linear layer, the choice of continuations
// and the reordering of the cache.
#pragma once

#include "attn.h"

struct sffn_linear8 {
  sffn_linear8_desc desc;
  int device = 0;
  int num_sms = 0;
  bool packed = false;
  int kp = 0;             // in_features rounded up to 128
  int tiles = 0;          // 128-row tiles of out_features
  uint8_t* codes = nullptr;   // [tiles][kp / 64][128][64 bytes], see linear8.cu
  float* scales = nullptr;    // [tiles * 128], zeros beyond out_features
  float* bias = nullptr;      // the same, zeros if none was given
  uint32_t* err = nullptr;
};

struct sffn_beam {
  sffn_beam_desc desc;
  int device = 0;
  int num_sms = 0;
  uint32_t* err = nullptr;
};

namespace sffn {

struct NormArgs {
  sffn_rows x, residual, sum, y, codes;
  const float* weight;
  float* scales;
  double eps;
  int rows, width, dtype, y_dtype;
  bool norm;   // false: the rows as they are
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);

sffn_status pack_linear8(sffn_linear8& L, const int8_t* codes, const float* scales, const float* bias, cudaStream_t st);
cudaError_t configure_linear8_kernels(sffn_linear8& L);
cudaError_t configure_linear8_tc(const sffn_linear8& L);
size_t linear8_tc_ws_bytes(const sffn_linear8& L, int B);
cudaError_t launch_linear8_tc(const sffn_linear8& L, const sffn_rows& x, const float* x_scales, int B,
                              const sffn_rows& residual, const sffn_rows& y, int dtype, void* ws, cudaStream_t st);
size_t linear8_ws_bytes(const sffn_linear8& L, int B);
cudaError_t launch_linear8(const sffn_linear8& L, const sffn_rows& x, const float* x_scales, int B,
                           const sffn_rows& residual, const sffn_rows& y, int dtype, void* ws, cudaStream_t st);

size_t beam_ws_bytes(const sffn_beam& H, int batch);
cudaError_t launch_beam(const sffn_beam& H, const sffn_rows& logits, const float* scores, const uint8_t* done,
                        int end_token, int batch, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                        int dtype, void* ws, cudaStream_t st);

constexpr int kMaxCaches = 128;   // of one sffn_kv_reorder
cudaError_t launch_kv_reorder(const sffn_kv* const* kvs, int n_kv, const sffn_kv_batch& b, const int32_t* parents,
                              int beams, int32_t* table_out, int out_stride, cudaStream_t st);

}  // namespace sffn
