// Host-side internals of the attention half of a decode step: the 4-bit
// linear layer, the paged 4-bit key/value cache, and their launchers.
#pragma once

#include "internal.h"

struct sffn_linear {
  sffn_linear_desc desc;
  int device = 0;
  int num_sms = 0;
  bool packed = false;
  int kp = 0;            // in_features rounded up to 128
  int tiles = 0;         // 16-row tiles of out_features, an even number
  uint32_t* codes = nullptr;   // [tiles][kp / 64][128 words], see linear.cu
  void* scales = nullptr;      // [tiles][kp / 128][8][128 / group][2] in scale_dtype
  void* zeros = nullptr;       // the same shape, or null
  float* bias = nullptr;       // [tiles * 16], zeros if none was given
  uint32_t* err = nullptr;
  // clusters of 1, 2, 4 and 8 blocks that the GPU holds, by column tiles (1, 2, 4, 8) and shared memory (linear.cuh)
  int fit_small[4][4] = {}, fit_large[4][4] = {};
};

struct sffn_kv {
  sffn_kv_desc desc;
  int device = 0;
  int num_sms = 0;
  size_t head_bytes = 0;   // one page of one head
  size_t page_bytes = 0;   // one page of every head
  uint8_t* pages = nullptr;
  uint32_t* err = nullptr;
};

namespace sffn {

sffn_status pack_linear(sffn_linear& L, const int8_t* codes, const void* scales, const void* zeros, const float* bias,
                        cudaStream_t st);
cudaError_t configure_linear_kernels(sffn_linear& L);
size_t linear_ws_bytes(const sffn_linear& L, int B);
cudaError_t launch_linear(const sffn_linear& L, const sffn_rows& x, int B, const sffn_rows& residual,
                          const sffn_rows& y, int dtype, void* ws, cudaStream_t st);

cudaError_t launch_kv_append(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                             const sffn_rows& k, const sffn_rows& v, const sffn_rows& q_out, const sffn_rope& rope,
                             int dtype, cudaStream_t st);
cudaError_t launch_kv_gather(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& k_out, const sffn_rows& v_out,
                             int dtype, cudaStream_t st);

cudaError_t configure_attend_kernels(const sffn_kv& C);
size_t attend_ws_bytes(const sffn_kv& C, int n_q_heads, int n_seq, int n_tokens);
cudaError_t launch_attend(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                          const sffn_rows& out, float* lse, float scale, int window, int dtype, void* ws,
                          cudaStream_t st);

}  // namespace sffn
