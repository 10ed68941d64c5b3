// Linear layer with 4-bit codes and group scales, for 1 to 32 tokens.
//
// Codes are packed once into blocks of 16 rows x 64 inputs, 512 bytes each, so
// that a warp (lane = 4 g + t) takes a block with one 16-byte load per lane:
// words (row g, inputs 8t..8t+7 of the first 32), (row g + 8, the same),
// (row g, of the second 32), (row g + 8, the same). In a word, the codes of
// inputs 2e and 2e + 1 of its eight stand at bits 4e of the two halves. Rows and
// inputs are padded with code 0 (stored as 8). Scales (and zeros) stand as
// [tile][group][8][2], rows g and g + 8 beside each other.
#include "attn.h"
#include "rows_io.cuh"

namespace sffn {

namespace {

__host__ __device__ __forceinline__ uint32_t weight_word(const uint8_t* u) {
  uint32_t w = 0;
  for (int e = 0; e < 4; ++e) w |= (uint32_t)u[2 * e] << (4 * e) | (uint32_t)u[2 * e + 1] << (16 + 4 * e);
  return w;
}

// One thread per word.
__global__ void k_pack_codes(const int8_t* codes, uint32_t* out, int n, int k, int kp, int tiles, uint32_t* err) {
  const size_t w = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const size_t per_tile = (size_t)(kp / 64) * 128;
  if (w >= per_tile * tiles) return;
  const int tile = (int)(w / per_tile), kb = (int)((w % per_tile) / 128), in = (int)(w % 128);
  const int lane = in / 4, j = in % 4, g = lane / 4, t = lane % 4;
  const int row = tile * 16 + g + 8 * (j & 1), col = kb * 64 + 32 * (j >> 1) + 8 * t;
  uint8_t u[8];
  bool bad = false;
  for (int e = 0; e < 8; ++e) {
    const int c = row < n && col + e < k ? codes[(size_t)row * k + col + e] : 0;
    bad |= c < -8 || c > 7;
    u[e] = (uint8_t)((c + 8) & 15);
  }
  if (bad) set_device_error(err, SFFN_ERR_DEVICE);
  out[w] = weight_word(u);
}

// Scales or zeros as 16- or 32-bit words.
template <typename T>
__global__ void k_pack_groups(const T* in, T* out, int n, int groups, int groups_p, int tiles) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (size_t)tiles * groups_p * 16) return;
  const int half = (int)(i % 2), g = (int)(i / 2 % 8), grp = (int)(i / 16 % groups_p), tile = (int)(i / 16 / groups_p);
  const int row = tile * 16 + g + 8 * half;
  out[i] = row < n && grp < groups ? in[(size_t)row * groups + grp] : T(0);
}

__global__ void k_pack_bias(const float* in, float* out, int n, int np) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < np) out[i] = in && i < n ? in[i] : 0.f;
}

struct LinearArgs {
  const uint32_t* codes;
  const void* scales;
  const void* zeros;
  const float* bias;
  int n, k, kp, group, sdtype, B, dtype;
  sffn_rows x, residual, y;
};

// One warp per (output, token).
__global__ void __launch_bounds__(128) k_linear(const LinearArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, n = blockIdx.x * 4 + (threadIdx.x >> 5), b = blockIdx.y;
  if (n >= a.n) return;
  const int tile = n / 16, r = n % 16, g = r % 8, half = r / 8, ngk = a.kp / a.group;
  float y = 0.f;
  for (int w = lane; w < a.k / 8; w += 32) {  // word: inputs 8w .. 8w + 7
    const int kb = w / 8, t = w % 4, second = (w / 4) & 1;
    const uint32_t c = __ldg(a.codes + ((size_t)tile * (a.kp / 64) + kb) * 128 + (g * 4 + t) * 4 + second * 2 + half);
    const size_t gi = (((size_t)tile * ngk + 8 * w / a.group) * 8 + g) * 2 + half;
    const float s = ld_elem(a.scales, gi, a.sdtype), z = a.zeros ? ld_elem(a.zeros, gi, a.sdtype) : 0.f;
    float v = 0.f;
    for (int e = 0; e < 8; ++e) {
      const float code = (float)((int)(c >> ((e & 1) * 16 + (e >> 1) * 4) & 15) - 8);
      v = fmaf(code - z, ld_elem(a.x.ptr, (size_t)(b * a.x.row_stride) + 8 * w + e, a.dtype), v);
    }
    y = fmaf(s, v, y);
  }
  y = warp_sum(y);
  if (lane == 0) {
    y += a.bias[n];
    if (a.residual.ptr) y += ld_elem(a.residual.ptr, (size_t)(b * a.residual.row_stride) + n, a.dtype);
    st_elem(a.y.ptr, (size_t)(b * a.y.row_stride) + n, y, a.dtype);
  }
}

}  // namespace

sffn_status pack_linear(sffn_linear& L, const int8_t* codes, const void* scales, const void* zeros, const float* bias,
                        cudaStream_t st) {
  const int n = L.desc.out_features, k = L.desc.in_features, groups = k / L.desc.group, gp = L.kp / L.desc.group;
  const size_t words = (size_t)L.tiles * (L.kp / 64) * 128, vals = (size_t)L.tiles * gp * 16;
  L.packed = false;
  cudaError_t e = cudaMemsetAsync(L.err, 0, 4, st);
  if (e != cudaSuccess) return cuda_fail(e, "sffn_linear_pack");
  k_pack_codes<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(codes, L.codes, n, k, L.kp, L.tiles, L.err);
  for (int which = 0; which < 2; ++which) {
    const void* in = which ? zeros : scales;
    void* out = which ? L.zeros : L.scales;
    if (!in) continue;
    const unsigned blocks = (unsigned)((vals + 255) / 256);
    if (L.desc.scale_dtype == SFFN_F32)
      k_pack_groups<uint32_t><<<blocks, 256, 0, st>>>((const uint32_t*)in, (uint32_t*)out, n, groups, gp, L.tiles);
    else
      k_pack_groups<uint16_t><<<blocks, 256, 0, st>>>((const uint16_t*)in, (uint16_t*)out, n, groups, gp, L.tiles);
  }
  k_pack_bias<<<(L.tiles * 16 + 255) / 256, 256, 0, st>>>(bias, L.bias, n, L.tiles * 16);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  uint32_t flag = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&flag, L.err, 4, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "sffn_linear_pack");
  if (flag) {
    set_error("sffn_linear_pack: a code lies outside [-8, 7]");
    return SFFN_ERR_DEVICE;
  }
  L.packed = true;
  return SFFN_OK;
}

cudaError_t configure_linear_kernels(const sffn_linear&) { return cudaSuccess; }

size_t linear_ws_bytes(const sffn_linear&, int) { return 0; }

cudaError_t launch_linear(const sffn_linear& L, const sffn_rows& x, int B, const sffn_rows& residual,
                          const sffn_rows& y, int dtype, void* ws, cudaStream_t st) {
  (void)ws;
  const LinearArgs a{L.codes, L.scales, L.zeros, L.bias, L.desc.out_features, L.desc.in_features, L.kp,
                     L.desc.group, L.desc.scale_dtype, B, dtype, x, residual, y};
  return launch_ex(k_linear, dim3((a.n + 3) / 4, B), dim3(128), 0, st, true, 1, a);
}

}  // namespace sffn
