// Linear layer with 4-bit codes and group scales, for 1 to 32 tokens.
//
// Codes are packed once into blocks of 16 rows x 64 inputs, 512 bytes each, so
// that a warp (lane = 4 g + t) takes a block with one 16-byte load per lane:
// words (row g, inputs 8t..8t+7 of the first 32), (row g + 8, the same),
// (row g, of the second 32), (row g + 8, the same). In a word, the codes of
// inputs 2e and 2e + 1 of its eight stand at bits 4e of the two halves
// (e = 0, 1 as they are, e = 2, 3 after a shift by 8: two bits of a half apart by
// four, which is all that linear.cuh has to undo). Rows and
// inputs are padded with code 0 (stored as 8), to an even number of tiles and to
// 128 inputs.
#include <algorithm>

#include "linear.cuh"

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

// Scales or zeros, 16- or 32-bit words: [tile][step of 128 inputs][8][128 / G][2], rows g and g + 8 beside each other.
template <typename T>
__global__ void k_pack_groups(const T* in, T* out, int n, int groups, int per_step, int steps, int tiles) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (size_t)tiles * steps * per_step * 16) return;
  const int half = (int)(i % 2), q = (int)(i / 2 % per_step), g = (int)(i / 2 / per_step % 8);
  const size_t st = i / 16 / per_step;
  const int step = (int)(st % steps), tile = (int)(st / steps), row = tile * 16 + g + 8 * half, grp = step * per_step + q;
  out[i] = row < n && grp < groups ? in[(size_t)row * groups + grp] : T(0);
}

__global__ void k_pack_bias(const float* in, float* out, int n, int np) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < np) out[i] = in && i < n ? in[i] : 0.f;
}

int column_tiles(int B, int dtype) {   // of eight columns, rounded up to a power of two
  const int cols = dtype == SFFN_F32 ? 2 * B : B;
  return cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 32 ? 4 : 8;
}

// What a cluster of 1, 2, 4 or 8 blocks costs, in bytes of codes an SM reads in that time: fitted on an earlier form of
// the kernels to 10240 x 8192 at one token, now 13.7, 12.7, 12.9 and 15.9 us (codes in L2), at 32 tokens 41.6, 34.8, 27.4
// and 52.4, at 4099 x 11008 with zeros and five 18.4, 15.3, 13.5 and 14.8. Of 17 sizes from 1024 x 1024 to 28672 x 8192,
// one to 32 tokens, the choice was the fastest or within 7% of it at eleven, 8 to 11% slower at five (8192 x 8192, one
// token: 11.7, two blocks 10.6) and 19% at one (2048 x 2048: 4.3, one block 3.6).
constexpr long long kClusterCost[4] = {0, 16 * 1024, 56 * 1024, 224 * 1024};

int scale_format(const sffn_linear& L) {
  return L.desc.scale_dtype == SFFN_F32 ? kScale32 : L.desc.has_zero ? kScale16Zero : kScale16;
}

}  // namespace

sffn_status pack_linear(sffn_linear& L, const int8_t* codes, const void* scales, const void* zeros, const float* bias,
                        cudaStream_t st) {
  const int n = L.desc.out_features, k = L.desc.in_features, groups = k / L.desc.group, per_step = 128 / L.desc.group;
  const size_t words = (size_t)L.tiles * (L.kp / 64) * 128, vals = (size_t)L.tiles * (L.kp / 128) * per_step * 16;
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
      k_pack_groups<uint32_t><<<blocks, 256, 0, st>>>((const uint32_t*)in, (uint32_t*)out, n, groups, per_step, L.kp / 128,
                                                 L.tiles);
    else
      k_pack_groups<uint16_t><<<blocks, 256, 0, st>>>((const uint16_t*)in, (uint16_t*)out, n, groups, per_step, L.kp / 128,
                                                 L.tiles);
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

cudaError_t configure_linear_kernels(sffn_linear& L) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
    LinearFit fit = {};
    const int nt = 1 << i, fmt = scale_format(L);
    e = L.desc.group == 32 ? prepare_linear_g32(nt, fmt, &fit)
                           : L.desc.group == 64 ? prepare_linear_g64(nt, fmt, &fit) : prepare_linear_g128(nt, fmt, &fit);
    for (int c = 0; c < 4; ++c) L.fit_small[i][c] = fit.small[c], L.fit_large[i][c] = fit.large[c];
  }
  return e;
}

namespace {

// x as halves, its scales and its sums over groups, for the kernel of more than eight columns.
struct LinearWs {
  size_t down, sum, total;
};
LinearWs linear_ws(const sffn_linear& L, int B, int dtype) {
  const int nt = column_tiles(B, dtype), cols = dtype == SFFN_F32 ? 2 * B : B;
  if (nt == 1) return LinearWs{0, 0, 0};
  LinearWs w;
  w.down = (size_t)cols * L.kp * 2;   // kp is a multiple of 128
  w.sum = w.down + 256;
  w.total = w.sum + (size_t)(L.kp / L.desc.group) * 8 * nt * sizeof(float);
  return w;
}

}  // namespace

size_t linear_ws_bytes(const sffn_linear& L, int B) { return linear_ws(L, B, SFFN_F32).total; }

cudaError_t launch_linear(const sffn_linear& L, const sffn_rows& x, int B, const sffn_rows& residual,
                          const sffn_rows& y, int dtype, void* ws, cudaStream_t st) {
  LinearArgs a = {};
  a.codes = L.codes, a.scales = L.scales, a.zeros = L.zeros, a.bias = L.bias, a.err = L.err;
  const LinearWs w = linear_ws(L, B, dtype);
  a.ws_x = static_cast<const __half*>(ws);
  a.ws_down = reinterpret_cast<const float*>(static_cast<const uint8_t*>(ws) + w.down);
  a.ws_sum = reinterpret_cast<const float*>(static_cast<const uint8_t*>(ws) + w.sum);
  a.n = L.desc.out_features, a.k = L.desc.in_features, a.kp = L.kp, a.B = B, a.dtype = dtype;
  a.sdtype = L.desc.scale_dtype, a.tiles = L.tiles, a.x = x, a.residual = residual, a.y = y;
  const int G = L.desc.group, steps = a.kp / 128;
  const int nt = column_tiles(B, dtype), nti = nt == 1 ? 0 : nt == 2 ? 1 : nt == 4 ? 2 : 3;
  const int cols = dtype == SFFN_F32 ? 2 * B : B, elems = 16 * B;
  auto up16 = [](int v) { return (v + 15) & ~15; };
  const int sum = 8 * nt * 4;   // bytes of the sums of a group of inputs
  int smem = 0, ci = 0;
  long long best = -1;
  if (nt == 1) {
    // The split of the inputs that gives a block the least to do, in bytes of codes that take as long: a cluster
    // costs two barriers and a pass over its sums; a run of 128 inputs of a token costs its warp 4 KB.
    for (int c = 0; c < 4; ++c) {
      const int slices = kLinWarps << c, own = (steps + slices - 1) / slices * 128;
      const int xbytes = up16(kLinWarps * cols * (own + 32) * 2) + kLinWarps * (own / G + 1) * sum;
      const int per_tile = (kLinWarps + 1) * elems * 4;
      for (int large = 0; large < 2; ++large) {
        const int room = (large ? kLinLarge : kLinSmall) - xbytes - 64;
        if (room < per_tile || (!large && room < 8 * per_tile)) continue;
        const int fit = std::max(1, large ? L.fit_large[0][c] : L.fit_small[0][c]);
        const int clusters = std::max(std::min(a.tiles, fit), (a.tiles + room / per_tile - 1) / (room / per_tile));
        const int most = (a.tiles + clusters - 1) / clusters, waves = (clusters + fit - 1) / fit;
        const long long cost = (long long)most * waves * own * kLinWarps * 8 * (large ? 1 : 2) + kClusterCost[c] +
                               (long long)(own / 128) * B * 4 * 1024;
        if (best >= 0 && cost >= best) break;
        best = cost, ci = c;
        a.clusters = clusters, a.chunk = own, a.chunk_stride = own + 32;
        a.off_sum = up16(kLinWarps * cols * a.chunk_stride * 2);
        a.off_part = up16(a.off_sum + kLinWarps * (own / G + 1) * sum);
        a.off_acc = a.off_part + most * kLinWarps * elems * 4;
        smem = a.off_acc + most * elems * 4;
        break;
      }
    }
  } else {
    // The split that gives an SM the least to read, among those that keep 40 KB of sums; chunks of x as large as
    // fit, since the loads in flight run dry between them, which costs about 64 KB. The warps' parts stand over x.
    const int warps = linear_warps(nt), rt = linear_tiles(nt), units = a.tiles / rt, uelems = rt * elems;
    const int most_units = std::max(1, 40 * 1024 / (uelems * 4));
    for (int c = 0; c < 4; ++c) {
      const int own = (steps + (1 << c) - 1) / (1 << c) * 128, fit = std::max(1, L.fit_large[nti][c]);
      const int clusters = std::max(std::min(units, fit), (units + most_units - 1) / most_units);
      const int most = (units + clusters - 1) / clusters, waves = (clusters + fit - 1) / fit;
      const int room = kLinLarge - most * uelems * 4 - 64;
      const int per128 = cols * 256 + 128 / G * sum, pad = cols * 64;
      const int runs = std::min(own / 128, (room - pad) / per128);
      if (runs < 1 || warps * uelems * 4 > room) continue;
      const int chunks = (own + runs * 128 - 1) / (runs * 128);
      const long long cost = ((long long)most * rt * 8 * own + chunks * 64 * 1024) * waves + kClusterCost[c];
      if (best >= 0 && cost >= best) continue;
      best = cost, ci = c;
      a.clusters = clusters, a.chunk = runs * 128, a.chunk_stride = a.chunk + 32;
      a.off_sum = up16(cols * a.chunk_stride * 2);
      a.off_acc = up16(std::max(a.off_sum + a.chunk / G * sum, warps * uelems * 4));   // parts stand where x stood
      smem = a.off_acc + most * uelems * 4;
    }
  }
  const int cs = 1 << ci, blocks = a.clusters * cs;
  const int fmt = scale_format(L);
  return G == 32 ? run_linear_g32(nt, fmt, cs, a, blocks, smem, st)
                 : G == 64 ? run_linear_g64(nt, fmt, cs, a, blocks, smem, st)
                           : run_linear_g128(nt, fmt, cs, a, blocks, smem, st);
}

}  // namespace sffn
