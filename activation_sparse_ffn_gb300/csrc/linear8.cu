// Linear layer with 8-bit codes for rows of 8-bit codes: packing, the choice of
// the kernel, and the kernel for few tokens (k_lin8_few).
//
// k_lin8_few: a cluster of blocks takes a run of rows (any number of them: equal
// shares to a row) and its blocks split the inputs, as do the 16 warps of a
// block, so that every code is read once, straight into the registers of the
// lane that needs it, and a token's codes are held once. A warp takes two or
// three tiles of 16 rows at a time, so that it widens a token's codes once for
// all of them. Sums leave the tensor cores as whole numbers and meet in shared
// memory, where the order of additions does not matter.
//
// Measured: 10240 x 8192 for 16 tokens about 20 us, 4.2 TB/s of codes; widening and
// address arithmetic (38% of issue slots) and the waits for codes that four warps a
// scheduler do not cover. 4099 x 11008 for five 11 us, 4096 x 4096 for one 6 us, of
// which a wave's beginning and end are five.
#include <algorithm>

#include "linear8.cuh"
#include "linear8_split.h"
#include "q4mma.cuh"
#include "rows_io.cuh"
#include "step.h"

namespace sffn {

namespace {

// One thread per 16-byte chunk of the packed codes.
__global__ void k_pack_codes8(const int8_t* codes, uint4* out, int n, int k, int kb, size_t chunks) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= chunks) return;
  const int in = (int)(i % (kL8Block / 16)), r = in / 4, t = (in & 3) ^ ((r >> 1) & 3);
  const size_t block = i / (kL8Block / 16);
  const int row = (int)(block / kb) * kL8Rows + r, col = (int)(block % kb) * kL8Inputs + t * 16;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (row < n && col < k) v = *reinterpret_cast<const uint4*>(codes + (size_t)row * k + col);   // k is a multiple of 16
  out[i] = make_uint4(v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u);
}

__global__ void k_pack_rows8(const float* in, float* out, int n, int np) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < np) out[i] = in && i < n ? in[i] : 0.f;
}

constexpr int kFewWarps = 16, kFewThreads = kFewWarps * 32;

struct Lin8Args {
  const uint8_t* codes;
  const float* scales;
  const float* bias;
  sffn_rows x, residual, y;
  const float* x_scales;
  int n, k, kb, B, dtype, clusters;
  int x_stride, off_sum;   // bytes of a token's codes held by a block, and where the sums begin
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster_int(uint32_t smem_addr, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Four stored codes u = c + 128 as four halves u 2^-24: a byte alone in a half is a subnormal number.
__device__ __forceinline__ void small_halves(uint32_t u, uint32_t& lo, uint32_t& hi) {
  lo = __byte_perm(u, 0, 0x4140), hi = __byte_perm(u, 0, 0x4342);
}

// NT column tiles of eight tokens, RT row tiles of 16 at a time, whose inputs are widened once for all of them. Codes of
// rows are widened to u 2^-24, which takes half of what c takes, and 128 times the sum of a token's codes is taken off at
// the end: a product is below 2^15, so that 512 inputs are summed exactly.
template <int NT, int RT>
__global__ void __launch_bounds__(kFewThreads, 1) k_lin8_few(const Lin8Args a, int cs) {
  constexpr int kAhead = NT == 1 ? 5 : 2, kExactBlocks = 512 / kL8Inputs;   // steps of codes that a lane has on their way
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int x_sum[8 * NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / cs;
  const int row0 = (int)((long long)a.n * cluster / a.clusters), row1 = (int)((long long)a.n * (cluster + 1) / a.clusters);
  const int kb0 = (int)((long long)a.kb * rank / cs), kb1 = (int)((long long)a.kb * (rank + 1) / cs);
  const int wk0 = kb0 + (kb1 - kb0) * warp / kFewWarps, wk1 = kb0 + (kb1 - kb0) * (warp + 1) / kFewWarps;
  const int tiles = (row1 - row0 + 15) / 16, nk = wk1 - wk0, groups = (tiles + RT - 1) / RT;
  int* sums = reinterpret_cast<int*>(smem + a.off_sum);   // [row][8 NT]

  pdl_launch_dependents();
  // a step: the rows of a group of tiles, 64 inputs; the first are on their way before the wait (codes are packed by a call
  // that synchronizes)
  uint4 next[kAhead][RT][2];
  const int tile_first = row0 / kL8Rows;
  const uint8_t* codes = a.codes + ((size_t)tile_first * a.kb + wk0) * kL8Block;
  const int per = tiles / max(groups, 1), rest = tiles - per * groups;   // tiles of a group; the first `rest` have one more
  int place[RT][2];      // of the lane's rows of the group that is fetched, from `codes` on; -1: none
  int fleft = 0, fgroup = -1, frow = row0, fstep = 0;   // steps left of it; its number; rows after it; bytes of the steps before
  auto fetch = [&](uint4 (*f)[2]) {
    if (fleft == 0) {
      const int count = ++fgroup < groups ? per + (fgroup < rest) : 0;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = frow + r * 16 + h * 8 + g;
          place[r][h] = r < count && row < row1
                            ? (row / kL8Rows - tile_first) * a.kb * kL8Block + l8_chunk(row % kL8Rows, t) : -1;
        }
      frow += count * 16, fleft = nk, fstep = 0;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (place[r][h] >= 0) f[r][h] = ldg_stream(codes + (uint32_t)(place[r][h] + fstep));
    --fleft, fstep += kL8Block;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int r = 0; r < RT; ++r) next[i][r][0] = next[i][r][1] = make_uint4(0, 0, 0, 0);
  if (nk) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(next[i]);
  }
  for (int i = tid; i < (row1 - row0) * 8 * NT; i += kFewThreads) sums[i] = 0;
  if (tid < 8 * NT) x_sum[tid] = 0;
  __syncthreads();
  pdl_wait();
  // a chunk of 16 bytes of every token a thread, eight on their way together
  const int own = (kb1 - kb0) * 4;   // chunks of a token
  for (int c0 = 0; c0 < own; c0 += kFewThreads) {
    const int c = c0 + tid, col = kb0 * kL8Inputs + c * 16;
    const int8_t* src = static_cast<const int8_t*>(a.x.ptr) + col;
#pragma unroll
    for (int b0 = 0; b0 < 8 * NT; b0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (b0 + i < a.B && c < own && col < a.k)
          v[i] = __ldcg(reinterpret_cast<const uint4*>(src + (b0 + i) * a.x.row_stride));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c < own)
          *reinterpret_cast<uint4*>(smem + (b0 + i) * a.x_stride + c * 16) =
              make_uint4(v[i].x ^ 0x80808080u, v[i].y ^ 0x80808080u, v[i].z ^ 0x80808080u, v[i].w ^ 0x80808080u);
        const int ones = 0x01010101;
        int p = __dp4a((int)v[i].x, ones, __dp4a((int)v[i].y, ones, __dp4a((int)v[i].z, ones, __dp4a((int)v[i].w, ones, 0))));
        p = __reduce_add_sync(SFFN_FULL_MASK, p);
        if (lane == 0 && b0 + i < a.B) atomicAdd(&x_sum[b0 + i], p);
      }
    }
  }
  __syncthreads();

  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][c][e] = 0.f;
  int group = 0, kk = 0, first = 0, count = per + (0 < rest);
  const uint8_t* xs = smem + (wk0 - kb0) * kL8Inputs + t * 16 + g * a.x_stride;
  auto leave = [&]() {   // sums of a group of tiles, to those of the other warps
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (first + r) * 16 + g + 8 * (e >> 1);
          if (r < count && row < row1 - row0)
            atomicAdd(&sums[row * 8 * NT + c * 8 + 2 * t + (e & 1)], __float2int_rn(acc[r][c][e] * 0x1p24f));
          acc[r][c][e] = 0.f;
        }
  };
  const int steps = groups * nk;
  for (int u = 0; u < steps; u += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u + i < steps) {
        uint32_t xf[NT][4][2];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const uint4 xv = *reinterpret_cast<const uint4*>(xs + kk * kL8Inputs + c * 8 * a.x_stride);
          l8_halves(xv.x, xf[c][0][0], xf[c][0][1]), l8_halves(xv.y, xf[c][1][0], xf[c][1][1]);
          l8_halves(xv.z, xf[c][2][0], xf[c][2][1]), l8_halves(xv.w, xf[c][3][0], xf[c][3][1]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r >= count) break;
          const uint4 w0 = next[i][r][0], w1 = next[i][r][1];
          const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t af[4];   // rows g, g + 8; inputs 16 t + 4 s + (0, 1), then (2, 3)
            small_halves(wa[s], af[0], af[2]);
            small_halves(wb[s], af[1], af[3]);
#pragma unroll
            for (int c = 0; c < NT; ++c) mma_f16(acc[r][c], af, xf[c][s][0], xf[c][s][1]);
          }
        }
        fetch(next[i]);
        ++kk;
        if (kk == nk || kk % kExactBlocks == 0) {
          leave();
          if (kk == nk) kk = 0, first += count, ++group, count = per + (group < rest);
        }
      }
    }
  }
  if (cs > 1) cluster_barrier(); else __syncthreads();
  // outputs, a share of the rows for each block of the cluster
  const int rows = row1 - row0, from = rows * rank / cs, to = rows * (rank + 1) / cs, mine = to - from;
  const uint32_t base = smem_u32(sums);
  for (int i = tid; i < mine * a.B; i += kFewThreads) {
    const int b = i / mine, r = from + i - b * mine, row = row0 + r;
    int s = 0;
    if (cs > 1) {
      for (int k = 0; k < cs; ++k)
        s += ld_cluster_int(base + (r * 8 * NT + b) * 4, k) - 128 * ld_cluster_int(smem_u32(x_sum + b), k);
    } else {
      s = sums[r * 8 * NT + b] - 128 * x_sum[b];
    }
    float v = l8_value(s, a.scales[row], __ldcg(a.x_scales + b), a.bias[row]);
    if (a.residual.ptr) v = __fadd_rn(v, ld_elem(a.residual.ptr, b * a.residual.row_stride + row, a.dtype));
    st_elem(a.y.ptr, b * a.y.row_stride + row, v, a.dtype);
  }
  if (cs > 1) cluster_barrier();   // sums are read by the others until here
}

template <int NT, int RT>
cudaError_t run_few(const Lin8Args& a, int cs, int smem, cudaStream_t st) {
  return launch_ex(k_lin8_few<NT, RT>, dim3(a.clusters * cs), dim3(kFewThreads), smem, st, true, cs, a, cs);
}

// Up to 32 tokens.
cudaError_t launch_few(const sffn_linear8& L, Lin8Args a, cudaStream_t st) {
  const L8Few p = l8_few(a.n, L.kp, a.B, L.num_sms);
  if (p.smem > kL8FewSmem) return cudaErrorInvalidConfiguration;   // not with l8_few_tokens
  a.clusters = p.clusters, a.x_stride = p.x_stride, a.off_sum = p.off_sum;
  return p.nt == 1   ? run_few<1, 2>(a, p.cs, p.smem, st)
         : p.nt == 2 ? run_few<2, 3>(a, p.cs, p.smem, st)
                     : run_few<4, 2>(a, p.cs, p.smem, st);
}

}  // namespace

sffn_status pack_linear8(sffn_linear8& L, const int8_t* codes, const float* scales, const float* bias, cudaStream_t st) {
  const int kb = L.kp / kL8Inputs, np = L.tiles * kL8Rows;
  const size_t chunks = (size_t)L.tiles * kb * (kL8Block / 16);
  L.packed = false;
  k_pack_codes8<<<(unsigned)((chunks + 255) / 256), 256, 0, st>>>(codes, reinterpret_cast<uint4*>(L.codes),
                                                                  L.desc.out_features, L.desc.in_features, kb, chunks);
  k_pack_rows8<<<(np + 255) / 256, 256, 0, st>>>(scales, L.scales, L.desc.out_features, np);
  k_pack_rows8<<<(np + 255) / 256, 256, 0, st>>>(bias, L.bias, L.desc.out_features, np);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "sffn_linear8_pack");
  L.packed = true;
  return SFFN_OK;
}

cudaError_t configure_linear8_kernels(sffn_linear8& L) {
  int optin = 0;
  cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, L.device);
  if (e == cudaSuccess) e = set_dynamic_smem_max(k_lin8_few<1, 2>, optin);
  if (e == cudaSuccess) e = set_dynamic_smem_max(k_lin8_few<2, 3>, optin);
  if (e == cudaSuccess) e = set_dynamic_smem_max(k_lin8_few<4, 2>, optin);
  if (e == cudaSuccess) e = configure_linear8_tc(L);
  return e;
}

size_t linear8_ws_bytes(const sffn_linear8& L, int B) { return B > kL8FewTokens ? linear8_tc_ws_bytes(L, B) : 0; }

cudaError_t launch_linear8(const sffn_linear8& L, const sffn_rows& x, const float* x_scales, int B,
                           const sffn_rows& residual, const sffn_rows& y, int dtype, void* ws, cudaStream_t st) {
  if (B > kL8FewTokens) return launch_linear8_tc(L, x, x_scales, B, residual, y, dtype, ws, st);
  Lin8Args a = {};
  a.codes = L.codes, a.scales = L.scales, a.bias = L.bias, a.n = L.desc.out_features, a.k = L.desc.in_features;
  a.kb = L.kp / kL8Inputs, a.dtype = dtype;
  const int elem = dtype == SFFN_F32 ? 4 : 2;
  const int most = l8_few_tokens(a.n, L.kp, L.num_sms);
  for (int b = 0; b < B; b += most) {
    a.B = std::min(most, B - b);
    a.x = x, a.y = y, a.residual = residual, a.x_scales = x_scales + b;
    a.x.ptr = static_cast<int8_t*>(x.ptr) + b * x.row_stride;
    a.y.ptr = static_cast<uint8_t*>(y.ptr) + b * y.row_stride * elem;
    if (residual.ptr) a.residual.ptr = static_cast<uint8_t*>(residual.ptr) + b * residual.row_stride * elem;
    const cudaError_t e = launch_few(L, a, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sffn
