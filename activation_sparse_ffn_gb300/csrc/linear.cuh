// The product kernel of the 4-bit linear layer, one instantiation per group
// size, number of 8-column tiles and scale format (linear_g*.cu).
//
// Mathematics. y[b][n] = sum over groups of s * (sum_k c x[b][k] - z sum_k
// x[b][k]). Weights are the 16-row operand of the tensor-core product: a code c
// = u - 8 becomes a half with one mask and one operation per pair (1024 + u -
// 1032 or (1024 + 16u) / 16 - 72, both exact), and scales and zeros are applied
// to the sums of a group in fp32. Codes go in centred although bare ones would
// cost nothing: the tensor core cuts its addends off at 2^-24 of the largest,
// and activations have large elements. Tokens are the 8-column operand,
// as halves: 16-bit activations exactly, up to a power of two per token and run
// of 128 inputs that brings the largest to 2^13; fp32 activations as two
// columns, the nearest half and the nearest half of what is left (22 bits).
//
// Work split. The codes are read once, straight to registers, with kAhead steps'
// loads in flight per warp, begun before the wait for the kernel that produces
// x. A cluster of blocks takes a run of 16-row tiles and its blocks split the
// inputs, so that a block converts only its share of x; their sums are added
// through distributed shared memory in rank order.
//   Up to eight columns (k_linear_few): the warps of a block split its inputs
// too, each goes over all tiles with the same share of x, which it converts for
// itself, and leaves one sum per tile and warp: no barrier before the end.
//   More columns (k_linear): those sums would not fit, so the (tile, run of
// inputs) steps are numbered through and each warp takes an equal run of them;
// x is converted once for all blocks by a small kernel before (k_linear_x),
// because every cluster would convert the same numbers again.
#pragma once

#include <type_traits>

#include "attn.h"
#include "q4mma.cuh"
#include "rows_io.cuh"

namespace sffn {

struct LinearArgs {
  const uint32_t* codes;
  const void* scales;
  const void* zeros;
  const float* bias;
  uint32_t* err;
  int n, k, kp, B, dtype, sdtype;
  int tiles;        // 16-row tiles
  int clusters, chunk, chunk_stride;   // inputs of x held at a time (a multiple of 128), halves of a row of xs
  int off_xg, off_acc, off_part;       // bytes in shared memory
  const __half* ws_x;    // k_linear: x as halves [columns][kp], and
  const float2* ws_xg;   // its (down, down * sum) pairs [groups][8 NT]
  sffn_rows x, residual, y;
};

constexpr int kLinWarps = 8;                   // of a block of k_linear_few
constexpr int kLinThreads = kLinWarps * 32;
// Of a block of k_linear: one block per SM, as many warps as 64 accumulators per thread leave registers for.
constexpr int linear_warps(int nt) { return nt == 8 ? 8 : 16; }

// Scale formats: 16-bit scales, 16-bit scales and zeros, 32-bit scales (and zeros if given).
enum { kScale16 = 0, kScale16Zero = 1, kScale32 = 2 };

// Shared-memory limits of the kernels of one number of column tiles, and how
// many clusters of 1, 2, 4 and 8 blocks the GPU holds with `small` and with
// `large` bytes each.
struct LinearFit {
  int small[4], large[4];
};
constexpr int kLinSmall = 100 * 1024, kLinLarge = 216 * 1024;

cudaError_t prepare_linear_g32(int nt, int fmt, LinearFit* fit);
cudaError_t prepare_linear_g64(int nt, int fmt, LinearFit* fit);
cudaError_t prepare_linear_g128(int nt, int fmt, LinearFit* fit);
cudaError_t run_linear_g32(int nt, int fmt, int cluster, const LinearArgs& a, int blocks, int smem, cudaStream_t st);
cudaError_t run_linear_g64(int nt, int fmt, int cluster, const LinearArgs& a, int blocks, int smem, cudaStream_t st);
cudaError_t run_linear_g128(int nt, int fmt, int cluster, const LinearArgs& a, int blocks, int smem, cudaStream_t st);

#ifdef SFFN_LINEAR_GROUP

namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t smem_addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// The code pairs u - 8 at bits 0-3 and 4-7 of both halves of a word.
__device__ __forceinline__ uint32_t weight_low(uint32_t w) {
  return h2_u32(__hadd2(code_bits(w, 0x000f000fu), u32_h2(0xe408e408u)));
}
__device__ __forceinline__ uint32_t weight_high(uint32_t w) {
  return h2_u32(__hfma2(code_bits(w, 0x00f000f0u), u32_h2(0x2c002c00u), u32_h2(0xd480d480u)));
}

template <int FMT>
struct ScaleWord {   // the scales (and zeros) of rows g and g + 8 as loaded
  static constexpr int N = FMT == kScale16 ? 1 : FMT == kScale16Zero ? 2 : 4;
  uint32_t w[N];
  // entry `at` of [..][8][2] arrays
  __device__ __forceinline__ void load(const LinearArgs& a, size_t at) {
    if (FMT == kScale32) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.scales) + at);
      uint2 z = make_uint2(0u, 0u);
      if (a.zeros) z = __ldg(reinterpret_cast<const uint2*>(a.zeros) + at);
      w[0] = v.x, w[1 % N] = v.y, w[2 % N] = z.x, w[3 % N] = z.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(a.scales) + at);
      if (FMT == kScale16Zero) w[1 % N] = __ldg(reinterpret_cast<const uint32_t*>(a.zeros) + at);
    }
  }
  __device__ __forceinline__ void get(int sdtype, float* sc, float* z) const {
    z[0] = z[1] = 0.f;
    if (FMT == kScale32) {
      sc[0] = __uint_as_float(w[0]), sc[1] = __uint_as_float(w[1 % N]);
      z[0] = __uint_as_float(w[2 % N]), z[1] = __uint_as_float(w[3 % N]);
    } else {
      two(w[0], sdtype, sc);
      if (FMT == kScale16Zero) two(w[1 % N], sdtype, z);
    }
  }
  __device__ __forceinline__ static void two(uint32_t v, int sdtype, float* o) {
    if (sdtype == SFFN_F16) {
      const float2 f = __half22float2(u32_h2(v));
      o[0] = f.x, o[1] = f.y;
    } else {
      o[0] = __uint_as_float(v << 16), o[1] = __uint_as_float(v & 0xffff0000u);
    }
  }
};

// y += one step: S inputs of a tile's codes c with their scales s, times the
// columns xcol[n] (this lane's column of each eight) at halves `at`, with the
// (down, down * sum) pairs of columns 2t, 2t + 1 of the step's groups at xq
// (xq_stride pairs from group to group).
template <int G, int NT, int FMT>
__device__ __forceinline__ void linear_step(const LinearArgs& a, const uint4* c, const ScaleWord<FMT>* s,
                                            const __half* const* xcol, int at, const float2* xq, float (*y)[4]) {
  constexpr int S = G > 64 ? G : 64, BL = S / 64;
  float d[NT][4];
#pragma unroll
  for (int b = 0; b < BL; ++b) {
    const uint32_t w[4] = {c[b].x, c[b].y, c[b].z, c[b].w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 32 inputs
      const uint32_t wa = w[2 * h], wb = w[2 * h + 1], ra = wa >> 8, rb = wb >> 8;
      const uint32_t a0[4] = {weight_low(wa), weight_low(wb), weight_high(wa), weight_high(wb)};
      const uint32_t a1[4] = {weight_low(ra), weight_low(rb), weight_high(ra), weight_high(rb)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xv = *reinterpret_cast<const uint4*>(xcol[n] + at + b * 64 + h * 32);
        if ((b * 64 + h * 32) % G == 0) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
        mma_f16(d[n], a0, xv.x, xv.y);
        mma_f16(d[n], a1, xv.z, xv.w);
      }
      if ((b * 64 + h * 32 + 32) % G == 0) {   // end of a group: scales
        const int q = (b * 64 + h * 32) / G;
        float sc[2], z[2];
        s[q].get(a.sdtype, sc, z);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 v = *reinterpret_cast<const float4*>(xq + q * (8 * NT) + 8 * n);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (FMT == kScale16) {
              y[n][2 * r] = fmaf(sc[r], d[n][2 * r] * v.x, y[n][2 * r]);
              y[n][2 * r + 1] = fmaf(sc[r], d[n][2 * r + 1] * v.z, y[n][2 * r + 1]);
            } else {
              y[n][2 * r] = fmaf(sc[r], fmaf(d[n][2 * r], v.x, -z[r] * v.y), y[n][2 * r]);
              y[n][2 * r + 1] = fmaf(sc[r], fmaf(d[n][2 * r + 1], v.z, -z[r] * v.w), y[n][2 * r + 1]);
            }
          }
        }
      }
    }
  }
}

// N runs of 128 inputs that one warp converts together, four inputs of each per
// lane, as halves: the nearest in hi, what is left in lo (fp32 rows only), both
// times a power of two that `down` undoes; f16 rows are taken as they are. With
// Sums, the sums of hi and lo over a group of G.
template <int G, int N, bool Sums>
__device__ __forceinline__ void convert_runs(const float (*v)[4], int dtype, uint32_t (*hi)[2], uint32_t (*lo)[2],
                                             float* sh, float* sl, float* down) {
  float up[N];
  if (dtype == SFFN_F16) {
#pragma unroll
    for (int i = 0; i < N; ++i) up[i] = down[i] = 1.f;
  } else {
    float big[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      big[i] = fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3])));
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) big[i] = fmaxf(big[i], __shfl_xor_sync(SFFN_FULL_MASK, big[i], o));
#pragma unroll
    for (int i = 0; i < N; ++i) scale_to_half_range(big[i], up[i], down[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) split_f16(v[i][2 * p] * up[i], v[i][2 * p + 1] * up[i], hi[i][p], lo[i][p]);
  if (Sums) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 a = __half22float2(u32_h2(hi[i][0])), b = __half22float2(u32_h2(hi[i][1]));
      const float2 c = __half22float2(u32_h2(lo[i][0])), d = __half22float2(u32_h2(lo[i][1]));
      sh[i] = (a.x + a.y) + (b.x + b.y);
      sl[i] = (c.x + c.y) + (d.x + d.y);
    }
#pragma unroll
    for (int o = 1; o < G / 4; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sh[i] += __shfl_xor_sync(SFFN_FULL_MASK, sh[i], o);
        sl[i] += __shfl_xor_sync(SFFN_FULL_MASK, sl[i], o);
      }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) sh[i] = sl[i] = 0.f;
  }
}

// The sums of a tile ([B][16]) from the fragments of one warp.
template <int NT>
__device__ __forceinline__ void store_tile(float* dst, const float (*y)[4], int B, bool split, bool add, int g, int t) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (split) {
        const int b = 4 * n + t;
        if (b < B) {
          float* p = dst + b * 16 + g + 8 * r;
          const float v = y[n][2 * r] + y[n][2 * r + 1];
          *p = add ? *p + v : v;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int b = 8 * n + 2 * t + c;
          if (b < B) {
            float* p = dst + b * 16 + g + 8 * r;
            *p = add ? *p + y[n][2 * r + c] : y[n][2 * r + c];
          }
        }
      }
    }
}

// Adds the sums acc_s (nt tiles, [B][16] each) of the cluster's blocks; every
// block writes a contiguous share of the outputs, four rows per thread.
__device__ __forceinline__ void write_outputs(const LinearArgs& a, const float* acc_s, int tile0, int nt, int cs, int rank,
                                              int threads) {
  const int quads = a.B * 4, all = nt * quads, share = (all + cs - 1) / cs;
  const uint32_t base = smem_u32(acc_s);
  if (cs > 1) cluster_barrier();
  for (int e = rank * share + threadIdx.x; e < min(all, (rank + 1) * share); e += threads) {
    const int tile = e / quads, in = e - tile * quads, b = in >> 2, n = (tile0 + tile) * 16 + (in & 3) * 4;
    float4 v = *reinterpret_cast<const float4*>(a.bias + n);   // padded to whole tiles
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.residual.ptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.n) r[i] = ld_elem(a.residual.ptr, (size_t)(b * a.residual.row_stride) + n + i, a.dtype);
    }
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (cs > 1) {
      float4 p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = k < cs ? ld_cluster(base + 16u * e, k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) s.x += p[k].x, s.y += p[k].y, s.z += p[k].z, s.w += p[k].w;
    } else {
      s = *reinterpret_cast<const float4*>(acc_s + 4 * e);
    }
    const float o[4] = {s.x + v.x + r[0], s.y + v.y + r[1], s.z + v.z + r[2], s.w + v.w + r[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n) st_elem(a.y.ptr, (size_t)(b * a.y.row_stride) + n + i, o[i], a.dtype);
  }
  if (cs > 1) cluster_barrier();
}

// At most eight columns. Shared memory: per warp its columns of x and their
// (down, down * sum) pairs; [tile][warp][B][16] sums; for clusters [tile][B][16].
template <int G, int FMT>
__global__ void __launch_bounds__(kLinThreads, 2) k_linear_few(const LinearArgs a, int cs) {
  constexpr int S = G > 64 ? G : 64, BL = S / 64, GS = S / G;
  constexpr int kAhead = FMT == kScale32 && G == 32 ? 4 : 8 / BL;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / cs;
  const bool split = a.dtype == SFFN_F32;
  const int cols = split ? 2 * a.B : a.B, elems = a.B * 16;
  // tiles of the cluster and steps of the warp: equal shares up to one
  const int tper = a.tiles / a.clusters, trest = a.tiles % a.clusters;
  const int tile0 = tper * cluster + min(cluster, trest), nt = tper + (cluster < trest);
  const int slices = cs * kLinWarps, slice = rank * kLinWarps + warp, all_steps = a.kp / S;
  const int sper = all_steps / slices, srest = all_steps % slices;
  const int k_first = sper * slice + min(slice, srest), spt = sper + (slice < srest);
  float* part = reinterpret_cast<float*>(smem + a.off_part);   // [tile][warp][elems]

  const uint4* cp = reinterpret_cast<const uint4*>(a.codes) + ((size_t)tile0 * (a.kp / 64) + (size_t)k_first * BL) * 32 + lane;
  size_t sp = ((size_t)tile0 * (a.kp / G) + (size_t)k_first * GS) * 8 + g;
  const size_t cp_skip = (size_t)(a.kp / 64 - spt * BL) * 32, sp_skip = (size_t)(a.kp / G - spt * GS) * 8;
  const int steps = nt * spt;
  uint4 cw[kAhead][BL];
  ScaleWord<FMT> sw[kAhead][GS];
  int left = steps, ld_k = 0;
  auto load = [&](uint4* c, ScaleWord<FMT>* s) {
    if (left > 0) {
      --left;
#pragma unroll
      for (int b = 0; b < BL; ++b) c[b] = ldg_stream(cp + b * 32);
#pragma unroll
      for (int q = 0; q < GS; ++q) s[q].load(a, sp + q * 8);
      cp += BL * 32;
      sp += GS * 8;
      if (++ld_k == spt) ld_k = 0, cp += cp_skip, sp += sp_skip;
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(cw[i], sw[i]);
  pdl_launch_dependents();
  pdl_wait();

  // ---- the warp's share of x, kBatch runs of 128 inputs at a time
  constexpr int kBatch = 4;
  __half* xs = reinterpret_cast<__half*>(smem) + (size_t)warp * cols * a.chunk_stride;
  float2* xg = reinterpret_cast<float2*>(smem + a.off_xg) + (size_t)warp * (a.chunk / G) * 8;
  const int k0 = k_first * S, kn = spt * S, runs = (kn + 127) / 128, tasks = runs * a.B;
  for (int task = 0, b = 0, run = 0; task < tasks; task += kBatch) {
    float v[kBatch][4], sh[kBatch], sl[kBatch], down[kBatch];
    uint32_t hi[kBatch][2], lo[kBatch][2];
    int at[kBatch], bs[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int kk = run * 128 + lane * 4;
      at[i] = task + i < tasks && kk < kn ? kk : -1;
      bs[i] = b;
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
      if (at[i] >= 0 && k0 + kk < a.k) ld_run<4>(a.x.ptr, (size_t)(b * a.x.row_stride) + k0 + kk, a.dtype, v[i]);
      if (++run == runs) run = 0, ++b;
    }
    convert_runs<G, kBatch, FMT != kScale16>(v, a.dtype, hi, lo, sh, sl, down);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at[i] < 0) continue;
      const int col = split ? 2 * bs[i] : bs[i];
      *reinterpret_cast<uint2*>(xs + (size_t)col * a.chunk_stride + at[i]) = make_uint2(hi[i][0], hi[i][1]);
      if (split) *reinterpret_cast<uint2*>(xs + (size_t)(col + 1) * a.chunk_stride + at[i]) = make_uint2(lo[i][0], lo[i][1]);
      if (lane % (G / 4) == 0) {
        float2* p = xg + (at[i] / G) * 8 + col;
        p[0] = make_float2(down[i], down[i] * sh[i]);
        if (split) p[1] = make_float2(down[i], down[i] * sl[i]);
      }
    }
  }
  __syncwarp();

  // ---- steps
  const __half* xcol[1] = {xs + (size_t)min(g, cols - 1) * a.chunk_stride + 8 * t};   // columns past the end: not used
  float y[1][4] = {{0.f, 0.f, 0.f, 0.f}};
  float* dst = part + (size_t)warp * elems;
  int kk = 0;
  for (int s = 0; s < steps;) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s < steps) {
        linear_step<G, 1, FMT>(a, cw[i], sw[i], xcol, kk * S, xg + kk * GS * 8 + 2 * t, y);
        load(cw[i], sw[i]);
        ++s;
        if (++kk == spt) {
          store_tile<1>(dst, y, a.B, split, false, g, t);
          y[0][0] = y[0][1] = y[0][2] = y[0][3] = 0.f;
          dst += kLinWarps * elems;
          kk = 0;
        }
      }
    }
  }
  if (spt == 0)   // a warp without inputs
    for (int i = 0; i < nt; ++i, dst += kLinWarps * elems) store_tile<1>(dst, y, a.B, split, false, g, t);
  __syncthreads();

  // ---- the block's sums, in warp order
  float* acc_s = reinterpret_cast<float*>(smem + a.off_acc);
  for (int e = threadIdx.x; e < nt * elems; e += kLinThreads) {
    const int tile = e / elems;
    const float* p = part + (size_t)tile * (kLinWarps - 1) * elems + e;
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < kLinWarps; ++w) r += p[w * elems];
    acc_s[e] = r;
  }
  __syncthreads();
  write_outputs(a, acc_s, tile0, nt, cs, rank, kLinThreads);
}

// x of a call as halves, and its pairs, for k_linear: one warp per token and run of 128 inputs.
template <int G, int FMT>
__global__ void __launch_bounds__(256) k_linear_x(const LinearArgs a, int pairs, __half* xh, float2* xg) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, runs = (a.kp + 127) / 128, task = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (task >= a.B * runs) return;
  const int b = task / runs, kk = (task - b * runs) * 128 + lane * 4;
  float v[1][4] = {{0.f, 0.f, 0.f, 0.f}}, sh[1], sl[1], down[1];
  uint32_t hi[1][2], lo[1][2];
  if (kk < a.k) ld_run<4>(a.x.ptr, (size_t)(b * a.x.row_stride) + kk, a.dtype, v[0]);
  convert_runs<G, 1, FMT != kScale16>(v, a.dtype, hi, lo, sh, sl, down);
  if (kk >= a.kp) return;
  const bool split = a.dtype == SFFN_F32;
  const int col = split ? 2 * b : b;
  *reinterpret_cast<uint2*>(xh + (size_t)col * a.kp + kk) = make_uint2(hi[0][0], hi[0][1]);
  if (split) *reinterpret_cast<uint2*>(xh + (size_t)(col + 1) * a.kp + kk) = make_uint2(lo[0][0], lo[0][1]);
  if (lane % (G / 4) == 0) {
    float2* p = xg + (size_t)(kk / G) * pairs + col;
    p[0] = make_float2(down[0], down[0] * sh[0]);
    if (split) p[1] = make_float2(down[0], down[0] * sl[0]);
  }
}

template <int G, int NT, int FMT>
__global__ void __launch_bounds__(linear_warps(NT) * 32, 1) k_linear(const LinearArgs a, int cs) {
  constexpr int kWarps = linear_warps(NT), kThreads = kWarps * 32;
  constexpr int S = G > 64 ? G : 64;        // inputs of a step
  constexpr int BL = S / 64, GS = S / G;    // 64-input blocks and groups of a step
  constexpr int kAhead = FMT == kScale32 && G == 32 ? 4 : 8 / BL;   // by registers
  extern __shared__ __align__(16) uint8_t smem[];
  __half* xs = reinterpret_cast<__half*>(smem);                  // [columns][chunk_stride]
  float2* xg = reinterpret_cast<float2*>(smem + a.off_xg);       // [groups of a chunk][8 NT]: down, down * sum(x)
  float* acc_s = reinterpret_cast<float*>(smem + a.off_acc);     // [tiles of the cluster][B][16]
  float* part = reinterpret_cast<float*>(smem + a.off_part);     // [warp][2][B][16]
  __shared__ int s_tile[kWarps][2];                              // tile of a part, -1: none
  __shared__ uint64_t s_bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / cs;
  const int tile0 = (int)((long long)cluster * a.tiles / a.clusters);
  const int nt = (int)((long long)(cluster + 1) * a.tiles / a.clusters) - tile0;
  // this block's inputs, in steps
  const int all_steps = (a.kp + S - 1) / S;
  const int k_step0 = all_steps * rank / cs, k_step1 = all_steps * (rank + 1) / cs;
  const bool split = a.dtype == SFFN_F32;
  const int cols = split ? 2 * a.B : a.B, elems = a.B * 16;
  const int chunk_steps = a.chunk / S;
  const int groups = a.kp / G, blocks64 = a.kp / 64;

  uint32_t phase = 0;
  for (int c0 = k_step0; c0 < k_step1 || c0 == k_step0; c0 += chunk_steps) {
    const int spt = min(chunk_steps, k_step1 - c0);   // steps of a tile in this chunk
    const int steps = nt * max(spt, 0);
    const int s0 = steps * warp / kWarps, s1 = steps * (warp + 1) / kWarps;

    // ---- the first loads of codes and scales: these do not depend on an earlier kernel
    uint4 cw[kAhead][BL];
    ScaleWord<FMT> sw[kAhead][GS];
    int ld_tile = spt > 0 ? s0 / spt : 0, ld_k = spt > 0 ? s0 % spt : 0, ld_s = s0;
    auto load = [&](uint4* c, ScaleWord<FMT>* s) {
      if (ld_s < s1) {
        const size_t tile = tile0 + ld_tile;
        const uint4* cp = reinterpret_cast<const uint4*>(a.codes) + (tile * blocks64 + (size_t)(c0 + ld_k) * BL) * 32 + lane;
#pragma unroll
        for (int b = 0; b < BL; ++b) c[b] = ldg_stream(cp + b * 32);   // kp is a multiple of S
        const size_t at = (tile * groups + (size_t)(c0 + ld_k) * GS) * 8 + g;
#pragma unroll
        for (int q = 0; q < GS; ++q) s[q].load(a, at + q * 8);
        if (++ld_k == spt) ld_k = 0, ++ld_tile;
        ++ld_s;
      }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(cw[i], sw[i]);

    if (c0 == k_step0) {
      if (threadIdx.x == 0) mbar_init(&s_bar, 1);
      fence_mbar_init();
      pdl_launch_dependents();
      pdl_wait();
      for (int i = threadIdx.x; i < nt * elems; i += kThreads) acc_s[i] = 0.f;
      if (threadIdx.x < 2 * kWarps) (&s_tile[0][0])[threadIdx.x] = -1;
    }
    __syncthreads();   // every warp is done with the chunk before

    // ---- x of the chunk: a bulk copy per column, and one for the pairs
    if (warp == 0 && spt > 0) {
      const uint32_t row = (uint32_t)spt * S * 2, pair = (uint32_t)spt * GS * 8 * NT * 8;
      if (lane == 0) mbar_arrive_expect_tx(&s_bar, row * cols + pair);
      __syncwarp();
      const uint64_t pol = l2_policy_keep();
      for (int c = lane; c < cols; c += 32)
        bulk_g2s(xs + (size_t)c * a.chunk_stride, a.ws_x + (size_t)c * a.kp + (size_t)c0 * S, row, &s_bar, pol);
      if (lane == 0) bulk_g2s(xg, a.ws_xg + (size_t)c0 * GS * 8 * NT, pair, &s_bar, pol);
    }
    if (spt > 0 && !mbar_wait_bounded(&s_bar, phase)) {
      set_device_error(a.err, SFFN_ERR_TIMEOUT);
      mbar_wait_bounded(&s_bar, phase);   // the copies must land before the block ends
    }
    phase ^= 1;

    // ---- the warp's steps
    float y[NT][4];
    int tile = spt > 0 ? s0 / spt : 0, kk = spt > 0 ? s0 % spt : 0;
    const int first_k = kk;
    bool fresh = true, first = true;
    const __half* xcol[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = 8 * n + g;   // columns past the end repeat the last one; their results are not used
      xcol[n] = xs + (size_t)min(c, cols - 1) * a.chunk_stride + 8 * t;
    }
    auto store = [&](float* dst, bool add) { store_tile<NT>(dst, y, a.B, split, add, g, t); };
    auto step = [&](const uint4* c, const ScaleWord<FMT>* s) {
      if (fresh) {
        fresh = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
      }
      linear_step<G, NT, FMT>(a, c, s, xcol, kk * S, xg + (size_t)kk * GS * (8 * NT) + 2 * t, y);
      if (++kk == spt) {
        // a tile that began in this warp's run is complete; the tail of an earlier warp's tile is a part
        if (first && first_k != 0) {
          store(part + (size_t)(warp * 2) * elems, false);
          if (lane == 0) s_tile[warp][0] = tile;
        } else {
          store(acc_s + (size_t)tile * elems, true);
        }
        first = false;
        fresh = true;
        kk = 0;
        ++tile;
      }
    };
    for (int s = s0; s < s1;) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s < s1) {
          step(cw[i], sw[i]);
          load(cw[i], sw[i]);
          ++s;
        }
      }
    }
    if (!fresh) {   // the head of a tile that a later warp completes
      store(part + (size_t)(warp * 2 + 1) * elems, false);
      if (lane == 0) s_tile[warp][1] = tile;
    }
    __syncthreads();
    // parts in warp order; a thread keeps to its elements, so no barrier is needed between them
    for (int e = threadIdx.x; e < elems; e += kThreads)
      for (int p = 0; p < 2 * kWarps; ++p) {
        const int pt = (&s_tile[0][0])[p];
        if (pt >= 0) acc_s[(size_t)pt * elems + e] += part[(size_t)p * elems + e];
      }
    __syncthreads();
    if (threadIdx.x < 2 * kWarps) (&s_tile[0][0])[threadIdx.x] = -1;
    if (spt <= 0) break;
  }

  write_outputs(a, acc_s, tile0, nt, cs, rank, kThreads);
}

// Calls f with the kernel of a number of column tiles and a scale format.
template <int G, typename F>
cudaError_t with_kernel(int nt, int fmt, F&& f) {
  auto by_fmt = [&](auto n) {
    constexpr int NT = decltype(n)::value;
    return fmt == kScale16 ? f(k_linear<G, NT, kScale16>)
                           : fmt == kScale16Zero ? f(k_linear<G, NT, kScale16Zero>) : f(k_linear<G, NT, kScale32>);
  };
  if (nt == 1)
    return fmt == kScale16 ? f(k_linear_few<G, kScale16>)
                           : fmt == kScale16Zero ? f(k_linear_few<G, kScale16Zero>) : f(k_linear_few<G, kScale32>);
  switch (nt) {
    case 2: return by_fmt(std::integral_constant<int, 2>());
    case 4: return by_fmt(std::integral_constant<int, 4>());
    default: return by_fmt(std::integral_constant<int, 8>());
  }
}

template <int G>
cudaError_t prepare(int nt, int fmt, LinearFit* fit) {
  return with_kernel<G>(nt, fmt, [&](auto* kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinLarge);
    for (int i = 0; i < 8 && e == cudaSuccess; ++i) {
      const int c = 1 << (i / 2);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(nt == 1 ? kLinThreads : linear_warps(nt) * 32);
      cfg.dynamicSmemBytes = i % 2 ? kLinLarge : kLinSmall;
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = c;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(i % 2 ? &fit->large[i / 2] : &fit->small[i / 2], kern, &cfg);
    }
    return e;
  });
}

template <int G>
cudaError_t run(int nt, int fmt, int cluster, const LinearArgs& a, int blocks, int smem, cudaStream_t st) {
  if (nt > 1) {
    auto* kx = fmt == kScale16 ? k_linear_x<G, kScale16> : k_linear_x<G, kScale32>;   // sums only where there are zeros
    const cudaError_t e = launch_ex(kx, dim3((a.B * ((a.kp + 127) / 128) + 7) / 8), dim3(256), 0, st, true, 1, a, 8 * nt,
                                    const_cast<__half*>(a.ws_x), const_cast<float2*>(a.ws_xg));
    if (e != cudaSuccess) return e;
  }
  return with_kernel<G>(nt, fmt, [&](auto* kern) {
    return launch_ex(kern, dim3(blocks), dim3(nt == 1 ? kLinThreads : linear_warps(nt) * 32), smem, st, true, cluster, a,
                     cluster);
  });
}

}  // namespace

#endif  // SFFN_LINEAR_GROUP

}  // namespace sffn
