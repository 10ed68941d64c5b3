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
// as halves: fp16 activations as they are; others after a power of two per token
// (and share of the inputs) that brings the largest to 2^13: bf16 activations
// exactly down to 2^-30 of it, fp32 activations as two columns, the nearest half
// and the nearest half of what is left (22 bits); of elements too small for that
// what is above 2^-38 of the largest counts.
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
// because every cluster would convert the same numbers again. A warp takes two
// tiles at a time with the same columns of x from shared memory.
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
  int off_sum, off_acc, off_part;      // bytes in shared memory
  const __half* ws_x;    // k_linear: x as halves [columns][kp], scaled;
  const float* ws_down;  // what undoes the scale, [8 NT];
  const float* ws_sum;   // sums over groups [groups][8 NT] (layers with zeros)
  sffn_rows x, residual, y;
};

constexpr int kLinWarps = 8;                   // of a block of k_linear_few
constexpr int kLinThreads = kLinWarps * 32;
// Of a block of k_linear, one per SM: tiles that a warp takes at a time, and as many warps as 64 sums per thread leave
// registers for (with four column tiles some values spill: 60 bytes with 16-bit scales of groups of 128, up to 512 with
// 32-bit scales of groups of 32).
constexpr int linear_tiles(int nt) { return nt == 8 ? 1 : 2; }
constexpr int linear_warps(int nt) { return nt == 8 ? 8 : 12; }

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

// The scales (and zeros) of rows g and g + 8 for the groups of one step, as loaded: [tile][step][8][GS] words of two
// 16-bit numbers, or pairs of 32-bit ones.
template <int G, int FMT>
struct StepScales {
  static constexpr int GS = 128 / G, N = FMT == kScale32 ? 2 * GS : GS;   // words of each array
  uint32_t sc[N], zr[FMT == kScale16 ? 1 : N];
  __device__ __forceinline__ static void words(const void* p, size_t at, uint32_t* w) {
    const uint32_t* q = static_cast<const uint32_t*>(p) + at * N;
    if (N == 1) {
      w[0] = __ldg(q);
    } else if (N == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
      w[0] = v.x, w[1 % N] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + i));
        w[i] = v.x, w[(i + 1) % N] = v.y, w[(i + 2) % N] = v.z, w[(i + 3) % N] = v.w;
      }
    }
  }
  __device__ __forceinline__ void load(const LinearArgs& a, size_t at) {   // at: (tile * steps + step) * 8 + g
    words(a.scales, at, sc);
    if (FMT == kScale16Zero) words(a.zeros, at, zr);
    if (FMT == kScale32) {
      if (a.zeros) {
        words(a.zeros, at, zr);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) zr[i % (sizeof(zr) / 4)] = 0u;
      }
    }
  }
  __device__ __forceinline__ static void two(const uint32_t* w, int q, int sdtype, float* o) {
    if (FMT == kScale32) {
      o[0] = __uint_as_float(w[2 * q % N]), o[1] = __uint_as_float(w[(2 * q + 1) % N]);
    } else if (sdtype == SFFN_F16) {
      const float2 f = __half22float2(u32_h2(w[q % N]));
      o[0] = f.x, o[1] = f.y;
    } else {
      o[0] = __uint_as_float(w[q % N] << 16), o[1] = __uint_as_float(w[q % N] & 0xffff0000u);
    }
  }
};

// y[r] += one step of 128 inputs of RT tiles: codes c[r] with scales s[r], times
// the columns xcol[n] (this lane's column of each eight) from half `at` on, whose
// sums over the step's groups stand at sums (rows of 8 NT).
template <int G, int NT, int RT, int FMT>
__device__ __forceinline__ void linear_step(const LinearArgs& a, const uint4 (*c)[2], const StepScales<G, FMT>* s,
                                            const __half* const* xcol, int at, const float* sums, float (*y)[NT][4]) {
  float d[RT][NT][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {   // 32 inputs
    uint32_t a0[RT][4], a1[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint4& v = c[r][h >> 1];
      const uint32_t wa = h & 1 ? v.z : v.x, wb = h & 1 ? v.w : v.y, ra = wa >> 8, rb = wb >> 8;
      a0[r][0] = weight_low(wa), a0[r][1] = weight_low(wb), a0[r][2] = weight_high(wa), a0[r][3] = weight_high(wb);
      a1[r][0] = weight_low(ra), a1[r][1] = weight_low(rb), a1[r][2] = weight_high(ra), a1[r][3] = weight_high(rb);
    }
    // two products go into a sum: those of other sums come between them
    constexpr int NP = NT > 1 ? 2 : 1;
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NP) {
      uint4 xv[NP];
#pragma unroll
      for (int n = 0; n < NP; ++n) xv[n] = *reinterpret_cast<const uint4*>(xcol[n0 + n] + at + h * 32);
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float* p = d[r][n0 + n];
          if (h * 32 % G == 0) p[0] = p[1] = p[2] = p[3] = 0.f;
          mma_f16(p, a0[r], xv[n].x, xv[n].y);
        }
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r) mma_f16(d[r][n0 + n], a1[r], xv[n].z, xv[n].w);
    }
    if ((h * 32 + 32) % G == 0) {   // end of a group: scales
      const int q = h * 32 / G;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float sc[2], z[2];
        s[r].two(s[r].sc, q, a.sdtype, sc);
        if (FMT != kScale16) s[r].two(s[r].zr, q, a.sdtype, z);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float2 v = make_float2(0.f, 0.f);
          if (FMT != kScale16) v = *reinterpret_cast<const float2*>(sums + q * (8 * NT) + 8 * n);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float d0 = FMT == kScale16 ? d[r][n][2 * k] : fmaf(-z[k], v.x, d[r][n][2 * k]);
            const float d1 = FMT == kScale16 ? d[r][n][2 * k + 1] : fmaf(-z[k], v.y, d[r][n][2 * k + 1]);
            y[r][n][2 * k] = fmaf(sc[k], d0, y[r][n][2 * k]);
            y[r][n][2 * k + 1] = fmaf(sc[k], d1, y[r][n][2 * k + 1]);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ float largest(const float* v) {   // of a lane's four inputs
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}

// Four inputs of a lane (of a run of 128) times a power of two as halves: the nearest in hi and, if split, what is left
// in lo. With Sums, the sums of hi and lo over a group of G.
template <int G, bool Sums>
__device__ __forceinline__ void convert_run(const float* v, float up, bool split, uint32_t* hi, uint32_t* lo, float& sh,
                                            float& sl) {
  sh = sl = 0.f;
  if (split) {
#pragma unroll
    for (int p = 0; p < 2; ++p) split_f16(v[2 * p] * up, v[2 * p + 1] * up, hi[p], lo[p]);
    if (Sums) {
      const float2 c = __half22float2(u32_h2(lo[0])), d = __half22float2(u32_h2(lo[1]));
      sl = (c.x + c.y) + (d.x + d.y);
#pragma unroll
      for (int o = 1; o < G / 4; o <<= 1) sl += __shfl_xor_sync(SFFN_FULL_MASK, sl, o);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) hi[p] = h2_u32(__floats2half2_rn(v[2 * p] * up, v[2 * p + 1] * up));
  }
  if (Sums) {
    const float2 a = __half22float2(u32_h2(hi[0])), b = __half22float2(u32_h2(hi[1]));
    sh = (a.x + a.y) + (b.x + b.y);
#pragma unroll
    for (int o = 1; o < G / 4; o <<= 1) sh += __shfl_xor_sync(SFFN_FULL_MASK, sh, o);
  }
}

// The sums of a tile ([B][16]) from the fragments of one warp; down undoes the scale of the lane's columns 2t, 2t + 1.
template <int NT>
__device__ __forceinline__ void store_tile(float* dst, const float (*y)[4], const float (*down)[2], int B, bool split,
                                           bool add, int g, int t) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (split) {
        const int b = 4 * n + t;
        if (b < B) {
          float* p = dst + b * 16 + g + 8 * r;
          const float v = (y[n][2 * r] + y[n][2 * r + 1]) * down[n][0];
          *p = add ? *p + v : v;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int b = 8 * n + 2 * t + c;
          if (b < B) {
            float* p = dst + b * 16 + g + 8 * r;
            const float v = y[n][2 * r + c] * down[n][c];
            *p = add ? *p + v : v;
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
    const size_t at = (size_t)(b * a.y.row_stride) + n;
    const int es = a.dtype == SFFN_F32 ? 4 : 2;
    if (n + 3 < a.n && (reinterpret_cast<uintptr_t>(a.y.ptr) + at * es) % (4 * es) == 0) {
      st_run<4>(a.y.ptr, at, a.dtype, o);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.n) st_elem(a.y.ptr, at + i, o[i], a.dtype);
    }
  }
  if (cs > 1) cluster_barrier();
}

// At most eight columns. Shared memory: per warp its columns of x, their sums
// over groups and scales; [tile][warp][B][16] sums; for clusters [tile][B][16].
//
// Bound: on paper by the codes (10240 x 8192: 43 MB, 6.4 us at the copy rate);
// in fact by how long one wave of blocks takes to begin (x converted, first
// codes from memory) and end (sums through distributed shared memory), about 5
// of its 13.7 us. Alone and cold it takes 17.9 us with DRAM 31% and issue slots
// 34% busy; 4096 x 4096 for one token 5.6, 4099 x 11008 with zeros for five
// 14.0 (replayed from a graph). A barrier between converting x and the products
// cost 4.6 us (20.5), one chunk of x after another instead of a share per warp
// is slower at every size.
template <int G, int FMT>
__global__ void __launch_bounds__(kLinThreads, 2) k_linear_few(const LinearArgs a, int cs) {
  constexpr int GS = 128 / G, kAhead = G == 32 && FMT != kScale16 ? (FMT == kScale32 ? 2 : 3) : 4;   // by registers
  constexpr bool kSums = FMT != kScale16;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / cs;
  const bool split = a.dtype == SFFN_F32;
  const int cols = split ? 2 * a.B : a.B, elems = a.B * 16;
  // tiles of the cluster and steps of the warp: equal shares up to one
  const int tper = a.tiles / a.clusters, trest = a.tiles % a.clusters;
  const int tile0 = tper * cluster + min(cluster, trest), nt = tper + (cluster < trest);
  const int slices = cs * kLinWarps, slice = rank * kLinWarps + warp, all_steps = a.kp / 128;
  const int sper = all_steps / slices, srest = all_steps % slices;
  const int k_first = sper * slice + min(slice, srest), spt = sper + (slice < srest);
  float* part = reinterpret_cast<float*>(smem + a.off_part);   // [tile][warp][elems]

  const uint4* cp = reinterpret_cast<const uint4*>(a.codes) + ((size_t)tile0 * all_steps + k_first) * 64 + lane;
  size_t sp = ((size_t)tile0 * all_steps + k_first) * 8 + g;
  const int skip = all_steps - spt, steps = nt * spt;
  uint4 cw[kAhead][1][2];
  StepScales<G, FMT> sw[kAhead][1];
  int left = steps, ld_k = 0;
  auto load = [&](uint4 (*c)[2], StepScales<G, FMT>* s) {
    if (left > 0) {
      --left;
      c[0][0] = ldg_stream(cp);
      c[0][1] = ldg_stream(cp + 32);
      s[0].load(a, sp);
      cp += 64;
      sp += 8;
      if (++ld_k == spt) ld_k = 0, cp += (size_t)skip * 64, sp += (size_t)skip * 8;
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(cw[i], sw[i]);
  pdl_launch_dependents();
  pdl_wait();

  // ---- the warp's share of x, token by token, kBatch runs of 128 inputs at a time
  constexpr int kBatch = 4;
  __half* xs = reinterpret_cast<__half*>(smem) + (size_t)warp * cols * a.chunk_stride;
  float* sums = reinterpret_cast<float*>(smem + a.off_sum) + (size_t)warp * (a.chunk / G + 1) * 8;   // last row: down
  float* downs = sums + (a.chunk / G) * 8;
  const int k0 = k_first * 128;
  if (a.dtype == SFFN_F16) {   // taken as they are
    if (lane < 8) downs[lane] = 1.f;
    const __half* px = static_cast<const __half*>(a.x.ptr) + k0 + lane * 4;
    const int tasks = a.B * spt;
    for (int task = 0, b = 0, run = 0; task < tasks; task += 2 * kBatch) {
      uint2 w[2 * kBatch];
      int b1 = b, run1 = run;
#pragma unroll
      for (int i = 0; i < 2 * kBatch; ++i) {
        w[i] = make_uint2(0u, 0u);
        if (task + i < tasks && k0 + run1 * 128 + lane * 4 < a.k)
          w[i] = __ldcg(reinterpret_cast<const uint2*>(px + b1 * a.x.row_stride + run1 * 128));
        if (++run1 == spt) run1 = 0, ++b1;
      }
#pragma unroll
      for (int i = 0; i < 2 * kBatch; ++i) {
        if (task + i >= tasks) break;
        *reinterpret_cast<uint2*>(xs + (size_t)b * a.chunk_stride + run * 128 + lane * 4) = w[i];
        if (kSums) {
          const float2 p = __half22float2(u32_h2(w[i].x)), q = __half22float2(u32_h2(w[i].y));
          float sum = (p.x + p.y) + (q.x + q.y);
#pragma unroll
          for (int o = 1; o < G / 4; o <<= 1) sum += __shfl_xor_sync(SFFN_FULL_MASK, sum, o);
          if (lane % (G / 4) == 0) sums[(run * GS + lane / (G / 4)) * 8 + b] = sum;
        }
        if (++run == spt) run = 0, ++b;
      }
    }
  }
  float v[kBatch][4], ahead[kBatch][4];   // of this token, and the first runs of the next
  auto fetch = [&](int b, int run0, float (*o)[4]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int kk = (run0 + i) * 128 + lane * 4;
      o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      if (run0 + i < spt && k0 + kk < a.k) ld_run<4>(a.x.ptr, (size_t)(b * a.x.row_stride) + k0 + kk, a.dtype, o[i]);
    }
  };
  const int others = a.dtype == SFFN_F16 ? 0 : a.B;
  if (others) fetch(0, 0, ahead);
#pragma unroll 1
  for (int b = 0; b < others; ++b) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = ahead[i][e];
    if (b + 1 < others) fetch(b + 1, 0, ahead);
    float big = 0.f, up, down;
    for (int run0 = 0; run0 < spt; run0 += kBatch) {
      if (run0) fetch(b, run0, v);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) big = fmaxf(big, largest(v[i]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(SFFN_FULL_MASK, big, o));
    scale_to_half_range(big, up, down);
    if (spt > kBatch) fetch(b, 0, v);
    const int col = split ? 2 * b : b;
    if (lane == 0) downs[col] = downs[split ? col + 1 : col] = down;
    for (int run0 = 0; run0 < spt; run0 += kBatch) {
      if (run0) fetch(b, run0, v);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (run0 + i >= spt) break;
        uint32_t hi[2], lo[2];
        float sh, sl;
        convert_run<G, kSums>(v[i], up, split, hi, lo, sh, sl);
        const int kk = (run0 + i) * 128 + lane * 4;
        *reinterpret_cast<uint2*>(xs + (size_t)col * a.chunk_stride + kk) = make_uint2(hi[0], hi[1]);
        if (split) *reinterpret_cast<uint2*>(xs + (size_t)(col + 1) * a.chunk_stride + kk) = make_uint2(lo[0], lo[1]);
        if (kSums && lane % (G / 4) == 0) {
          sums[kk / G * 8 + col] = sh;
          if (split) sums[kk / G * 8 + col + 1] = sl;
        }
      }
    }
  }
  __syncwarp();

  // ---- steps
  const __half* xcol[1] = {xs + (size_t)min(g, cols - 1) * a.chunk_stride + 8 * t};   // columns past the end: not used
  const float down[1][2] = {{downs[2 * t], downs[2 * t + 1]}};
  float y[1][1][4] = {{{0.f, 0.f, 0.f, 0.f}}};
  float* dst = part + (size_t)warp * elems;
  int kk = 0;
  for (int s = 0; s < steps;) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s < steps) {
        linear_step<G, 1, 1, FMT>(a, cw[i], sw[i], xcol, kk * 128, sums + kk * GS * 8 + 2 * t, y);
        load(cw[i], sw[i]);
        ++s;
        if (++kk == spt) {
          store_tile<1>(dst, y[0], down, a.B, split, false, g, t);
          y[0][0][0] = y[0][0][1] = y[0][0][2] = y[0][0][3] = 0.f;
          dst += kLinWarps * elems;
          kk = 0;
        }
      }
    }
  }
  if (spt == 0)   // a warp without inputs
    for (int i = threadIdx.x & 31; i < nt * elems; i += 32) part[((size_t)(i / elems) * kLinWarps + warp) * elems + i % elems] = 0.f;
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

// x of a call as halves, and its sums over groups, for k_linear: one block per token.
// Two passes over a token's row, the first for its largest element; the second
// takes what a warp kept of the first from registers. Bound by latency: 6.7 us
// for 32 tokens of 8192 alone, of which the next kernel's loads hide a part.
template <int G, bool Sums>
__global__ void __launch_bounds__(512) k_linear_x(const LinearArgs a, int columns, __half* xh, float* downs, float* sums) {
  constexpr int kKeep = 4;   // runs of 128 inputs that a warp keeps between the two passes
  __shared__ float s_big[16];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x, runs = a.kp / 128;
  float v[kKeep][4], big = 0.f;
  auto fetch = [&](int run, float* o) {
    const int kk = run * 128 + lane * 4;
    o[0] = o[1] = o[2] = o[3] = 0.f;
    if (run < runs && kk < a.k) ld_run<4>(a.x.ptr, (size_t)(b * a.x.row_stride) + kk, a.dtype, o);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) fetch(warp + 16 * i, v[i]);
#pragma unroll
  for (int i = 0; i < kKeep; ++i) big = fmaxf(big, largest(v[i]));
  for (int run = warp + 16 * kKeep; run < runs; run += 16) {
    float o[4];
    fetch(run, o);
    big = fmaxf(big, largest(o));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(SFFN_FULL_MASK, big, o));
  if (lane == 0) s_big[warp] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) big = fmaxf(big, s_big[w]);
  float up = 1.f, down = 1.f;
  if (a.dtype != SFFN_F16) scale_to_half_range(big, up, down);   // fp16 rows are taken as they are
  const bool split = a.dtype == SFFN_F32;
  const int col = split ? 2 * b : b;
  if (threadIdx.x == 0) downs[col] = downs[split ? col + 1 : col] = down;
  auto put = [&](int run, const float* o) {
    uint32_t hi[2], lo[2];
    float sh, sl;
    convert_run<G, Sums>(o, up, split, hi, lo, sh, sl);
    const int kk = run * 128 + lane * 4;
    *reinterpret_cast<uint2*>(xh + (size_t)col * a.kp + kk) = make_uint2(hi[0], hi[1]);
    if (split) *reinterpret_cast<uint2*>(xh + (size_t)(col + 1) * a.kp + kk) = make_uint2(lo[0], lo[1]);
    if (Sums && lane % (G / 4) == 0) {
      sums[(size_t)(kk / G) * columns + col] = sh;
      if (split) sums[(size_t)(kk / G) * columns + col + 1] = sl;
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (warp + 16 * i < runs) put(warp + 16 * i, v[i]);
  for (int run = warp + 16 * kKeep; run < runs; run += 16) {
    float o[4];
    fetch(run, o);
    put(run, o);
  }
}

// More than eight columns.
//
// Bound: by the warp-level product. At 32 columns each code enters four of them;
// 2.7e9 products of a 10240 x 8192 layer with 32 tokens are 21K cycles an SM at
// the rate measured here (850 multiply-adds a cycle and SM), of 31K in the loop
// and 55K in all: 29 us with k_linear_x before it, 187 TFLOP/s; 32 fp32 tokens,
// 64 columns, 45 us, with zeros and groups of 32 68. Two tiles a warp
// halve the reads of x from shared memory (one: 39 us); three chunks of x
// instead of one cost 10 us, so the warps' parts take the place of x once it is
// read (45 us before). Cold: 32.3 us, tensor pipe 34%, DRAM 17%, most waits for
// codes between steps.
template <int G, int NT, int FMT>
__global__ void __launch_bounds__(linear_warps(NT) * 32, 1) k_linear(const LinearArgs a, int cs) {
  constexpr int kWarps = linear_warps(NT), kThreads = kWarps * 32, RT = linear_tiles(NT), GS = 128 / G;
  constexpr int kAhead = RT == 2 ? (FMT == kScale16 || G == 128 ? 3 : 2) : (FMT == kScale32 && G == 32 ? 2 : 4);  // by registers
  constexpr bool kSums = FMT != kScale16;
  extern __shared__ __align__(16) uint8_t smem[];
  __half* xs = reinterpret_cast<__half*>(smem);                  // [columns][chunk_stride]
  float* sums = reinterpret_cast<float*>(smem + a.off_sum);      // [groups of a chunk][8 NT]
  float* acc_s = reinterpret_cast<float*>(smem + a.off_acc);     // [tiles of the cluster][B][16]
  float* part = reinterpret_cast<float*>(smem);                  // [warp][RT][B][16], over xs once that is read
  __shared__ int s_unit[kWarps];                                 // unit (RT tiles) of a part, -1: none
  __shared__ uint64_t s_bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)cluster_rank() : 0, cluster = blockIdx.x / cs;
  // units of the cluster and steps of the block: equal shares up to one
  const int all_units = a.tiles / RT, uper = all_units / a.clusters, urest = all_units % a.clusters;
  const int unit0 = uper * cluster + min(cluster, urest), nu = uper + (cluster < urest);
  const int all_steps = a.kp / 128, sper = all_steps / cs, srest = all_steps % cs;
  const int k_step0 = sper * rank + min(rank, srest), k_step1 = k_step0 + sper + (rank < srest);
  const bool split = a.dtype == SFFN_F32;
  const int cols = split ? 2 * a.B : a.B, elems = a.B * 16, uelems = RT * elems;
  const int chunk_steps = a.chunk / 128;

  uint32_t phase = 0;
  float down[NT][2];
  for (int c0 = k_step0; c0 < k_step1 || c0 == k_step0; c0 += chunk_steps) {
    const int spt = max(0, min(chunk_steps, k_step1 - c0));   // steps of a unit in this chunk
    const int steps = nu * spt, s0 = steps * warp / kWarps, s1 = steps * (warp + 1) / kWarps;

    // ---- the first loads of codes and scales: these do not depend on an earlier kernel
    uint4 cw[kAhead][RT][2];
    StepScales<G, FMT> sw[kAhead][RT];
    int unit = spt > 0 ? s0 / spt : 0, kk = spt > 0 ? s0 - unit * spt : 0;
    const size_t first = (size_t)(unit0 + unit) * RT * all_steps + c0 + kk;
    const uint4* cp = reinterpret_cast<const uint4*>(a.codes) + first * 64 + lane;
    size_t sp = first * 8 + g;
    int left = s1 - s0, ld_k = kk;
    auto load = [&](uint4 (*c)[2], StepScales<G, FMT>* s) {
      if (left > 0) {
        --left;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          c[r][0] = ldg_stream(cp + (size_t)r * all_steps * 64);
          c[r][1] = ldg_stream(cp + (size_t)r * all_steps * 64 + 32);
          s[r].load(a, sp + (size_t)r * all_steps * 8);
        }
        cp += 64;
        sp += 8;
        if (++ld_k == spt) {
          ld_k = 0;
          cp += (size_t)(RT * all_steps - spt) * 64;
          sp += (size_t)(RT * all_steps - spt) * 8;
        }
      }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(cw[i], sw[i]);

    if (c0 == k_step0) {
      if (threadIdx.x == 0) mbar_init(&s_bar, 1);
      fence_mbar_init();
      pdl_launch_dependents();
      pdl_wait();
      for (int i = threadIdx.x; i < nu * uelems; i += kThreads) acc_s[i] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = 8 * n + 2 * t;
        down[n][0] = c < cols ? ld_dep(a.ws_down + c) : 0.f;
        down[n][1] = c + 1 < cols ? ld_dep(a.ws_down + c + 1) : 0.f;
      }
    }
    if (lane == 0) s_unit[warp] = -1;
    __syncthreads();   // every warp is done with the chunk before

    // ---- x of the chunk: a bulk copy per column, and one for the sums
    if (warp == 0 && spt > 0) {
      fence_proxy_async_smem();   // the parts of the chunk before stood where the copies go
      const uint32_t row = (uint32_t)spt * 256, sum = kSums ? (uint32_t)spt * GS * 8 * NT * 4 : 0u;
      if (lane == 0) mbar_arrive_expect_tx(&s_bar, row * cols + sum);
      __syncwarp();
      const uint64_t pol = l2_policy_keep();
      for (int c = lane; c < cols; c += 32)
        bulk_g2s(xs + (size_t)c * a.chunk_stride, a.ws_x + (size_t)c * a.kp + (size_t)c0 * 128, row, &s_bar, pol);
      if (kSums && lane == 0) bulk_g2s(sums, a.ws_sum + (size_t)c0 * GS * 8 * NT, sum, &s_bar, pol);
    }
    if (spt > 0) {
      if (!mbar_wait_bounded(&s_bar, phase)) {
        set_device_error(a.err, SFFN_ERR_TIMEOUT);
        mbar_wait_bounded(&s_bar, phase);   // the copies must land before the block ends
      }
      phase ^= 1;
    }

    // ---- the warp's steps
    float y[RT][NT][4];
    bool fresh = true;
    const __half* xcol[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)   // columns past the end repeat the last one; their results are not used
      xcol[n] = xs + (size_t)min(8 * n + g, cols - 1) * a.chunk_stride + 8 * t;
    auto store = [&](float* dst, bool add) {
#pragma unroll
      for (int r = 0; r < RT; ++r) store_tile<NT>(dst + r * elems, y[r], down, a.B, split, add, g, t);
    };
    for (int s = s0; s < s1;) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s < s1) {
          if (fresh) {
            fresh = false;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int n = 0; n < NT; ++n) y[r][n][0] = y[r][n][1] = y[r][n][2] = y[r][n][3] = 0.f;
          }
          linear_step<G, NT, RT, FMT>(a, cw[i], sw[i], xcol, kk * 128, sums + kk * GS * (8 * NT) + 2 * t, y);
          load(cw[i], sw[i]);
          ++s;
          if (++kk == spt) {
            store(acc_s + (size_t)unit * uelems, true);   // of the warps of a unit, only the one that ends it does this
            fresh = true;
            kk = 0;
            ++unit;
          }
        }
      }
    }
    __syncthreads();
    if (!fresh) {   // the head of a unit that a later warp ended
      store(part + (size_t)warp * uelems, false);
      if (lane == 0) s_unit[warp] = unit;
    }
    __syncthreads();
    // the first warp with a part of a unit adds all of that unit, in warp order
    const int mine = s_unit[warp];
    const unsigned same = __ballot_sync(SFFN_FULL_MASK, lane < kWarps && s_unit[min(lane, kWarps - 1)] == mine);
    if (mine >= 0 && __ffs(same) - 1 == warp) {
      float4* dst = reinterpret_cast<float4*>(acc_s + (size_t)mine * uelems);
#pragma unroll 4
      for (int e = lane; e < uelems / 4; e += 32) {
        float4 v = dst[e];
        for (unsigned left = same; left; left &= left - 1) {
          const float4 x = reinterpret_cast<const float4*>(part + (size_t)(__ffs(left) - 1) * uelems)[e];
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        dst[e] = v;
      }
    }
    __syncthreads();
    if (spt == 0) break;
  }

  // ---- the cluster's blocks add their sums; each writes its share of the outputs
  write_outputs(a, acc_s, unit0 * RT, nu * RT, cs, rank, kThreads);
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
    auto* kx = fmt == kScale16 ? k_linear_x<G, false> : k_linear_x<G, true>;   // sums only where there are zeros
    const cudaError_t e = launch_ex(kx, dim3(a.B), dim3(512), 0, st, true, 1, a, 8 * nt, const_cast<__half*>(a.ws_x),
                                    const_cast<float*>(a.ws_down), const_cast<float*>(a.ws_sum));
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
