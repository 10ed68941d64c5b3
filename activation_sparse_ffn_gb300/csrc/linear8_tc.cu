// The 8-bit linear layer for many tokens, on the fifth-generation tensor cores.
//
// GB300 has no 8-bit whole-number kind of the product, so codes become halves
// (linear8.cuh). Two blocks of a cluster compute 256 rows x up to 192 tokens
// together (cta_group::2). The rows of the layer are the product's operand A:
// each block brings 128 rows of 64 codes to shared memory by bulk copies, the
// thread of a row widens them and writes them to tensor memory, from where the
// product takes A, so that the widened codes cross shared memory neither way.
// The tokens are operand B, each block holding half of them. They are widened
// once, by k_lin8_widen before, into the order in which a tile stands in shared
// memory (128-byte swizzle), so that a block's half is one run of bytes;
// widened on the way like the rows they took more instructions than the
// product left time for.
//
// Sums leave their fp32 accumulators as whole numbers every 1024 inputs, into
// registers, while the product goes on in a second accumulator.
//
// A step is 128 inputs: eight products a turn, since what surrounds them (a
// wait, two commits) takes 500 cycles of the thread that issues them, as long as
// five products, however many there are (64 inputs a step: 10240 x 8192 for 4096
// tokens 775 us).
//
// Tiles that fill whole waves are computed one at a time; the steps of those
// left over are shared out evenly. A block that has part of
// a tile leaves its sums in the workspace, and whichever comes last adds them:
// whole numbers, so that the order does not matter.
//
// Measured: 10240 x 8192 for 4096 tokens 370 us, 1.86 PFLOP/s of halves, the tensor
// cores active 80% of the time (a step takes 845 cycles, its products 768); for 150
// tokens 33 us (42 from cold caches), of which the steps are 16, and leaving, joining
// and writing the parts of tiles up to 14.
#include <algorithm>
#include <type_traits>

#include "linear8.cuh"
#include "linear8_split.h"
#include "rows_io.cuh"
#include "step.h"
#include "tcgen05.cuh"

namespace sffn {

namespace {

// Warps 0-3 widen even steps and 4-7 odd ones, 8-15 take the sums, and one thread each of 16 to 19 copies codes, copies
// tokens, reports their arrival and issues products. Registers go where the sums are: 2 x 88 + 2 x 136 + 32 of
// the 5 x 96 a thread has at launch.
constexpr int kConvWarps = 4, kEpiWarps = 8, kEpiWarp0 = 8, kTcThreads = 640;
constexpr int kWarpW = 16, kWarpX = 17, kWarpTold = 18, kWarpMma = 19;
constexpr int kMaxTokens = 192;                          // of a tile
constexpr int kStep = 2 * kL8Inputs, kStepW = 2 * kL8Block;
constexpr int kSlots = 2, kSlotCols = 64;                // of A in tensor memory, one for each set of warps that widen
constexpr int kAccCols = 192, kTmemCols = 512;           // accumulators at 0 and 192, A at 384
constexpr int kStagesW = 6, kStagesX = 4;                // the first even: a set of warps keeps its own
constexpr int kStepsExact = kL8Exact / kStep;
constexpr int CG = 2;                                    // blocks of a cluster

struct TcArgs {
  const uint8_t* codes;   // [tiles of 128 rows][steps][16 KB]
  const uint8_t* xh;      // [2 steps][tokens][128 bytes]
  const float* scales;
  const float* bias;
  const float* x_scales;
  sffn_rows residual, y;
  int32_t* parts;         // [block][2][tokens of a tile][128]
  uint32_t* tickets;      // [tiles left over][CG], zeros from k_lin8_widen: nothing stays of a call that gave up
  uint32_t* err;
  int n, B, dtype, steps, nt, token_tiles, tokens;   // nt: tokens of a tile; tokens: token_tiles * nt
  L8Split split;
};

// True in one lane of the warp, always the same. The warps that issue copies and products run their loops with every lane
// and pick one for the instruction alone: the instructions take their operands from uniform registers, and in a branch
// that one lane enters everything has to be brought there first (2 x 150 cycles for the two commits of a step).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Arrives on the barrier of the pair's first block.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}

// Waits for the phase of the given parity, a second at most. The clock is looked at rarely: a wait that reads it first is
// longer than most.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i % 256 == 0) {
      const uint64_t t = globaltimer_ns();
      if (!t0) t0 = t;
      if (t - t0 > kWaitLimitNs) return false;
    }
  }
}

// A place in a ring of N and the parity of its turn, STEP places at a time.
template <int N, int STEP>
struct Ring {
  int at;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int from) : at(from) {}
  __device__ __forceinline__ void next() {
    at += STEP;
    if (at >= N) at -= N, phase ^= 1;
  }
};

// Instruction descriptor of kind::f16 with fp32 sums and halves on both sides, both K-major, 256 rows, n columns.
__device__ __forceinline__ uint32_t half_desc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 * CG >> 4) << 24);
}

// d (tensor memory) += a (tensor memory) b (shared memory), of both blocks.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}

// One arrival on the barrier of both blocks once the thread's products so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t t) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(kTmemCols) : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of 32-bit words of the warp's 32 lanes.
__device__ __forceinline__ void tmem_store32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of the warp's 32 lanes, there when this returns.
__device__ __forceinline__ void tmem_load16(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
// An element as its bits. The load stays where it is written: brought forward, all 96 of an output's residuals would want
// registers at once.
template <typename T>
__device__ __forceinline__ uint32_t load_here(const T* p) {
  if constexpr (sizeof(T) == 4) {
    uint32_t v;
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  } else {
    unsigned short v;
    asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
  }
}
template <typename T>
__device__ __forceinline__ float as_float(uint32_t u) {
  if constexpr (std::is_same<T, float>::value) return __uint_as_float(u);
  if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)u));
  return __uint_as_float(u << 16);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Outputs v of row n and `tokens` tokens from token0 on. The type is settled outside: 96 times a choice of three types, code
// that no cache of instructions holds, took longer than a tile's products.
template <typename T>
__device__ __forceinline__ void put_outputs(const TcArgs& a, const int (&v)[96], int n, int token0, int tokens) {
  if (n >= a.n) tokens = 0;
  T* y = static_cast<T*>(a.y.ptr) + token0 * a.y.row_stride + n;
  if (a.residual.ptr) {
    const T* res = static_cast<const T*>(a.residual.ptr) + token0 * a.residual.row_stride + n;
    uint32_t r[2][8];   // eight residuals on their way while eight outputs are written
    auto load = [&](int b, uint32_t* to) {
#pragma unroll
      for (int i = 0; i < 8; ++i, res += a.residual.row_stride)
        if (b + i < tokens) to[i] = load_here(res);
    };
    load(0, r[0]);
#pragma unroll
    for (int b = 0; b < 96; b += 8) {
      if (b + 8 < 96) load(b + 8, r[(b / 8 + 1) & 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i, y += a.y.row_stride)
        if (b + i < tokens) *y = from_float<T>(__fadd_rn(__int_as_float(v[b + i]), as_float<T>(r[(b / 8) & 1][i])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 96; ++i, y += a.y.row_stride)
      if (i < tokens) *y = from_float<T>(__int_as_float(v[i]));
  }
}

__global__ void __launch_bounds__(kTcThreads, 1)
    k_lin8_tc(const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* smem = dyn_smem + (1024 - (smem_u32(dyn_smem) & 1023)) % 1024;   // the swizzle counts from there
  __shared__ uint64_t wfull[kStagesW], wempty[kStagesW], xfull[kStagesX], xempty[kStagesX];
  __shared__ uint64_t ready[kSlots], freed[kSlots], accfull[2], accempty[2], drain, meeting;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  const int tid = threadIdx.x, warp = __shfl_sync(SFFN_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x % CG, cluster = blockIdx.x / CG;   // clusters are consecutive blocks
  const int x_bytes = a.nt / CG * 128;          // of the block's tokens, 64 inputs
  uint8_t* ring_w = smem;                       // codes of 128 rows
  uint8_t* ring_x = smem + kStagesW * kStepW;   // widened tokens, two times 64 inputs a stage
  if (tid == 0) {
    for (int s = 0; s < kStagesW; ++s) mbar_init(&wfull[s], 1), mbar_init(&wempty[s], kConvWarps);
    for (int s = 0; s < kStagesX; ++s) mbar_init(&xfull[s], 1), mbar_init(&xempty[s], 1);
    for (int s = 0; s < kSlots; ++s) mbar_init(&ready[s], (kConvWarps + 1) * CG), mbar_init(&freed[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&accfull[s], 1), mbar_init(&accempty[s], kEpiWarps * CG);
    mbar_init(&drain, 1), mbar_init(&meeting, kEpiWarps);
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == kWarpMma) tmem_alloc(&s_tmem);
  tc::fence_before();
  __syncthreads();
  cluster_sync_all();   // the other block's barriers are initialised too
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  pdl_launch_dependents();

  auto fail = [&]() {
    set_device_error(a.err, SFFN_ERR_TIMEOUT);
    atomicExch(&s_abort, 1);
  };
  auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };
  L8Segments work(a.split, cluster);
  L8Segment seg;

  if (warp < 2 * kConvWarps) {
    // ------------------------------------------------------------ codes to halves
    fewer_registers<88>();
    pdl_wait();
    const int row = tid & 127, set = warp / kConvWarps;
    const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 2 * kAccCols;
    Ring<kStagesW, 2> w(set);
    Ring<kSlots, 2> out(set);
    int it = 0;
    bool ok = true;
    while (ok && work.next(a.split, seg)) {
      const int len = seg.s1 - seg.s0;
      for (int k = (it ^ set) & 1; k < len; k += 2) {
        ok = wait_for(&wfull[w.at], w.phase);
        const uint8_t* src = ring_w + w.at * kStepW;
        uint32_t h[64];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + (t >> 2) * kL8Block + l8_chunk(row, t & 3));
          l8_halves(v.x, h[8 * t], h[8 * t + 1]), l8_halves(v.y, h[8 * t + 2], h[8 * t + 3]);
          l8_halves(v.z, h[8 * t + 4], h[8 * t + 5]), l8_halves(v.w, h[8 * t + 6], h[8 * t + 7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[w.at]);
        ok = wait_for(&freed[out.at], out.phase ^ 1) && ok;   // passes at once the first time round
        if (!__all_sync(SFFN_FULL_MASK, ok)) break;
        tc::fence_after();
        tmem_store32(mine + out.at * kSlotCols, h);
        tmem_store32(mine + out.at * kSlotCols + 32, h + 32);
        tmem_store_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&ready[out.at]);
        w.next(), out.next();
      }
      it += len;
      ok = __all_sync(SFFN_FULL_MASK, ok);
      if (!ok && lane == 0) fail();
    }
  } else if (warp < kEpiWarp0 + kEpiWarps) {
    // ------------------------------------------------------------ sums to whole numbers to outputs
    more_registers<136>();
    pdl_wait();
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2, blocks = a.nt / 16;
    const int b0 = half ? (blocks + 1) / 2 : 0, nb = half ? blocks - b0 : (blocks + 1) / 2;   // of 16 tokens, at most 6
    const uint32_t mine = tmem + ((uint32_t)(q * 32) << 16) + b0 * 16;
    const int r = q * 32 + lane;
    int chunk = 0, met = 0;
    bool ok = true;
    auto meet = [&]() {   // of the eight warps, one of which may have given up
      __syncwarp();
      if (lane == 0) mbar_arrive(&meeting);
      return __all_sync(SFFN_FULL_MASK, wait_for(&meeting, (uint32_t)(met++ & 1)));
    };
    while (ok && work.next(a.split, seg)) {
      int sum[96];
#pragma unroll
      for (int i = 0; i < 96; ++i) sum[i] = 0;
      for (int k = seg.s0; k < seg.s1; k += kStepsExact, ++chunk) {
        const int buf = chunk & 1;
        ok = __all_sync(SFFN_FULL_MASK, wait_for(&accfull[buf], (uint32_t)((chunk / 2) & 1)));
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int b = 0; b < 6; ++b)
          if (b < nb) {
            float v[16];
            tmem_load16(mine + buf * kAccCols + b * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[b * 16 + i] += __float2int_rn(v[i]);
          }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&accempty[buf]);
      }
      if (!ok) {
        if (lane == 0) fail();
        break;
      }
      const int row_tile = seg.tile / a.token_tiles * CG + rank, token0 = seg.tile % a.token_tiles * a.nt + b0 * 16;
      if (seg.part) {
        // this block's sums to its place; the last to arrive adds the others'
        const int left = seg.tile - a.split.whole * a.split.groups;
        const size_t tile_ints = (size_t)a.nt * kL8Rows, at = (size_t)b0 * 16 * kL8Rows + r;
        int32_t* place = a.parts + ((size_t)blockIdx.x * 2 + seg.slot) * tile_ints + at;
#pragma unroll
        for (int i = 0; i < 96; ++i)
          if (i / 16 < nb) __stcg(place + (size_t)i * kL8Rows, sum[i]);
        __threadfence();
        ok = meet();
        const L8Sharers sharers = l8_sharers(a.split, left, cluster);
        if (ok && warp == kEpiWarp0 && lane == 0)
          s_last = (int)atomicAdd(a.tickets + left * CG + rank, 1u) == sharers.to - sharers.from;
        ok = ok && meet();
        const bool join = s_last;
        ok = ok && meet();   // read by all before it is written again
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        if (!join) continue;
        __threadfence();
        for (int c = sharers.from; c <= sharers.to; ++c) {
          if (c == cluster) continue;
          const int32_t* other = a.parts + ((size_t)(c * CG + rank) * 2 + l8_slot(a.split, left, c)) * tile_ints + at;
#pragma unroll
          for (int i = 0; i < 96; ++i)
            if (i / 16 < nb) sum[i] += __ldcg(other + (size_t)i * kL8Rows);
        }
      }
      const int n = row_tile * kL8Rows + r;
      const float scale = a.scales[n], bias = a.bias[n];   // padded to whole tiles
      float xs[3];   // the tokens' scales, one a lane
#pragma unroll
      for (int i = 0; i < 3; ++i) xs[i] = token0 + 32 * i + lane < a.B ? __ldcg(a.x_scales + token0 + 32 * i + lane) : 0.f;
      const int tokens = min(nb * 16, a.B - token0);
#pragma unroll
      for (int i = 0; i < 96; ++i)   // the outputs but for the residual, in the registers of their sums
        sum[i] = __float_as_int(l8_value(sum[i], scale, __shfl_sync(SFFN_FULL_MASK, xs[i / 32], i % 32), bias));
      if (a.dtype == SFFN_F32)
        put_outputs<float>(a, sum, n, token0, tokens);
      else if (a.dtype == SFFN_F16)
        put_outputs<__half>(a, sum, n, token0, tokens);
      else
        put_outputs<__nv_bfloat16>(a, sum, n, token0, tokens);
      __syncwarp();
    }
  } else {
    fewer_registers<32>();
    if (warp == kWarpW) {
      // ---------------------------------------------------------- codes of rows, which are no earlier kernel's
      const uint64_t policy = a.token_tiles > 1 ? tc::l2_policy_evict_last() : l2_policy_evict_first();
      Ring<kStagesW, 1> w(0);
      int it = 0;
      bool ok = true;
      while (ok && work.next(a.split, seg)) {
        const int row_tile = seg.tile / a.token_tiles * CG + rank;
        const uint8_t* src = a.codes + ((size_t)row_tile * a.steps + seg.s0) * kStepW;
        for (int k = seg.s0; k < seg.s1; ++k, ++it, src += kStepW, w.next()) {
          ok = __all_sync(SFFN_FULL_MASK, wait_for(&wempty[w.at], w.phase ^ 1));
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&wfull[w.at], kStepW);
            bulk_g2s(ring_w + w.at * kStepW, src, kStepW, &wfull[w.at], policy);
          }
        }
      }
      if (!ok && lane == 0) fail();
      if (aborted())   // copies in flight land before the block ends
        for (int q = max(0, it - kStagesW); q < it; ++q) wait_for(&wfull[q % kStagesW], (uint32_t)((q / kStagesW) & 1));
      pdl_wait();
    } else if (warp == kWarpX) {
      // ---------------------------------------------------------- tokens
      pdl_wait();
      const uint64_t policy = tc::l2_policy_evict_last();
      Ring<kStagesX, 1> x(0);
      int it = 0;
      bool ok = true;
      while (ok && work.next(a.split, seg)) {
        const int token0 = seg.tile % a.token_tiles * a.nt + rank * (a.nt / CG);
        const uint8_t* src = a.xh + ((size_t)seg.s0 * 2 * a.tokens + token0) * 128;
        for (int k = seg.s0; k < seg.s1; ++k, ++it, src += (size_t)a.tokens * 256, x.next()) {
          ok = __all_sync(SFFN_FULL_MASK, wait_for(&xempty[x.at], x.phase ^ 1));
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&xfull[x.at], 2 * x_bytes);
            bulk_g2s(ring_x + 2 * x.at * x_bytes, src, x_bytes, &xfull[x.at], policy);
            bulk_g2s(ring_x + (2 * x.at + 1) * x_bytes, src + (size_t)a.tokens * 128, x_bytes, &xfull[x.at], policy);
          }
        }
      }
      if (!ok && lane == 0) fail();
      if (aborted())
        for (int q = max(0, it - kStagesX); q < it; ++q) wait_for(&xfull[q % kStagesX], (uint32_t)((q / kStagesX) & 1));
    } else if (warp == kWarpTold) {
      // ---------------------------------------------------------- tokens that have arrived are reported to the pair's first block
      pdl_wait();
      Ring<kStagesX, 1> x(0);
      Ring<kSlots, 1> slot(0);
      bool ok = true;
      while (ok && work.next(a.split, seg))
        for (int k = seg.s0; ok && k < seg.s1; ++k, x.next(), slot.next()) {
          // a slot's report counts for the product that comes next in it
          ok = wait_for(&xfull[x.at], x.phase) && wait_for(&freed[slot.at], slot.phase ^ 1);
          ok = __all_sync(SFFN_FULL_MASK, ok);
          if (ok && elect_one()) arrive_first(&ready[slot.at]);
        }
      if (!ok && lane == 0) fail();
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- products, one thread of the pair
      pdl_wait();
      if (rank == 0) {
        const uint32_t idesc = half_desc(a.nt), first_x = smem_u32(ring_x);
        Ring<kStagesX, 1> x(0);
        Ring<kSlots, 1> slot(0);
        int chunk = 0;
        bool ok = true;
        while (ok && work.next(a.split, seg)) {
          for (int k = seg.s0; ok && k < seg.s1; ++chunk) {
            const int end = min(k + kStepsExact, seg.s1), buf = chunk & 1;
            ok = chunk < 2 || __all_sync(SFFN_FULL_MASK, wait_for(&accempty[buf], (uint32_t)((chunk / 2 - 1) & 1)));
            const uint32_t acc = tmem + buf * kAccCols;
            bool add = false;
            for (; ok && k < end; ++k, x.next(), slot.next(), add = true) {
              ok = __all_sync(SFFN_FULL_MASK, wait_for(&ready[slot.at], slot.phase));
              if (!ok) break;
              tc::fence_after();
              const uint32_t xs = first_x + 2 * x.at * x_bytes, as = tmem + 2 * kAccCols + slot.at * kSlotCols;
              if (elect_one()) {
#pragma unroll
                for (int step = 0; step < 8; ++step)
                  mma_ts(acc, as + step * 8, tc::smem_desc(xs + (step >> 2) * x_bytes + (step & 3) * 32, 16, 1024), idesc,
                         add || step);
                commit_pair(&freed[slot.at]);
                commit_pair(&xempty[x.at]);
              }
            }
            if (ok && elect_one()) commit_pair(&accfull[buf]);
          }
        }
        if (!ok && lane == 0) fail();
        // every product has ended before tensor memory is given back
        if (elect_one()) commit_own(&drain);
        wait_for(&drain, 0u);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  cluster_sync_all();
  tc::fence_after();
  if (warp == kWarpMma) tmem_free(tmem);
}

// Tokens' codes as halves: inputs 64 k .., token b: 128 bytes at (k * tokens + b) * 128, their 16-byte chunk j (inputs 8 j ..) at
// chunk position j ^ (b & 7). A thread widens 16 codes. The first clear the tickets, at most 150.
__global__ void k_lin8_widen(sffn_rows x, int B, int k, int runs, int tokens, uint4* xh, uint32_t* tickets, int n_tickets) {
  pdl_launch_dependents();
  pdl_wait();
  const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;   // at most 65536 tokens of 4096 runs, and a tile's padding
  if (i < n_tickets) tickets[i] = 0;
  const int b = i / runs, c = i % runs, col = c * 16;
  if (b >= tokens) return;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (b < B && col < k) v = __ldcg(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(x.ptr) + b * x.row_stride + col));
  uint4 lo, hi;
  l8_halves(v.x ^ 0x80808080u, lo.x, lo.y), l8_halves(v.y ^ 0x80808080u, lo.z, lo.w);
  l8_halves(v.z ^ 0x80808080u, hi.x, hi.y), l8_halves(v.w ^ 0x80808080u, hi.z, hi.w);
  uint4* row = xh + ((size_t)(c / 4) * tokens + b) * 8;
  const int j = (c & 3) * 2, w = b & 7;
  row[j ^ w] = lo, row[(j + 1) ^ w] = hi;
}

// Tokens of a tile and tiles of tokens.
struct TcShape {
  int nt, token_tiles, tokens;
};
TcShape tc_shape(int B) {
  TcShape s;
  s.token_tiles = (B + kMaxTokens - 1) / kMaxTokens;
  s.nt = ((B + s.token_tiles - 1) / s.token_tiles + 15) / 16 * 16;
  s.tokens = s.nt * s.token_tiles;
  return s;
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct TcWs {
  size_t xh, parts, total;   // the tickets come first
};
TcWs tc_ws(const sffn_linear8& L, const TcShape& s) {
  TcWs w;
  w.xh = up256((size_t)L.num_sms * sizeof(uint32_t));
  w.parts = w.xh + up256((size_t)s.tokens * L.kp * 2);
  const int nt = s.token_tiles > 1 ? kMaxTokens : s.nt;   // the workspace of a batch serves every smaller one
  w.total = w.parts + (size_t)L.num_sms * 2 * nt * kL8Rows * 4;
  return w;
}

}  // namespace

cudaError_t configure_linear8_tc(const sffn_linear8& L) {
  int optin = 0;
  cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, L.device);
  return e == cudaSuccess ? set_dynamic_smem_max(k_lin8_tc, optin) : e;
}

size_t linear8_tc_ws_bytes(const sffn_linear8& L, int B) { return tc_ws(L, tc_shape(B)).total; }

cudaError_t launch_linear8_tc(const sffn_linear8& L, const sffn_rows& x, const float* x_scales, int B,
                              const sffn_rows& residual, const sffn_rows& y, int dtype, void* ws, cudaStream_t st) {
  const TcShape s = tc_shape(B);
  const TcWs w = tc_ws(L, s);
  uint8_t* base = static_cast<uint8_t*>(ws);
  TcArgs a = {};
  a.codes = L.codes, a.xh = base + w.xh, a.scales = L.scales, a.bias = L.bias, a.x_scales = x_scales;
  a.residual = residual, a.y = y, a.tickets = static_cast<uint32_t*>(ws);
  a.parts = reinterpret_cast<int32_t*>(base + w.parts);
  a.err = L.err, a.n = L.desc.out_features, a.B = B, a.dtype = dtype, a.steps = L.kp / kStep;
  a.nt = s.nt, a.token_tiles = s.token_tiles, a.tokens = s.tokens;
  a.split = l8_split(L.tiles / CG * a.token_tiles, a.steps, L.num_sms / CG);
  const int runs = L.kp / 16;
  const unsigned threads = (unsigned)s.tokens * runs;
  cudaError_t e = launch_ex(k_lin8_widen, dim3((threads + 255) / 256), dim3(256), 0, st, true, 1, x, B, L.desc.in_features,
                            runs, s.tokens, reinterpret_cast<uint4*>(base + w.xh), a.tickets, a.split.left * CG);
  if (e != cudaSuccess) return e;
  const int smem = 1024 + kStagesW * kStepW + kStagesX * (a.nt / CG * 256);
  return launch_ex(k_lin8_tc, dim3((a.split.whole ? a.split.groups : a.split.parted) * CG), dim3(kTcThreads), smem, st, true, CG, a);
}

}  // namespace sffn
