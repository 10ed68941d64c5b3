// The 8-bit linear layer for many tokens, on the fifth-generation tensor cores.
//
// GB300 has no 8-bit whole-number kind of the product, so codes become halves
// on the way (linear8.cuh). The rows of the layer are the product's operand A:
// 128 of them a block, whose codes arrive in shared memory by bulk copies, are
// widened in registers by the thread of their row and written to tensor memory,
// from where the product takes A, so that the widened codes cross shared memory
// neither way. The tokens are operand B, widened once by k_lin8_widen before
// and laid out in the order in which a tile's rows stand in shared memory
// (128-byte swizzle), so that a tile is one run of bytes. CG = 2: two blocks of
// a cluster work on 256 rows together and hold half of the tokens each.
//
// Sums leave their fp32 accumulators as whole numbers every 1024 inputs, into
// registers, while the product goes on in a second accumulator.
//
// Tiles that fill whole waves are computed one at a time; the steps (of 64
// inputs) of those left over are shared out evenly. A block that has part of
// a tile leaves its sums in the workspace, and whichever comes last adds them:
// whole numbers, so that the order does not matter.
#include <algorithm>

#include "linear8.cuh"
#include "rows_io.cuh"
#include "step.h"
#include "tcgen05.cuh"

namespace sffn {

namespace {

constexpr int kConvWarps = 4, kEpiWarps = 8, kTcThreads = 512;
constexpr int kWarpW = 12, kWarpX = 13, kWarpMma = 14;   // one thread each; warps 0-3 widen, 4-11 take the sums
constexpr int kMaxTokens = 192;                          // of a tile
constexpr int kSlots = 4, kSlotCols = 32;                // of A in tensor memory
constexpr int kAccCols = 192, kTmemCols = 512;           // accumulators at 0 and 192, A at 384
constexpr int kStagesW = 8, kMaxStagesX = 8;
constexpr int kStepsExact = kL8Exact / kL8Inputs;
constexpr bool kPair = false;
constexpr int kLeastSteps = 8;                           // of a tile that a block takes a part of

struct TcArgs {
  const uint8_t* codes;   // [tiles of 128 rows][steps][8 KB]
  const uint8_t* xh;      // [steps][tokens][128 bytes]
  const float* scales;
  const float* bias;
  const float* x_scales;
  sffn_rows residual, y;
  int32_t* parts;         // [block][2][tokens of a tile][128]
  uint32_t* tickets;      // [tiles left over][CG]
  uint32_t* err;
  int n, B, dtype, steps, nt, token_tiles, tokens;   // nt: tokens of a tile; tokens: token_tiles * nt
  int stages_x, groups;                              // groups: clusters
  int whole, left, parted;                           // whole waves of tiles, tiles after them, clusters that share those
};

// What a cluster computes: tiles cluster + i * groups for i < whole, then its share [from, to) of the steps left over.
struct Segment {
  int tile, s0, s1;
  bool part;    // others have the rest of the tile
  int slot;     // of the workspace, for its sums
};
struct Segments {
  int cluster, i = 0;
  long long at, to;
  __device__ Segments(const TcArgs& a, int c) : cluster(c) {
    const long long units = (long long)a.left * a.steps;
    at = c < a.parted ? units * c / a.parted : 0, to = c < a.parted ? units * (c + 1) / a.parted : 0;
  }
  __device__ bool next(const TcArgs& a, Segment& s) {
    if (i < a.whole) {
      s.tile = cluster + i * a.groups, s.s0 = 0, s.s1 = a.steps, s.part = false, s.slot = 0;
      ++i;
      return true;
    }
    if (at >= to) return false;
    const int t = (int)(at / a.steps);
    const long long begin = (long long)t * a.steps, end = min(begin + a.steps, to);
    s.tile = a.whole * a.groups + t, s.s0 = (int)(at - begin), s.s1 = (int)(end - begin);
    s.part = s.s1 - s.s0 < a.steps, s.slot = at == (long long)a.left * a.steps * cluster / a.parted ? 0 : 1;
    at = end;
    return true;
  }
};

__device__ __forceinline__ uint32_t block_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Arrives on the barrier of the pair's first block (CG = 2) or on its own.
template <int CG>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if (CG == 1) {
    mbar_arrive(bar);
  } else {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
  }
}

__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int CG>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  if (CG == 1) return mbar_wait_bounded(bar, parity);
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!try_wait_cluster(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// Instruction descriptor of kind::f16 with fp32 sums and halves on both sides, both K-major.
template <int CG>
__device__ __forceinline__ uint32_t half_desc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 * CG >> 4) << 24);
}

// d (tensor memory) += a (tensor memory) b (shared memory).
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool add) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// One arrival on the barrier (of both blocks) once the thread's products so far have completed.
template <int CG>
__device__ __forceinline__ void commit_to(uint64_t* bar) {
  if (CG == 1)
    tc::commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
  if (CG == 1) {
    tc::alloc(dst, kTmemCols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t t) {
  if (CG == 1)
    tc::dealloc(t, kTmemCols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(kTmemCols) : "memory");
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

// The barrier of the eight warps that take the sums.
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int CG>
__global__ void __launch_bounds__(kTcThreads, 1) k_lin8_tc(const TcArgs a) {
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* smem = dyn_smem + (1024 - (smem_u32(dyn_smem) & 1023)) % 1024;   // the swizzle counts from there
  __shared__ uint64_t wfull[kStagesW], wempty[kStagesW], xfull[kMaxStagesX], xempty[kMaxStagesX];
  __shared__ uint64_t ready[kSlots], aempty[kSlots], accfull[2], accempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 2 ? (int)block_rank() : 0, cluster = blockIdx.x / CG;
  const int x_bytes = a.nt / CG * 128;                    // of a step's tokens in this block
  uint8_t* ring_w = smem;
  uint8_t* ring_x = smem + kStagesW * kL8Block;
  if (tid == 0) {
    for (int s = 0; s < kStagesW; ++s) mbar_init(&wfull[s], 1), mbar_init(&wempty[s], kConvWarps);
    for (int s = 0; s < kMaxStagesX; ++s) mbar_init(&xfull[s], 1), mbar_init(&xempty[s], 1);
    for (int s = 0; s < kSlots; ++s) mbar_init(&ready[s], kConvWarps * CG), mbar_init(&aempty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&accfull[s], 1), mbar_init(&accempty[s], kEpiWarps * CG);
    mbar_init(&drain, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == kWarpMma) tmem_alloc<CG>(&s_tmem);
  tc::fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();   // the other block's barriers are initialised too
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  pdl_launch_dependents();

  auto fail = [&]() {
    set_device_error(a.err, SFFN_ERR_TIMEOUT);
    atomicExch(&s_abort, 1);
  };
  auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };
  Segments work(a, cluster);
  Segment seg;

  if (warp == kWarpW) {
    // ------------------------------------------------------------ codes; they are no earlier kernel's
    if (lane == 0) {
      const uint64_t policy = a.token_tiles > 1 ? tc::l2_policy_evict_last() : l2_policy_evict_first();
      int it = 0;
      bool ok = true;
      while (ok && work.next(a, seg)) {
        const int row_tile = seg.tile / a.token_tiles * CG + rank;
        const uint8_t* src = a.codes + ((size_t)row_tile * a.steps + seg.s0) * kL8Block;
        for (int k = seg.s0; k < seg.s1; ++k, ++it, src += kL8Block) {
          const int s = it % kStagesW;
          ok = it < kStagesW || mbar_wait_bounded(&wempty[s], (uint32_t)((it / kStagesW - 1) & 1));
          if (!ok || aborted()) break;
          mbar_arrive_expect_tx(&wfull[s], kL8Block);
          bulk_g2s(ring_w + s * kL8Block, src, kL8Block, &wfull[s], policy);
        }
        if (!ok) fail();
        if (aborted()) break;
      }
      if (aborted())   // copies in flight land before the block ends
        for (int q = max(0, it - kStagesW); q < it; ++q) mbar_wait_bounded(&wfull[q % kStagesW], (uint32_t)((q / kStagesW) & 1));
    }
    pdl_wait();
  } else if (warp == kWarpX) {
    // ------------------------------------------------------------ tokens
    pdl_wait();
    if (lane == 0) {
      const uint64_t policy = tc::l2_policy_evict_last();
      int it = 0;
      bool ok = true;
      while (ok && work.next(a, seg)) {
        const int token0 = seg.tile % a.token_tiles * a.nt + rank * (a.nt / CG);
        const uint8_t* src = a.xh + ((size_t)seg.s0 * a.tokens + token0) * 128;
        for (int k = seg.s0; k < seg.s1; ++k, ++it, src += (size_t)a.tokens * 128) {
          const int s = it % a.stages_x;
          ok = it < a.stages_x || wait_for<CG>(&xempty[s], (uint32_t)((it / a.stages_x - 1) & 1));
          if (!ok || aborted()) break;
          mbar_arrive_expect_tx(&xfull[s], x_bytes);
          bulk_g2s(ring_x + s * x_bytes, src, x_bytes, &xfull[s], policy);
        }
        if (!ok) fail();
        if (aborted()) break;
      }
      if (aborted())
        for (int q = max(0, it - a.stages_x); q < it; ++q)
          mbar_wait_bounded(&xfull[q % a.stages_x], (uint32_t)((q / a.stages_x) & 1));
    }
  } else if (warp < kConvWarps) {
    // ------------------------------------------------------------ codes to halves in tensor memory, a row a thread
    pdl_wait();
    const int row = tid;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16) + 2 * kAccCols;
    int it = 0;
    bool ok = true;
    while (ok && work.next(a, seg)) {
      for (int k = seg.s0; k < seg.s1; ++k, ++it) {
        const int s = it % kStagesW, sa = it % kSlots, sx = it % a.stages_x;
        ok = mbar_wait_bounded(&wfull[s], (uint32_t)((it / kStagesW) & 1));
        ok = __all_sync(SFFN_FULL_MASK, ok);
        if (!ok || __any_sync(SFFN_FULL_MASK, aborted())) break;
        uint32_t h[32];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint4 v = *reinterpret_cast<const uint4*>(ring_w + s * kL8Block + l8_chunk(row, t));
          l8_halves(v.x, h[8 * t], h[8 * t + 1]), l8_halves(v.y, h[8 * t + 2], h[8 * t + 3]);
          l8_halves(v.z, h[8 * t + 4], h[8 * t + 5]), l8_halves(v.w, h[8 * t + 6], h[8 * t + 7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[s]);
        ok = it < kSlots || wait_for<CG>(&aempty[sa], (uint32_t)((it / kSlots - 1) & 1));
        ok = __all_sync(SFFN_FULL_MASK, ok);
        if (!ok) break;
        tc::fence_after();
        tmem_store32(lane_base + sa * kSlotCols, h);
        tmem_store_wait();
        tc::fence_before();
        // the step's tokens too are there before the product is told
        ok = mbar_wait_bounded(&xfull[sx], (uint32_t)((it / a.stages_x) & 1));
        ok = __all_sync(SFFN_FULL_MASK, ok);
        if (!ok) break;
        if (lane == 0) arrive_first<CG>(&ready[sa]);
      }
      if (!ok && lane == 0) fail();
      if (__any_sync(SFFN_FULL_MASK, aborted())) break;
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ products, one thread of the pair
    pdl_wait();
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = half_desc<CG>(a.nt);
      int it = 0, chunk = 0;
      bool ok = true, issued = false;
      while (ok && work.next(a, seg)) {
        for (int k = seg.s0; ok && k < seg.s1;) {
          const int end = min(k + kStepsExact, seg.s1), buf = chunk & 1;
          ok = chunk < 2 || wait_for<CG>(&accempty[buf], (uint32_t)((chunk / 2 - 1) & 1));
          tc::fence_after();
          for (bool add = false; ok && k < end; ++k, ++it) {
            const int sa = it % kSlots, sx = it % a.stages_x;
            ok = wait_for<CG>(&ready[sa], (uint32_t)((it / kSlots) & 1));
            if (!ok || aborted()) break;
            tc::fence_after();
            const uint32_t xs = smem_u32(ring_x + sx * x_bytes), as = tmem + 2 * kAccCols + sa * kSlotCols;
#pragma unroll
            for (int step = 0; step < 4; ++step) {
              mma_ts<CG>(tmem + buf * kAccCols, as + step * 8, tc::smem_desc(xs + step * 32, 16, 1024), idesc, add);
              add = true;
            }
            commit_to<CG>(&aempty[sa]);
            commit_to<CG>(&xempty[sx]);
            issued = true;
          }
          if (!ok || aborted()) break;
          commit_to<CG>(&accfull[buf]);
          ++chunk;
        }
        if (!ok) fail();
        if (aborted()) break;
      }
      if (issued) {   // every product has ended before tensor memory is given back
        tc::fence_before();
        if (CG == 1)
          tc::commit(&drain);
        else
          asm volatile(
              "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&drain))
              : "memory");
        mbar_wait_bounded(&drain, 0u);
      }
    }
  } else if (warp >= kConvWarps && warp < kConvWarps + kEpiWarps) {
    // ------------------------------------------------------------ sums to whole numbers to outputs
    pdl_wait();
    const int q = warp & 3, half = (warp - kConvWarps) >> 2, blocks = a.nt / 16;
    const int b0 = half ? (blocks + 1) / 2 : 0, nb = half ? blocks - b0 : (blocks + 1) / 2;   // of 16 tokens, at most 6
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + b0 * 16;
    const int r = q * 32 + lane;
    int chunk = 0;
    bool ok = true;
    while (ok && work.next(a, seg)) {
      int sum[96];
#pragma unroll
      for (int i = 0; i < 96; ++i) sum[i] = 0;
      for (int k = seg.s0; k < seg.s1; k += kStepsExact, ++chunk) {
        const int buf = chunk & 1;
        ok = wait_for<CG>(&accfull[buf], (uint32_t)((chunk / 2) & 1));
        ok = __all_sync(SFFN_FULL_MASK, ok);
        if (!ok || __any_sync(SFFN_FULL_MASK, aborted())) break;
        tc::fence_after();
#pragma unroll
        for (int b = 0; b < 6; ++b)
          if (b < nb) {
            float v[16];
            tmem_load16(lane_base + buf * kAccCols + b * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[b * 16 + i] += __float2int_rn(v[i]);
          }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CG>(&accempty[buf]);
      }
      if (!ok && lane == 0) fail();
      if (__any_sync(SFFN_FULL_MASK, aborted())) break;
      const int row_tile = seg.tile / a.token_tiles * CG + rank, token0 = seg.tile % a.token_tiles * a.nt + b0 * 16;
      if (seg.part) {
        // this block's sums to its place; the last to arrive adds the others'
        const int left = seg.tile - a.whole * a.groups;
        const size_t tile_ints = (size_t)a.nt * kL8Rows;
        const size_t own = (size_t)b0 * 16 * kL8Rows + r;
        int32_t* mine = a.parts + ((size_t)blockIdx.x * 2 + seg.slot) * tile_ints + own;
#pragma unroll
        for (int i = 0; i < 96; ++i)
          if (i / 16 < nb) __stcg(mine + (size_t)i * kL8Rows, sum[i]);
        __threadfence();
        epilogue_barrier();
        // clusters that share the tile: those whose steps reach into it
        const long long units = (long long)a.left * a.steps, begin = (long long)left * a.steps, end = begin + a.steps;
        int first = (int)(begin * a.parted / units), last = (int)((end - 1) * a.parted / units);
        while (units * first / a.parted > begin) --first;
        while (units * (first + 1) / a.parted <= begin) ++first;
        while (units * last / a.parted >= end) --last;
        while (units * (last + 1) / a.parted < end) ++last;
        if (warp == kConvWarps && lane == 0)
          s_last = atomicAdd(&a.tickets[left * CG + rank], 1u) == (uint32_t)(last - first);
        epilogue_barrier();
        const bool join = s_last;
        epilogue_barrier();   // read by all before it is written again
        if (!join) continue;
        __threadfence();
        for (int c = first; c <= last; ++c) {
          if (c == cluster) continue;
          const int slot = units * c / a.parted >= begin ? 0 : 1;   // its first steps are this tile's, or its last
          const int32_t* other = a.parts + ((size_t)(c * CG + rank) * 2 + slot) * tile_ints + own;
#pragma unroll
          for (int i = 0; i < 96; ++i)
            if (i / 16 < nb) sum[i] += __ldcg(other + (size_t)i * kL8Rows);
        }
      }
      const int n = row_tile * kL8Rows + r;
      const float scale = a.scales[n], bias = a.bias[n];   // padded to whole tiles
#pragma unroll
      for (int i = 0; i < 96; ++i) {
        const int token = token0 + i;
        if (i / 16 < nb && token < a.B && n < a.n) {
          float v = l8_value(sum[i], scale, __ldcg(a.x_scales + token), bias);
          if (a.residual.ptr) v = __fadd_rn(v, ld_elem(a.residual.ptr, token * a.residual.row_stride + n, a.dtype));
          st_elem(a.y.ptr, token * a.y.row_stride + n, v, a.dtype);
        }
      }
      __syncwarp();
    }
  } else {
    pdl_wait();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc::fence_after();
  if (warp == kWarpMma) tmem_free<CG>(tmem);
}

// Tokens' codes as halves: step k, token b: 128 bytes at (k * tokens + b) * 128, their 16-byte chunk j (inputs 8 j ..) at
// chunk position j ^ (b & 7). A thread widens 16 codes. Clears the tickets.
__global__ void k_lin8_widen(sffn_rows x, int B, int k, int steps, int tokens, uint4* xh, uint32_t* tickets,
                             unsigned n_tickets) {
  pdl_launch_dependents();
  pdl_wait();
  const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;   // at most 65536 tokens of 4096 runs
  if (i < n_tickets) tickets[i] = 0;
  const int per = steps * 4, b = i / per, c = i % per, col = c * 16;
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
  size_t parts, tickets, total;
};
TcWs tc_ws(const sffn_linear8& L, const TcShape& s) {
  TcWs w;
  w.parts = up256((size_t)s.tokens * L.kp * 2);
  const int nt = s.token_tiles > 1 ? kMaxTokens : s.nt;   // the workspace of a batch serves every smaller one
  w.tickets = w.parts + up256((size_t)L.num_sms * 2 * nt * kL8Rows * 4);
  w.total = w.tickets + up256((size_t)L.num_sms * 2 * 4);
  return w;
}

template <int CG>
cudaError_t run_tc(const sffn_linear8& L, TcArgs a, cudaStream_t st) {
  a.groups = L.num_sms / CG;
  const int tiles = L.tiles / CG * a.token_tiles;
  a.whole = tiles / a.groups, a.left = tiles % a.groups;
  a.parted = a.left ? (int)std::min<long long>(a.groups, std::max<long long>(a.left, (long long)a.left * a.steps / kLeastSteps)) : 0;
  const int x_bytes = a.nt / CG * 128;
  a.stages_x = std::min(kMaxStagesX, 128 * 1024 / x_bytes);
  const int smem = 1024 + kStagesW * kL8Block + a.stages_x * x_bytes;
  const int clusters = a.whole ? a.groups : a.parted;
  return launch_ex(k_lin8_tc<CG>, dim3(clusters * CG), dim3(kTcThreads), smem, st, true, CG, a);
}

}  // namespace

cudaError_t configure_linear8_tc(const sffn_linear8& L) {
  int optin = 0;
  cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, L.device);
  if (e == cudaSuccess) e = set_dynamic_smem_max(k_lin8_tc<1>, optin);
  if (e == cudaSuccess) e = set_dynamic_smem_max(k_lin8_tc<2>, optin);
  return e;
}

size_t linear8_tc_ws_bytes(const sffn_linear8& L, int B) { return tc_ws(L, tc_shape(B)).total; }

cudaError_t launch_linear8_tc(const sffn_linear8& L, const sffn_rows& x, const float* x_scales, int B,
                              const sffn_rows& residual, const sffn_rows& y, int dtype, void* ws, cudaStream_t st) {
  const TcShape s = tc_shape(B);
  const TcWs w = tc_ws(L, s);
  uint8_t* base = static_cast<uint8_t*>(ws);
  TcArgs a = {};
  a.codes = L.codes, a.xh = base, a.scales = L.scales, a.bias = L.bias, a.x_scales = x_scales;
  a.residual = residual, a.y = y, a.parts = reinterpret_cast<int32_t*>(base + w.parts);
  a.tickets = reinterpret_cast<uint32_t*>(base + w.tickets), a.err = L.err;
  a.n = L.desc.out_features, a.B = B, a.dtype = dtype, a.steps = L.kp / kL8Inputs;
  a.nt = s.nt, a.token_tiles = s.token_tiles, a.tokens = s.tokens;
  const long long threads = std::max<long long>((long long)s.tokens * a.steps * 4, L.num_sms * 2);
  cudaError_t e = launch_ex(k_lin8_widen, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, true, 1, x, B,
                            L.desc.in_features, a.steps, s.tokens, reinterpret_cast<uint4*>(base), a.tickets,
                            L.num_sms * 2);
  if (e != cudaSuccess) return e;
  return kPair ? run_tc<2>(L, a, st) : run_tc<1>(L, a, st);
}

}  // namespace sffn
