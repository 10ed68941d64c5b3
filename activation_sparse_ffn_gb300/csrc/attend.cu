// Attention of decode tokens over the paged 4-bit cache.
//
// Mathematics. For query row r (a token and one of the gq query heads of a key
// head) and position j, in units of log2: S = f q_r . K_j with f = scale *
// log2(e). A cached key is mid + step * (2u - 15) per group of channels, so
// S / f = sum over groups (step * (q_g . (2u - 15)) + mid * sum(q_g)): the
// tensor cores multiply q with 2u - 15, exact as halves, and step and
// mid are applied once per group in fp32. In the same way sum_j p_j V_j = sum_j
// (p_j step_j) (2u_j - 15) + sum_j p_j mid_j, with the running maximum and sum
// of the softmax in fp32.
//
// Operands. Sixteen positions are the 16-row operand of the score product and
// eight query rows its 8-column operand; for the values, sixteen channels and
// again the eight rows. The weights change from the first product's result
// layout to the second's operand layout by an 8 x 8 transpose in registers.
//
// Arithmetic. A weight times its step is carried by two halves (22 bits) in two
// products, after a power of two per row and group that brings the largest of the
// unit to 2^13: what a row does not see, or sees with no weight, or the size of
// other groups leaves its bits alone. (One power of two from the unit's largest
// step, whoever sees it, cost 2 to 7% less: 24 ragged sequences with groups of 32
// 94 us, so 101; 131072 positions 52.6 and 54.1.) With one half the results of
// fp16 rows were a quarter further from the exact ones than fp32 arithmetic leaves
// them (2.7e-4 and 2.1e-4 of their norm). q of 16-bit rows (Exact = false) is one
// half: fp16 as it is, bf16 after a power of two per row and group, exactly down to
// 2^-30 of the group's largest; q of fp32 rows (Exact = true) is two halves after
// one. Codes are centred, because the tensor core truncates its sums: bare value codes, all
// weights being positive, add up over a long history (131072 positions of fp16
// rows: 2.3e-4 instead of 2.1e-4), bare key codes left the result of fp32 rows off
// by 1.3e-6 instead of 0.5e-6 and lse of 16-bit rows by 8e-8 instead of 3e-8, and
// cost q of 16-bit rows four bits. (Bare, they would be one mask per pair and no
// arithmetic: 32 x 32768 of bf16 265 us, centred 276.) The sums of one unit's
// positions leave the tensor core and are added up in fp32, like the denominator
// and the mids.
//
// Work split. The visible blocks of U positions (`units`) of every (sequence,
// key head, tile of eight rows) are numbered through, and each warp of the grid
// takes an equal run of that list, whatever the lengths are; where runs are long
// an item counts a unit more, for its beginning and end, and short items are kept
// within a block (kItem and kWhole below). A warp streams its
// units through a private ring in shared memory with bulk copies per page for
// keys, values and params, so warps never wait for one another in the loop.
// Rows whose units lie within one warp are finished by it; the others are
// merged within the block at its end, and those cut by a block border by the
// last of their blocks to end, in block order, so that the bits do not depend
// on which one that is. (A kernel of its own for that cost 3 to 8 us a call.)
//
// What bounds it. The warps' own instructions, of which an SM issues 1.5 to 2 a
// cycle here (registers allow 8 to 16 warps; fixed latencies and instruction
// fetches stand between them): 32 sequences of 32768, 64 heads over 8 of 128 in
// bf16, 1.14 GB, take 275 us, 4.1 TB/s; one sequence of 131072 51 us (2.8 TB/s)
// and in fp32 rows, which need two products for the scores too, 54; rows of 32
// codes a group need four times the params and scales, 24 ragged sequences up to
// 4099 of 32 heads 109 us (2.4 TB/s); eight proposed tokens of 16 heads a key
// head read each unit 16 times, 38 us; heads of 256, 8 sequences of 8192 of 32
// over 8, 64 us in bf16 and 70 in fp32 (a part of their registers spills). A
// call's beginning (lengths, page table, first copies) and end (parts of blocks
// through global memory) are 7 to 16 us of each: 33 positions take 8 us, 1024 12,
// 16384 19. Tiles of sixteen rows, which decode a unit for twice the rows, hold
// half as many units in registers and came out even or slower.
#include "attn.h"
#include "kv_layout.cuh"
#include "q4mma.cuh"
#include "rows_io.cuh"

namespace sffn {

namespace {

constexpr int kMaxWarps = 16;
constexpr int kRows = 8;   // query rows of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, int G, bool Exact>
struct Att {
  static constexpr int NG = D / G;
  static constexpr int U = D == 256 ? 32 : 64;             // positions of a unit
  // Positions whose code is unrolled: with four groups and 64 of them the step and weight registers spill (24 ragged
  // sequences: 129 us, with 32 of them 109); with fewer groups 32 are slower (131072 positions of fp32 rows: 58 us, with 64
  // of them 54; 32 x 32768 of bf16: 287 and 276; 4 x 8 x 16 rows of 64 channels: 41 and 38; the exception is two groups of
  // 16-bit rows, 8 x 4 x 8 rows over 8192: 97 and 103).
  static constexpr int SU = NG >= 4 ? 32 : U;
  static constexpr int kStage = U * (D + 8 * NG);          // bytes
  // as many warps as the registers of the inner loop and two stages each allow; where a few values spill all the same,
  // fewer warps were slower (32 x 32768 of bf16: 276 us with 12, 302 with 8 and no spills)
  static constexpr int kByRegs = D == 64 ? (Exact ? 12 : 16) : D == 128 && !Exact && NG < 4 ? 12 : 8;
  static constexpr int kBudget = 224 * 1024;
  static constexpr int kBySmem = kBudget / (2 * kStage);
  static constexpr int kWarps = (kByRegs < kBySmem ? kByRegs : kBySmem) / 4 * 4;   // the same on each of an SM's four schedulers
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = kStage * kWarps * 3 <= kBudget ? 3 : 2;
  static constexpr int kPitch = D + 4;                     // floats of a row of sums: rows two apart use other banks
  static constexpr int kPart = kRows * kPitch + 2 * kRows; // floats of a partial result: sums, maxima, totals
  // Items of up to so many units are not cut by a block border where the list has at most 32 sequences: another two units
  // a warp cost less than a join by way of global memory (8 rows over 1024 positions: 12.5 us, joined 14.1; with 16 rows of
  // each of 32 sequences of 512, D = 64: 15.5 and 19.0; three units a warp are no better). More sequences are placed by the
  // block, whose borders stay where they fall (33 of 512: 21.7).
  static constexpr int kWhole = 2 * kWarps;
  // What the beginning and the end of an item cost, in units; counted where warps take several units each, so that blocks
  // with many short items do not end last (24 ragged sequences: 117 us without, 109 with; two units instead of one are as
  // good there and cost 17.9 instead of 15.5 us with 16 rows of each of 32 sequences of 512).
  static constexpr int kItem = 1;
  static constexpr int kSmem = kStage * kStages * kWarps;
  static_assert(kWarps >= kRows && kWarps <= kMaxWarps && kSmem >= kPart * 4 * kWarps, "");
};

// Equal runs of a list of `total` units: block b of `blocks` takes those from
// floor(b * total / blocks), and so on for the warps of a block.
struct Runs {
  int total, per, rest, blocks;
  __device__ __forceinline__ Runs(int total_, int blocks_)
      : total(total_), per(total_ / blocks_), rest(total_ % blocks_), blocks(blocks_) {}
  __device__ __forceinline__ int start(int b) const { return per * b + rest * b / blocks; }
};
template <int W>
__device__ __forceinline__ int warp_start(int u0, int u1, int w) {
  const int n = u1 - u0;
  return u0 + n / W * w + n % W * w / W;
}

// The block that takes unit u: start(b) <= u holds exactly for b < (u + 1) * blocks / total.
__device__ __forceinline__ int block_of(int u, int total, int blocks) {
  return (int)((((long long)u + 1) * blocks - 1) / total);
}

// The number of blocks that have left their part of an item, in the low half of a word whose high half tells whether
// the word has been in use as such: the workspace comes with any contents.
constexpr unsigned long long kTicketMark = 0x9e3779b97f4a7c15ull & 0xffffffff00000000ull;
__device__ __forceinline__ int take_ticket(unsigned long long* word) {
  for (;;) {
    unsigned long long old = atomicAdd(word, 1ull);
    if ((old & 0xffffffff00000000ull) == kTicketMark) return (int)(uint32_t)old;
    // contents of before: the first block to replace them takes ticket 0, others count again
    for (++old; (old & 0xffffffff00000000ull) != kTicketMark;) {
      const unsigned long long seen = atomicCAS(word, old, kTicketMark | 1ull);
      if (seen == old) return 0;
      old = seen;
    }
  }
}

struct AttendArgs {
  const uint8_t* pages;
  size_t page_bytes, head_bytes;
  int n_pages, P, P_log2, hkv;
  uint32_t* err;
  sffn_kv_batch b;
  sffn_rows q, out;
  float* lse;
  int hq, gq, dtype, window;
  float scale;
  unsigned long long* tickets;   // [blocks], of the items that begin in a block and end in another
  float* warp_parts;   // [blocks * warps][kPart]
  float* block_parts;  // [blocks][2][kPart]
};

// A sequence's rows and length, made safe for indexing; n is -1 if the rows are out of order or not the call's.
struct Seq {
  int q0, n, len;
};

__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int s) {
  Seq q;
  q.len = kv_len_of(a.b, s, a.P, a.err);
  if (a.b.q_start) {
    KvSpan rows;
    const bool ok = kv_span(a.b, s, rows);
    q.q0 = rows.from;
    q.n = ok ? rows.to - rows.from : -1;
  } else {
    q.q0 = s;
    q.n = 1;
  }
  return q;
}

// Tiles of a sequence, and units given to each of them: enough for the widest
// visible range any eight consecutive rows can have, at least one.
__device__ __forceinline__ int tiles_of(const AttendArgs& a, const Seq& q) { return (q.n * a.gq + kRows - 1) / kRows; }
__device__ __forceinline__ int units_of(const AttendArgs& a, const Seq& q, int U) {
  int units = (q.len + U - 1) / U;
  if (a.window > 0) {
    const int span = min(q.n, (kRows - 2 + a.gq) / a.gq + 1);  // tokens that eight consecutive rows can touch
    const long long seen = (long long)a.window + span - 1;
    units = (int)min((long long)units, (seen + U - 2) / U + 1);
  }
  return max(units, 1);
}
__device__ __forceinline__ int items_of(const AttendArgs& a, const Seq& q) {
  return q.n > 0 ? a.hkv * tiles_of(a, q) : 0;
}

// A place in the list of units.
struct Cursor {
  int s, kh, tile, u;        // sequence, key head, tile, unit within the tile
  int tiles, units;          // of the sequence
  int q0, n, len;
  int base0, first, last;    // position of the tile's unit 0, of its first row, and of its last row
  int extra;                 // units past the last that an item is given for its beginning and end

  __device__ __forceinline__ void set_tile(const AttendArgs& a, int U) {
    const int r0 = tile * kRows, r1 = min(r0 + kRows, n * a.gq) - 1;
    first = len - n + r0 / a.gq;
    last = len - n + r1 / a.gq;
    const int lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
    base0 = lo / U * U;
  }
  __device__ __forceinline__ void set_seq(const AttendArgs& a, const Seq& q, int U) {
    q0 = q.q0, n = q.n, len = q.len;
    tiles = tiles_of(a, q);
    units = units_of(a, q, U) + extra;
  }
  __device__ __forceinline__ void advance(const AttendArgs& a, int U) {
    if (++u < units) return;
    u = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++kh == a.hkv) {
        kh = 0;
        Seq q;
        do {
          ++s;
          if (s >= a.b.n_seq) return;  // past the end of the list: never used
          q = load_seq(a, s);
        } while (q.n <= 0);
        set_seq(a, q, U);
      }
    }
    set_tile(a, U);
  }
  __device__ __forceinline__ int base(int U) const { return base0 + u * U; }
  __device__ __forceinline__ bool empty(int U) const { return base0 + u * U > last; }
};

template <int D>
__device__ __forceinline__ void write_row(const AttendArgs& a, int q0, int n, int kh, int row, int lane, const float* o,
                                          float m, float l) {
  // o: channels lane * (D/32) .. of the row
  constexpr int CPL = D / 32;
  if (row >= n * a.gq) return;
  const int i = q0 + row / a.gq, h = kh * a.gq + row % a.gq;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float v[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) v[e] = o[e] * inv;
  st_run<CPL>(a.out.ptr, (size_t)(i * a.out.row_stride + h * a.out.head_stride) + lane * CPL, a.dtype, v);
  if (a.lse && lane == 0)
    a.lse[(size_t)i * a.hq + h] = l == 0.f ? __int_as_float(0xff800000) : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, o));
  return v;
}

// A lane's channels of a row of sums, from shared or (written by another block or warp) global memory.
template <int N>
__device__ __forceinline__ void part_row(const float* p, bool in_smem, float* x) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2* q = reinterpret_cast<const float2*>(p + e);
    const float2 v = in_smem ? *q : __ldcg(q);
    x[e] = v.x, x[e + 1] = v.y;
  }
}

template <int D, int G, bool Exact>
__global__ void __launch_bounds__(Att<D, G, Exact>::kThreads, 1) k_attend(const AttendArgs a) {
  using T = Att<D, G, Exact>;
  constexpr int U = T::U, SU = T::SU, NG = T::NG, CPL = D / 32, kAttWarps = T::kWarps, kAttThreads = T::kThreads, kPitch = T::kPitch;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_bar[kAttWarps][T::kStages];
  __shared__ int s_scan[kAttWarps], s_seq[kAttWarps], s_off[kAttWarps];
  __shared__ Seq s_rows[kAttWarps];
  struct Entry {
    int item_start, item_end, q0, n, kh, tile, where;  // where: 0 none, 1 shared memory, 2 the warp's global slot
  };
  __shared__ Entry s_entry[2 * kAttWarps];
  __shared__ int s_last[2];   // whether the block is the last with a part of an item cut by its borders
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x < kAttWarps * T::kStages) mbar_init(&s_bar[0][0] + threadIdx.x, 1);
  if (threadIdx.x < 2 * kAttWarps) s_entry[threadIdx.x].where = 0;
  fence_mbar_init();
  __syncthreads();   // the first warps initialise the barriers and entries of all
  pdl_launch_dependents();
  pdl_wait();

  // ---- the block's and the warp's run of units, and the sequence of the warp's first unit
  Seq sq{0, 0, 0};       // that sequence's rows; before that, of the sequence a thread looks at
  int mine = 0, items = 0, total, lo_u = 0, first_seq = 0, first_off = 0, extra = 0;
  bool bad = false;      // starts out of order: rows could lie in many sequences and the list outgrow 32 bits
  auto look = [&](int s) {
    mine = items = 0;
    if (s < a.b.n_seq) {
      sq = load_seq(a, s);
      bad |= sq.n < 0;
      items = items_of(a, sq);
      if (items) mine = items * (units_of(a, sq, U) + extra);
    }
  };
  auto warp_scan = [&](int v) {   // sum over this and earlier lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(SFFN_FULL_MASK, v, o);
      if (lane >= o) v += w;
    }
    return v;
  };
  int block_u0, block_u1, u0, u1;
  auto extra_of = [&](int units) { return units > (int)gridDim.x * kAttWarps ? T::kItem : 0; };
  auto warp_run = [&]() {
    u0 = warp_start<kAttWarps>(block_u0, block_u1, warp), u1 = warp_start<kAttWarps>(block_u0, block_u1, warp + 1);
  };
  if (a.b.n_seq <= 32) {   // each warp on its own, lane s for sequence s
    look(lane);
    if (__any_sync(SFFN_FULL_MASK, bad)) {
      if (bad) set_device_error(a.err, SFFN_ERR_DEVICE);
      return;
    }
    extra = extra_of(__reduce_add_sync(SFFN_FULL_MASK, mine));
    mine += items * extra;
    const int upto = warp_scan(mine);
    total = __shfl_sync(SFFN_FULL_MASK, upto, 31);
    const Runs runs(total, gridDim.x);
    auto owner = [&](int u) { return __ffs(__ballot_sync(SFFN_FULL_MASK, u < upto)) - 1; };
    // a border within a short item moves to the nearer end of it
    const int item_units = mine ? mine / items : 1;
    auto border = [&](int b) {
      const int u = runs.start(b), src = max(owner(u), 0);
      const int off = u - __shfl_sync(SFFN_FULL_MASK, upto - mine, src), n = __shfl_sync(SFFN_FULL_MASK, item_units, src);
      if (u >= total || n == 1 || n - extra > T::kWhole) return u;
      const int past = off % n;
      return 2 * past <= n ? u - past : u - past + n;
    };
    block_u0 = border(blockIdx.x), block_u1 = border(blockIdx.x + 1);
    warp_run();
    const int src = owner(u0);
    if (src >= 0) {
      first_seq = src;
      first_off = u0 - __shfl_sync(SFFN_FULL_MASK, upto - mine, src);
      sq.q0 = __shfl_sync(SFFN_FULL_MASK, sq.q0, src);
      sq.n = __shfl_sync(SFFN_FULL_MASK, sq.n, src);
      sq.len = __shfl_sync(SFFN_FULL_MASK, sq.len, src);
    }
  } else {                 // the block together, once for the total and once for the places
    auto block_scan = [&](int v, int& sum) {   // sum over earlier threads; over all of them
      const int upto = warp_scan(v);
      __syncthreads();
      if (lane == 31) s_scan[warp] = upto;
      __syncthreads();
      int below = 0;
      sum = 0;
#pragma unroll 1
      for (int w = 0; w < kAttWarps; ++w) {
        if (w < warp) below += s_scan[w];
        sum += s_scan[w];
      }
      return below + upto - v;
    };
    int all_items = 0;
    for (int s = threadIdx.x; s < a.b.n_seq; s += kAttThreads) {
      look(s);
      lo_u += mine;
      all_items += items;
    }
    if (__syncthreads_or(bad)) {
      if (bad) set_device_error(a.err, SFFN_ERR_DEVICE);
      return;
    }
    block_scan(lo_u, total);
    extra = extra_of(total);
    if (extra) {
      block_scan(all_items, all_items);
      total += all_items * extra;
    }
    const Runs runs(total, gridDim.x);
    block_u0 = runs.start(blockIdx.x), block_u1 = runs.start(blockIdx.x + 1);
    warp_run();
    int before = 0;
    for (int s0 = 0; s0 < a.b.n_seq; s0 += kAttThreads) {
      look(s0 + threadIdx.x);
      int sum;
      lo_u = before + block_scan(mine, sum);
      before += sum;
#pragma unroll 1
      for (int w = 0; w < kAttWarps; ++w) {
        const int want = warp_start<kAttWarps>(block_u0, block_u1, w);
        if (want >= lo_u && want < lo_u + mine) {
          s_seq[w] = s0 + threadIdx.x;
          s_off[w] = want - lo_u;
          s_rows[w] = sq;
        }
      }
    }
    __syncthreads();
    first_seq = s_seq[warp], first_off = s_off[warp], sq = s_rows[warp];   // of use if the warp's start is below total
  }

  const bool any = u0 < u1;
  Cursor cur{};
  if (any) {
    cur.s = first_seq;
    cur.extra = extra;
    cur.set_seq(a, sq, U);
    const int item = first_off / cur.units;
    cur.u = first_off - item * cur.units;
    cur.kh = item / cur.tiles;
    cur.tile = item - cur.kh * cur.tiles;
    cur.set_tile(a, U);
  }

  // ---- copies: the warp's ring
  // 2^rp_log2 positions of a unit share a page; `parts` such runs make up the unit
  const int rp_log2 = min(a.P_log2, U == 32 ? 5 : 6), RP = 1 << rp_log2, parts = U >> rp_log2;
  const uint64_t pol = l2_policy_evict_first();
  uint8_t* ring = smem + (size_t)warp * T::kStages * T::kStage;
  Cursor nxt = cur;
  int nu = u0;             // next unit to copy
  int issued = 0, taken = 0;
  auto slot_of = [](int k) { return k % T::kStages; };
  auto phase_of = [](int k) { return (uint32_t)(k / T::kStages) & 1u; };
  int page = 0;            // lane i: page of run i of unit nu
  auto fetch_page = [&]() {
    if (nu < u1 && !nxt.empty(U)) {
      const int base = nxt.base(U);
      if (lane < parts && base + lane * RP <= nxt.last)
        page = ld_dep(a.b.table + (size_t)nxt.s * a.b.table_stride + ((base + lane * RP) >> a.P_log2));
    }
  };
  // copies the next unit that shows something; false: none left
  auto issue = [&]() {
    while (nu < u1 && nxt.empty(U)) {
      nxt.advance(a, U);
      ++nu;
      fetch_page();
    }
    if (nu >= u1) return;
    const int st = slot_of(issued), base = nxt.base(U);
    uint8_t* dst = ring + st * T::kStage;
    const int n_runs = min(parts, ((nxt.last - base) >> rp_log2) + 1);
    // runs that lie before the window hold nothing any row sees, and their pages may be gone
    const int run0 = a.window > 0 ? max(0, nxt.first - a.window + 1 - base) >> rp_log2 : 0;
    if (lane == 0) mbar_arrive_expect_tx(&s_bar[warp][st], (uint32_t)(((n_runs - run0) << rp_log2) * (D + 8 * NG)));
    __syncwarp();
    if (lane >= run0 && lane < n_runs) {
      if (page < 0 || page >= a.n_pages) {
        set_device_error(a.err, SFFN_ERR_DEVICE);
        page = 0;
      }
      const uint8_t* src = a.pages + (size_t)page * a.page_bytes + (size_t)nxt.kh * a.head_bytes;
      const int slot = base & (a.P - 1);  // zero unless a page holds several units
      bulk_g2s(dst + lane * RP * (D / 2), src + slot * (D / 2), RP * (D / 2), &s_bar[warp][st], pol);
      bulk_g2s(dst + U * (D / 2) + lane * RP * (D / 2), src + kv_value_off(a.P, D) + slot * (D / 2), RP * (D / 2),
               &s_bar[warp][st], pol);
      bulk_g2s(dst + U * D + lane * RP * 8 * NG, src + kv_param_off(a.P, D) + slot * 8 * NG, RP * 8 * NG,
               &s_bar[warp][st], pol);
    }
    __syncwarp();
    ++issued;
    nxt.advance(a, U);
    ++nu;
    fetch_page();
  };
  if (any) fetch_page();

  const int dtype = Exact ? (int)SFFN_F32 : a.dtype;
  const float ninf = __int_as_float(0xff800000);
  constexpr int QL = Exact ? 2 : 1;          // halves that carry a query element
  uint32_t q[QL][D / 16][2];                 // column g of the operand
  float qs[NG][2];                           // sums of q over a group, rows 2t and 2t + 1 as everything below
  float gs[NG][2];                           // what the products of a group are multiplied with to match the row's others
  float o[D / 16][4];                        // channels 16x + g and 16x + 8 + g, each for both rows
  float l[2] = {0.f, 0.f};                   // the lane's share of sum p
  float mid_sum[NG][2];                      // and of sum p mid
  float f[2] = {1.f, 1.f}, m[2] = {ninf, ninf};
  int pos[2], lo[2];                         // position of the row and the first it sees
  bool dead = false, fresh = true;
  int item_start = u0 - cur.u;
  const int kt = kv_pos_of_col(g);           // position, of eight, of row g of a key operand
  const int ta = kv_pos_of_col(2 * t), tb = kv_pos_of_col(2 * t + 1);  // of columns 2t, 2t + 1 of a value operand

  // after a wait that ran out: copies still under way must land before the ring is used for anything else
  auto drain = [&]() {
    if (dead)
      for (; taken < issued; ++taken) mbar_wait_bounded(&s_bar[warp][slot_of(taken)], phase_of(taken));
  };
  // the end of a segment, the warp's units of one item; true: the whole item lies within the warp
  auto finish = [&](bool last) {
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float s = row_sum(mid_sum[n][r]);
#pragma unroll
        for (int x = n * G / 16; x < (n + 1) * G / 16; ++x) o[x][r] += s, o[x][2 + r] += s;
      }
    const float lt[2] = {row_sum(l[0]), row_sum(l[1])};
    const float mt[2] = {m[0] == ninf ? ninf : m[0] * f[0], m[1] == ninf ? ninf : m[1] * f[1]};
    const int item_end = item_start + cur.units;
    if (item_start >= u0 && item_end <= u1) {   // finish the rows here
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = cur.tile * kRows + 2 * t + r;
        if (row >= cur.n * a.gq) continue;
        const int i = cur.q0 + row / a.gq, h = cur.kh * a.gq + row % a.gq;
        const size_t at = (size_t)(i * a.out.row_stride + h * a.out.head_stride) + g;
        const float inv = lt[r] == 0.f ? 0.f : 1.f / lt[r];
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          st_elem(a.out.ptr, at + 16 * x, o[x][r] * inv, dtype);
          st_elem(a.out.ptr, at + 16 * x + 8, o[x][2 + r] * inv, dtype);
        }
        if (a.lse && g == 0) a.lse[(size_t)i * a.hq + h] = lt[r] == 0.f ? ninf : (mt[r] + log2f(lt[r])) * kLn2;
      }
      return true;
    }
    // the last segment of the warp goes to shared memory (once every ring is idle), an earlier one to the warp's slot
    if (last) {
      drain();
      __syncthreads();
    }
    float* dst = last ? reinterpret_cast<float*>(smem) + warp * T::kPart : a.warp_parts + (size_t)(blockIdx.x * kAttWarps + warp) * T::kPart;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float* row = dst + (2 * t + r) * kPitch + g;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) row[16 * x] = o[x][r], row[16 * x + 8] = o[x][2 + r];
      if (g == 0) {
        dst[kRows * kPitch + 2 * t + r] = mt[r];
        dst[kRows * kPitch + kRows + 2 * t + r] = lt[r];
      }
    }
    if (lane == 0) {
      Entry& e = s_entry[2 * warp + (last ? 1 : 0)];
      e.item_start = item_start, e.item_end = item_end;
      e.q0 = cur.q0, e.n = cur.n, e.kh = cur.kh, e.tile = cur.tile;
      e.where = last ? 1 : 2;
    }
    return false;
  };

  // SU positions of a unit, from its copy in shared memory
  auto unit = [&](auto masked, const uint8_t* sk, const uint8_t* sv, const uint8_t* sp, int base) {
    constexpr bool Masked = decltype(masked)::value;   // some row does not see some of the positions
    const int lo_min = a.window > 0 ? max(0, cur.first - a.window + 1) : 0;   // before it nothing is seen
    // the (step, mid) pairs of slot g of eight positions, all groups
    auto params = [&](int tile, int which, uint32_t* v) {
      const uint8_t* at = sp + tile * NG * 64 + which * NG * 32 + g * NG * 4;
      if (NG == 1) {
        v[0] = *reinterpret_cast<const uint32_t*>(at);
      } else if (NG == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        v[0] = x.x, v[1 % NG] = x.y;
      } else {
#pragma unroll
        for (int n = 0; n < NG; n += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(at + 4 * n);
          v[n] = x.x, v[(n + 1) % NG] = x.y, v[(n + 2) % NG] = x.z, v[(n + 3) % NG] = x.w;
        }
      }
    };

    // ---- scores of U positions: s[i] rows 16i + slot g and 16i + 8 + slot g, each for both query rows
    float s[SU / 16][4];
#pragma unroll
    for (int i = 0; i < SU / 16; ++i) {
      uint32_t w[2][D / 32];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint8_t* row = sk + (16 * i + 8 * k + kt) * (D / 2);
        if (D == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(row + key_word_off<D>(kt, t, 0));
          w[k][0] = v.x, w[k][1] = v.y;
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; j += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + key_word_off<D>(kt, t, j));
            w[k][j] = v.x, w[k][j + 1] = v.y, w[k][j + 2] = v.z, w[k][j + 3] = v.w;
          }
        }
      }
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      uint32_t kp[2][NG];
      params(2 * i, 0, kp[0]);
      params(2 * i + 1, 0, kp[1]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = n * G / 32; j < (n + 1) * G / 32; ++j) {
          uint32_t p0[4], p1[4];
          key_halves(w[0][j], p0);
          key_halves(w[1][j], p1);
          const uint32_t a0[4] = {p0[0], p1[0], p0[1], p1[1]}, a1[4] = {p0[2], p1[2], p0[3], p1[3]};
#pragma unroll
          for (int h = 0; h < QL; ++h) {
            mma_f16(c, a0, q[h][2 * j][0], q[h][2 * j][1]);
            mma_f16(c, a1, q[h][2 * j + 1][0], q[h][2 * j + 1][1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 sm = __half22float2(u32_h2(kp[k][n]));
          const float st[2] = {NG == 1 ? sm.x : sm.x * gs[n][0], NG == 1 ? sm.x : sm.x * gs[n][1]};
          s[i][2 * k] = fmaf(st[0], c[2 * k], fmaf(sm.y, qs[n][0], s[i][2 * k]));
          s[i][2 * k + 1] = fmaf(st[1], c[2 * k + 1], fmaf(sm.y, qs[n][1], s[i][2 * k + 1]));
        }
      }
    }
    uint32_t unseen = 0u;   // bit 4i + e: the row does not see the position of s[i][e]
    if (Masked) {
#pragma unroll
      for (int i = 0; i < SU / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = base + 16 * i + 8 * (e >> 1) + kt;
          if (j > pos[e & 1] || j < lo[e & 1]) s[i][e] = ninf, unseen |= 1u << (4 * i + e);
        }
    }
    float mu[2] = {m[0], m[1]};
#pragma unroll
    for (int i = 0; i < SU / 16; ++i) {
      mu[0] = fmaxf(mu[0], fmaxf(s[i][0], s[i][2]));
      mu[1] = fmaxf(mu[1], fmaxf(s[i][1], s[i][3]));
    }
    mu[0] = row_max(mu[0]);
    mu[1] = row_max(mu[1]);
    if (__any_sync(SFFN_FULL_MASK, mu[0] > m[0] || mu[1] > m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float back = mu[r] == m[r] ? 1.f : ex2((m[r] - mu[r]) * f[r]);   // m = -inf: 0
        m[r] = mu[r];
        l[r] *= back;
#pragma unroll
        for (int n = 0; n < NG; ++n) mid_sum[n][r] *= back;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) o[x][r] *= back, o[x][2 + r] *= back;
      }
    }
    const float mf[2] = {m[0] == ninf ? 0.f : m[0] * f[0], m[1] == ninf ? 0.f : m[1] * f[1]};

    uint32_t vw[SU / 16][4][D / 64];   // the lane's words of four positions per 16
#pragma unroll
    for (int k = 0; k < SU / 16; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int p8 = (r & 1) ? tb : ta;
        const uint8_t* c = sv + (16 * k + 8 * (r >> 1) + p8) * (D / 2) + value_word_off<D>(p8, g, 0);
        if (D == 64) {
          vw[k][r][0] = *reinterpret_cast<const uint32_t*>(c);
        } else if (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2*>(c);
          vw[k][r][0] = v.x, vw[k][r][1 % (D / 64)] = v.y;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(c);
          vw[k][r][0] = v.x, vw[k][r][1 % (D / 64)] = v.y, vw[k][r][2 % (D / 64)] = v.z, vw[k][r][3 % (D / 64)] = v.w;
        }
      }
    constexpr int GW = G >= 64 ? 1 : 64 / G;   // groups that the 64 channels of a word lie in

    float step[SU / 16][2][NG];
#pragma unroll
    for (int i = 0; i < SU / 16; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = ex2(fmaf(s[i][e], f[e & 1], -mf[e & 1]));
      l[0] += s[i][0] + s[i][2];
      l[1] += s[i][1] + s[i][3];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t vp[NG];
        params(2 * i + k, 1, vp);
        if (Masked) {   // what no row sees is cleared; the weights of rows that do not see it are 0 already
          const int j = base + 16 * i + 8 * k + kt;
          if (j > cur.last || j < lo_min) {
#pragma unroll
            for (int n = 0; n < NG; ++n) vp[n] = 0u;
          }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const float2 sm = __half22float2(u32_h2(vp[n]));
          step[i][k][n] = sm.x;
          mid_sum[n][0] = fmaf(s[i][2 * k], sm.y, mid_sum[n][0]);
          mid_sum[n][1] = fmaf(s[i][2 * k + 1], sm.y, mid_sum[n][1]);
        }
      }
    }
    float down[GW][2];   // of a group and query row
    uint32_t wt[2][GW][SU / 16][2];
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      if (w * 64 % G == 0) {
#pragma unroll
        for (int n = 0; n < GW; ++n) {
          float x[SU / 16][4], top[2] = {0.f, 0.f}, up[2];
#pragma unroll
          for (int i = 0; i < SU / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[i][e] = s[i][e] * step[i][e >> 1][w * 64 / G + n];
              if (Masked) {   // a step may be NaN for the rows that see it, also where their weight has become 0
                if (unseen >> (4 * i + e) & 1u) x[i][e] = 0.f;
              }
              top[e & 1] = fmaxf(top[e & 1], x[i][e]);
            }
          // the upper halves of both maxima, which order as they do and hold the exponents, in one word
          uint32_t both = __byte_perm(__float_as_uint(top[0]), __float_as_uint(top[1]), 0x7632);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) both = __vmaxu2(both, __shfl_xor_sync(SFFN_FULL_MASK, both, o));
          scale_to_half_range(__uint_as_float(both << 16), up[0], down[n][0]);
          scale_to_half_range(__uint_as_float(both), up[1], down[n][1]);
#pragma unroll
          for (int i = 0; i < SU / 16; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t hi, lw;
              split_f16(x[i][2 * k] * up[0], x[i][2 * k + 1] * up[1], hi, lw);
              wt[0][n][i][k] = transpose_8x8(hi);
              wt[1][n][i][k] = transpose_8x8(lw);
            }
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float acc[2][4];
#pragma unroll
        for (int k = 0; k < SU / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {   // channel tiles 4 hh + 2e and the next
            const int n = (2 * hh + e) * 16 / G % GW;
            // the low and the high nibble of a byte
            const int pick = hh ? (e ? 0x6723 : 0x7632) : (e ? 0x4501 : 0x5410);
            const uint32_t x0 = __byte_perm(vw[k][0][w], vw[k][1][w], pick);
            const uint32_t x1 = __byte_perm(vw[k][2][w], vw[k][3][w], pick);
            const uint32_t av[4] = {value_low(x0), value_high(x0), value_low(x1), value_high(x1)};
            if (k == 0) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
            mma_f16(acc[e], av, wt[0][n][k][0], wt[0][n][k][1]);
            mma_f16(acc[e], av, wt[1][n][k][0], wt[1][n][k][1]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* ox = o[4 * w + 2 * hh + e];
          const float* dn = down[(2 * hh + e) * 16 / G % GW];
          ox[0] = fmaf(acc[e][0], dn[0], ox[0]);
          ox[1] = fmaf(acc[e][1], dn[1], ox[1]);
          ox[2] = fmaf(acc[e][2], dn[0], ox[2]);
          ox[3] = fmaf(acc[e][3], dn[1], ox[3]);
        }
      }
    }
  };

  bool at_barrier = false;
  for (int uu = u0; uu < u1; ++uu) {
    if (fresh) {   // first unit of the warp in this item: query rows
      fresh = false;
      item_start = uu - cur.u;
      const int rows = cur.n * a.gq, row = cur.tile * kRows + g, rg = min(row, rows - 1);
      const int pos_g = cur.len - cur.n + rg / a.gq;
      const int lo_g = a.window > 0 ? max(0, pos_g - a.window + 1) : 0;
      const size_t at = (size_t)((cur.q0 + rg / a.gq) * a.q.row_stride + (cur.kh * a.gq + rg % a.gq) * a.q.head_stride);
      // the sign of the scale goes with q, its size with f; rows past the end are zero
      const float sign = row >= rows || a.scale == 0.f ? 0.f : a.scale < 0.f ? -1.f : 1.f;
      float big[NG], fg[NG], up[NG], sum[NG], x[D / 32][8];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) ld_run<8>(a.q.ptr, at + 32 * j + 8 * t, dtype, x[j]);
      if (uu == u0) {   // the first copies, while the rows are on their way
#pragma unroll 1
        for (int i = 0; i < T::kStages - 1; ++i) issue();
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) big[n] = sum[n] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) big[j * 32 / G] = fmaxf(big[j * 32 / G], fabsf(x[j][e]));
      float row_fg = 0.f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        scale_to_half_range(quad_max(big[n]), up[n], fg[n]);
        if (!Exact && dtype == SFFN_F16) up[n] = fg[n] = 1.f;   // fp16 rows are taken as they are
        row_fg = fmaxf(row_fg, fg[n]);
      }
      const float f_g = a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * kLog2e * row_fg, 1.1754944e-38f);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[j][e] = sign == 0.f ? 0.f : x[j][e] * (up[j * 32 / G] * sign);
          sum[j * 32 / G] += x[j][e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t* hi = &q[0][2 * j + (e >> 1)][e & 1];
          if (Exact)
            split_f16(x[j][2 * e], x[j][2 * e + 1], *hi, q[QL - 1][2 * j + (e >> 1)][e & 1]);
          else
            *hi = h2_u32(__floats2half2_rn(x[j][2 * e], x[j][2 * e + 1]));
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        fg[n] /= row_fg;   // powers of two
        sum[n] = quad_sum(sum[n]) * fg[n];
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int src = 4 * (2 * t + r);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          qs[n][r] = __shfl_sync(SFFN_FULL_MASK, sum[n], src);
          gs[n][r] = NG == 1 ? 1.f : __shfl_sync(SFFN_FULL_MASK, fg[n], src);
        }
        f[r] = __shfl_sync(SFFN_FULL_MASK, f_g, src);
        pos[r] = __shfl_sync(SFFN_FULL_MASK, pos_g, src);
        lo[r] = __shfl_sync(SFFN_FULL_MASK, lo_g, src);
        m[r] = ninf;
        l[r] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) mid_sum[n][0] = mid_sum[n][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
    }
    if (!cur.empty(U) && !dead) {
      issue();
      const int st = slot_of(taken);
      if (!mbar_wait_bounded(&s_bar[warp][st], phase_of(taken))) {
        set_device_error(a.err, SFFN_ERR_TIMEOUT);
        dead = true;
      }
      ++taken;
      const uint8_t* sk = ring + st * T::kStage;
#pragma unroll 1
      for (int part = 0; part < U; part += SU) {
        const int base = cur.base(U) + part;
        if (base > cur.last) break;
        const uint8_t *pk = sk + part * (D / 2), *pv = pk + U * (D / 2), *pp = sk + U * D + part * 8 * NG;
        if (base + SU - 1 > cur.first || (a.window > 0 && base < cur.last - a.window + 1))
          unit(std::true_type(), pk, pv, pp, base);
        else
          unit(std::false_type(), pk, pv, pp, base);
      }
      __syncwarp();
    }
    const bool last = uu + 1 == u1;
    if (last || cur.u + 1 == cur.units) {
      const bool whole = finish(last);
      at_barrier = last && !whole;
      fresh = true;
    }
    cur.advance(a, U);
  }
  if (!at_barrier) {   // the barrier that the other warps have met in finish()
    drain();
    __syncthreads();
  }
  __syncthreads();

  // ---- partial results of the block: four warps per item, two rows each; lane e looks at entry e
  static_assert(2 * kAttWarps <= 32, "");
  const float* sm = reinterpret_cast<const float*>(smem);
  const bool used = lane < 2 * kAttWarps && s_entry[lane].where != 0;
  const unsigned used_mask = __ballot_sync(SFFN_FULL_MASK, used), below = used_mask & ((1u << lane) - 1u);
  const int of_item = used ? s_entry[lane].item_start : 0;
  const int of_prev = __shfl_sync(SFFN_FULL_MASK, of_item, below ? 31 - __clz(below) : lane);
  const bool head = used && (below == 0u || of_prev != of_item);   // the first entry of an item
  const unsigned heads = __ballot_sync(SFFN_FULL_MASK, head);
  const unsigned cut_heads = __ballot_sync(SFFN_FULL_MASK, head && (of_item < block_u0 || s_entry[lane].item_end > block_u1));
  const int cuts = __popc(cut_heads);   // at most two
  auto nth = [](unsigned mask, int n) {
    for (; n > 0; --n) mask &= mask - 1u;
    return __ffs(mask) - 1;
  };
  auto part_of = [&](int e) {   // a warp's last segment is in shared memory, an earlier one in its slot
    return e & 1 ? sm + (e >> 1) * T::kPart : a.warp_parts + (size_t)(blockIdx.x * kAttWarps + (e >> 1)) * T::kPart;
  };
  const int row0 = warp & 3;
  float me[2] = {ninf, ninf}, le[2] = {0.f, 0.f};
  if (used) {
    const float* p = part_of(lane) + kRows * kPitch + row0;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      me[z] = lane & 1 ? p[4 * z] : __ldcg(p + 4 * z);
      le[z] = lane & 1 ? p[kRows + 4 * z] : __ldcg(p + kRows + 4 * z);
    }
  }
#pragma unroll 1
  for (int j = warp >> 2; j < __popc(heads); j += kAttWarps / 4) {
    const Entry& it = s_entry[nth(heads, j)];
    const bool inside = it.item_start >= block_u0 && it.item_end <= block_u1;
    const bool member = used && of_item == it.item_start;
    float mt[2], lt[2], w[2], ot[2][CPL];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      mt[z] = warp_max(member ? me[z] : ninf);
      w[z] = !member ? 0.f : me[z] == mt[z] ? 1.f : ex2(me[z] - mt[z]);
      lt[z] = warp_sum(member ? le[z] * w[z] : 0.f);
#pragma unroll
      for (int c = 0; c < CPL; ++c) ot[z][c] = 0.f;
    }
    for (unsigned todo = __ballot_sync(SFFN_FULL_MASK, member); todo;) {
      constexpr int kAhead = 4;
      float x[kAhead][2][CPL];
      int e[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        e[i] = __ffs(todo) - 1;
        todo &= todo - 1u;
        if (e[i] < 0) continue;
#pragma unroll
        for (int z = 0; z < 2; ++z) part_row<CPL>(part_of(e[i]) + (row0 + 4 * z) * kPitch + lane * CPL, e[i] & 1, x[i][z]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (e[i] < 0) break;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float wi = __shfl_sync(SFFN_FULL_MASK, w[z], e[i]);
#pragma unroll
          for (int c = 0; c < CPL; ++c) ot[z][c] = fmaf(x[i][z][c], wi, ot[z][c]);
        }
      }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int row = row0 + 4 * z;
      if (inside) {
        write_row<D>(a, it.q0, it.n, it.kh, it.tile * kRows + row, lane, ot[z], mt[z], lt[z]);
        continue;
      }
      float* dst = a.block_parts + ((long long)blockIdx.x * 2 + (it.item_start < block_u0 ? 0 : 1)) * T::kPart;
#pragma unroll
      for (int c = 0; c < CPL; c += 2)
        *reinterpret_cast<float2*>(dst + row * kPitch + lane * CPL + c) = make_float2(ot[z][c], ot[z][c + 1]);
      if (lane == 0) {
        dst[kRows * kPitch + row] = mt[z];
        dst[kRows * kPitch + kRows + row] = lt[z];
      }
    }
  }
  if (cuts == 0) return;
  __threadfence();   // the block's parts before its tickets
  __syncthreads();
  if (threadIdx.x < cuts) {
    const Entry& it = s_entry[nth(cut_heads, threadIdx.x)];
    const int b0 = block_of(it.item_start, total, gridDim.x), b1 = block_of(it.item_end - 1, total, gridDim.x);
    // every block has a unit, or every block that has one has one only
    const int parts_of_item = total >= (int)gridDim.x ? b1 - b0 + 1 : it.item_end - it.item_start;
    const bool is_last = take_ticket(a.tickets + b0) == parts_of_item - 1;
    if (is_last) a.tickets[b0] = kTicketMark;   // for the next call
    s_last[threadIdx.x] = is_last;
    __threadfence();
  }
  __syncthreads();
  const Runs runs(total, gridDim.x);
#pragma unroll 1
  for (int pair = warp; pair < cuts * kRows; pair += kAttWarps) {
    const int row = pair % kRows, c = pair / kRows;
    if (!s_last[c]) continue;
    const Entry& it = s_entry[nth(cut_heads, c)];
    const int b0 = block_of(it.item_start, total, gridDim.x), count = block_of(it.item_end - 1, total, gridDim.x) - b0 + 1;
    auto part = [&](int k) { return a.block_parts + (size_t)((b0 + k) * 2 + (k == 0 ? 1 : 0)) * T::kPart; };
    float mt = ninf, lt = 0.f, ot[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) ot[e] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {   // lane k looks at the k-th part
      const int k = k0 + lane;
      const bool has = k < count && runs.start(b0 + k + 1) > runs.start(b0 + k);   // an empty block has no part
      const float me = has ? __ldcg(part(k) + kRows * kPitch + row) : ninf;
      const float le = has ? __ldcg(part(k) + kRows * kPitch + kRows + row) : 0.f;
      const float mn = fmaxf(warp_max(me), mt);
      const float back = mt == mn ? 1.f : ex2(mt - mn), w = !has ? 0.f : me == mn ? 1.f : ex2(me - mn);
      mt = mn;
      lt = lt * back + warp_sum(le * w);
#pragma unroll
      for (int e = 0; e < CPL; ++e) ot[e] *= back;
      const unsigned mask = __ballot_sync(SFFN_FULL_MASK, has);
      const int here = min(32, count - k0);
      constexpr int kAhead = 8;
      for (int i0 = 0; i0 < here; i0 += kAhead) {
        float x[kAhead][CPL];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)   // past the last part: that one again, not used
          part_row<CPL>(part(min(k0 + i0 + i, count - 1)) + row * kPitch + lane * CPL, false, x[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float wi = __shfl_sync(SFFN_FULL_MASK, w, (i0 + i) & 31);
          if (i0 + i < 32 && (mask >> (i0 + i) & 1)) {
#pragma unroll
            for (int e = 0; e < CPL; ++e) ot[e] = fmaf(x[i][e], wi, ot[e]);
          }
        }
      }
    }
    write_row<D>(a, it.q0, it.n, it.kh, it.tile * kRows + row, lane, ot, mt, lt);
  }
}


template <typename F>
auto by_shape(const sffn_kv& C, F&& f) {
  const int D = C.desc.head_dim, G = C.desc.group;
#define SFFN_SHAPE(d, g) \
  if (D == d && G == g) return f(std::integral_constant<int, d>(), std::integral_constant<int, g>());
  SFFN_SHAPE(64, 32)
  SFFN_SHAPE(64, 64)
  SFFN_SHAPE(128, 32)
  SFFN_SHAPE(128, 64)
  SFFN_SHAPE(128, 128)
  SFFN_SHAPE(256, 32)
  SFFN_SHAPE(256, 64)
#undef SFFN_SHAPE
  return f(std::integral_constant<int, 256>(), std::integral_constant<int, 128>());
}

constexpr size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct AttWs {
  size_t warp_parts, block_parts, total;
};
AttWs att_ws(const sffn_kv& C) {
  const size_t part = (size_t)(kRows * (C.desc.head_dim + 4) + 2 * kRows) * 4, blocks = C.num_sms;
  AttWs w;
  w.warp_parts = up256(blocks * sizeof(unsigned long long));
  w.block_parts = up256(w.warp_parts + blocks * kMaxWarps * part);
  w.total = up256(w.block_parts + blocks * 2 * part);
  return w;
}

}  // namespace

cudaError_t configure_attend_kernels(const sffn_kv& C) {
  return by_shape(C, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    const cudaError_t e = cudaFuncSetAttribute(k_attend<D, G, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Att<D, G, false>::kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(k_attend<D, G, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Att<D, G, true>::kSmem);
  });
}

size_t attend_ws_bytes(const sffn_kv& C, int, int, int) { return att_ws(C).total; }

cudaError_t launch_attend(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                          const sffn_rows& out, float* lse, float scale, int window, int dtype, void* ws,
                          cudaStream_t st) {
  if ((long long)window >= (long long)b.table_stride * C.desc.page_size) window = 0;   // no position is that far back
  const AttWs w = att_ws(C);
  uint8_t* p = static_cast<uint8_t*>(ws);
  const AttendArgs a{C.pages, C.page_bytes, C.head_bytes, C.desc.n_pages, C.desc.page_size,
                     C.desc.page_size == 16 ? 4 : C.desc.page_size == 32 ? 5 : 6, C.desc.n_kv_heads, C.err,
                     b, q, out, lse, n_q_heads, n_q_heads / C.desc.n_kv_heads, dtype, window, scale,
                     reinterpret_cast<unsigned long long*>(p), reinterpret_cast<float*>(p + w.warp_parts),
                     reinterpret_cast<float*>(p + w.block_parts)};
  const int blocks = C.num_sms;
  return by_shape(C, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    auto run = [&](auto* kern, int threads, int smem) {
      return launch_ex(kern, dim3(blocks), dim3(threads), smem, st, true, 1, a);
    };
    using E = Att<D, G, true>;
    using N = Att<D, G, false>;
    return dtype == SFFN_F32 ? run(k_attend<D, G, true>, E::kThreads, E::kSmem)
                             : run(k_attend<D, G, false>, N::kThreads, N::kSmem);
  });
}

}  // namespace sffn
