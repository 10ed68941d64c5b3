// Attention of decode tokens over the paged 4-bit cache.
//
// Mathematics. For query row r (a token and one of the gq query heads of a key
// head) and position j, in units of log2: S = q' . K_j with q' = q * scale *
// log2(e). A cached key is mid + step * c per group of channels with c = 2u - 15
// an odd integer, so S = sum over groups (step * (q'_g . c_g) + mid * sum(q'_g)):
// the tensor cores multiply q' with the bare codes, exact as halves, and step
// and mid are applied to eight positions at a time in fp32. In the same way
// sum_j p_j V_j = sum_j (p_j step_j) c_j + sum_j p_j mid_j, with the running
// maximum and sum of the softmax in fp32.
//
// Precision. q' and p * step are fp32 numbers carried by two halves each (22
// bits): the eight query rows of a tile stand in rows 0-7 of the 16-row operand
// and what the first halves leave in rows 8-15, so that the split costs no
// products (the tile holds at most eight rows). Powers of two bring the row's
// largest q' and the tile's largest step to 2^13 first, so that small numbers
// keep their bits. The sums of 64 positions leave the tensor core and are added
// to the running output in fp32: its own additions truncate, and over a long
// history that would show.
//
// Work split. The visible blocks of U positions (`units`) of every (sequence,
// key head, tile of eight rows) are numbered through, and each warp of the grid
// takes an equal run of that list, whatever the lengths are. A warp streams its
// units through a private ring in shared memory with one bulk copy per page for
// keys, values and params, so warps never wait for one another in the loop.
// Rows whose units lie within one warp are finished by it; the others are
// merged within the block at its end, and those cut by a block border by
// k_attend_join.
#include "attn.h"
#include "kv_layout.cuh"
#include "q4mma.cuh"
#include "rows_io.cuh"

namespace sffn {

namespace {

constexpr int kAttWarps = 8;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kRows = 8;   // query rows of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, int G>
struct Att {
  static constexpr int NG = D / G;
  static constexpr int U = D == 256 ? 32 : 64;             // positions of a unit
  static constexpr int kStage = U * (D + 8 * NG);          // bytes
  static constexpr int kStages = kStage * kAttWarps * 3 <= 212 * 1024 ? 3 : 2;
  static constexpr int kRing = kStage * kStages * kAttWarps;
  static constexpr int kPart = kRows * D + 2 * kRows;      // floats of a partial result: sums, maxima, totals
  static constexpr int kParts = kPart * 4 * kAttWarps;
  static constexpr int kSmem = kRing > kParts ? kRing : kParts;
};

// What a block tells k_attend_join about the item its first unit lies in.
struct Border {
  long long start, item_start, item_end;
  int q0, n, kh, tile;
  int pad[2];
};
static_assert(sizeof(Border) == 48, "");

struct AttendArgs {
  const uint8_t* pages;
  size_t page_bytes, head_bytes;
  int n_pages, P, hkv;
  uint32_t* err;
  sffn_kv_batch b;
  sffn_rows q, out;
  float* lse;
  int hq, gq, dtype, window;
  float scale;
  Border* borders;     // [blocks]
  float* warp_parts;   // [blocks * kAttWarps][kPart]
  float* block_parts;  // [blocks][2][kPart]
};

// A sequence's rows and length, made safe for indexing.
struct Seq {
  int q0, n, len;
};

__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int s) {
  Seq q;
  const long long most = (long long)a.b.table_stride * a.P;
  int len = ld_dep(a.b.kv_len + s);
  if (len < 0 || len > most) {
    set_device_error(a.err, SFFN_ERR_DEVICE);
    len = len < 0 ? 0 : (int)most;
  }
  q.len = len;
  if (a.b.q_start) {
    q.q0 = min(max(ld_dep(a.b.q_start + s), 0), a.b.n_tokens);
    q.n = min(max(ld_dep(a.b.q_start + s + 1), q.q0), a.b.n_tokens) - q.q0;
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
__device__ __forceinline__ long long total_of(const AttendArgs& a, const Seq& q, int U) {
  return q.n > 0 ? (long long)a.hkv * tiles_of(a, q) * units_of(a, q, U) : 0;
}

// A place in the list of units.
struct Cursor {
  int s, kh, tile, u;        // sequence, key head, tile, unit within the tile
  int tiles, units;          // of the sequence
  int q0, n, len;
  int base0, first, last;    // position of the tile's unit 0, of its first row, and of its last row

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
    units = units_of(a, q, U);
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
        } while (q.n == 0);
        set_seq(a, q, U);
      }
    }
    set_tile(a, U);
  }
  __device__ __forceinline__ int base(int U) const { return base0 + u * U; }
  __device__ __forceinline__ bool empty(int U) const { return base0 + u * U > last; }
};

template <int D, int G>
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

template <int D, int G>
__global__ void __launch_bounds__(kAttThreads, 1) k_attend(const AttendArgs a) {
  using T = Att<D, G>;
  constexpr int U = T::U, NG = T::NG, CPL = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_bar[kAttWarps][T::kStages];
  __shared__ long long s_scan[kAttWarps + 1];
  __shared__ int s_seq[kAttWarps];
  __shared__ long long s_off[kAttWarps];
  struct Entry {
    long long item_start, item_end;
    int q0, n, kh, tile, where;  // where: 0 none, 1 shared memory, 2 the warp's global slot
  };
  __shared__ Entry s_entry[2 * kAttWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x < kAttWarps * T::kStages) mbar_init(&s_bar[0][0] + threadIdx.x, 1);
  if (threadIdx.x < 2 * kAttWarps) s_entry[threadIdx.x].where = 0;
  fence_mbar_init();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the block's and the warp's run of units
  long long total = 0;
  for (int s = threadIdx.x; s < a.b.n_seq; s += kAttThreads) total += total_of(a, load_seq(a, s), U);
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(SFFN_FULL_MASK, total, o);
  if (lane == 0) s_scan[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) total += s_scan[w];
  const long long n_warps = (long long)gridDim.x * kAttWarps, gw = (long long)blockIdx.x * kAttWarps + warp;
  // start of warp w's run: floor(w * total / n_warps), without overflow
  const long long per = total / n_warps, rest = total % n_warps;
  auto start_of = [&](long long w) { return per * w + rest * w / n_warps; };
  const long long u0 = start_of(gw), u1 = start_of(gw + 1), block_u0 = start_of((long long)blockIdx.x * kAttWarps);
  const long long block_u1 = start_of((long long)(blockIdx.x + 1) * kAttWarps);
  // sequence of every warp's first unit
  long long before = 0;
  for (int s0 = 0; s0 < a.b.n_seq; s0 += kAttThreads) {
    const int s = s0 + threadIdx.x;
    const long long mine = s < a.b.n_seq ? total_of(a, load_seq(a, s), U) : 0;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(SFFN_FULL_MASK, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long chunk = 0, below = 0;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      if (w < warp) below += s_scan[w];
      chunk += s_scan[w];
    }
    const long long lo = before + below + upto - mine;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      const long long want = start_of((long long)blockIdx.x * kAttWarps + w);
      if (want >= lo && want < lo + mine) {
        s_seq[w] = s;
        s_off[w] = want - lo;
      }
    }
    before += chunk;
  }
  __syncthreads();

  const bool any = u0 < u1;
  Cursor cur{};
  if (any || (warp == 0 && block_u0 < total)) {
    const long long off = s_off[warp];
    cur.s = s_seq[warp];
    cur.set_seq(a, load_seq(a, cur.s), U);
    const long long item = off / cur.units;
    cur.u = (int)(off % cur.units);
    cur.kh = (int)(item / cur.tiles);
    cur.tile = (int)(item % cur.tiles);
    cur.set_tile(a, U);
    if (warp == 0 && lane == 0) {
      Border bd;
      bd.start = u0;
      bd.item_start = u0 - cur.u;
      bd.item_end = bd.item_start + cur.units;
      bd.q0 = cur.q0, bd.n = cur.n, bd.kh = cur.kh, bd.tile = cur.tile;
      bd.pad[0] = bd.pad[1] = 0;
      a.borders[blockIdx.x] = bd;
    }
  } else if (warp == 0 && lane == 0) {
    Border bd{};
    bd.start = total;
    a.borders[blockIdx.x] = bd;
  }

  // ---- copies: the warp's ring
  const int RP = min(a.P, U), parts = U / RP;   // positions of a unit that share a page, and how many such runs
  uint8_t* ring = smem + (size_t)warp * T::kStages * T::kStage;
  Cursor nxt = cur;
  long long nu = u0;       // next unit to copy
  int issued = 0, taken = 0;
  int page = 0;            // lane i: page of run i of unit nu
  auto fetch_page = [&]() {
    if (nu < u1 && !nxt.empty(U)) {
      const int base = nxt.base(U);
      if (lane < parts && base + lane * RP <= nxt.last)
        page = ld_dep(a.b.table + (size_t)nxt.s * a.b.table_stride + (base + lane * RP) / a.P);
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
    const int st = issued % T::kStages, base = nxt.base(U);
    uint8_t* dst = ring + st * T::kStage;
    const int runs = min(parts, (nxt.last - base) / RP + 1);
    if (lane == 0) mbar_arrive_expect_tx(&s_bar[warp][st], (uint32_t)(runs * RP * (D + 8 * NG)));
    __syncwarp();
    if (lane < runs) {
      if (page < 0 || page >= a.n_pages) {
        set_device_error(a.err, SFFN_ERR_DEVICE);
        page = 0;
      }
      const uint8_t* src = a.pages + (size_t)page * a.page_bytes + (size_t)nxt.kh * a.head_bytes;
      const int slot = base % a.P;  // zero unless a page holds several units
      const uint64_t pol = l2_policy_evict_first();
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
  if (any) {
    fetch_page();
    for (int i = 0; i < T::kStages - 1; ++i) issue();
  }

  const float ninf = __int_as_float(0xff800000);
  uint32_t q[D / 16][4];
  float qs[NG], mv[NG], o[D / 8][2];
  float f = 1.f, m = ninf, l = 0.f;
  int pos = 0, lo = 0;     // the row's position and the first it sees
  int pos_min = 0, lo_max = 0;   // over the tile's rows
  bool dead = false, fresh = true;
  long long item_start = u0 - cur.u;

  // after a wait that ran out: copies still under way must land before the ring is used for anything else
  auto drain = [&]() {
    if (dead)
      for (; taken < issued; ++taken) mbar_wait_bounded(&s_bar[warp][taken % T::kStages], (taken / T::kStages) & 1);
  };
  // the end of a segment, the warp's units of one item (lane: row g, channels 8x + 2t, + 1); true: the item lies within the warp
  auto finish = [&](bool last) {
    const float lt = quad_sum(l);
#pragma unroll
    for (int n = 0; n < NG; ++n) mv[n] = quad_sum(mv[n]);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
      o[x][0] += mv[x * 8 / G];
      o[x][1] += mv[x * 8 / G];
    }
    const long long item_end = item_start + cur.units;
    const float mt = m == ninf ? ninf : m * f;
    if (item_start >= u0 && item_end <= u1) {   // finish the rows here
      const int row = cur.tile * kRows + g;
      if (row < cur.n * a.gq) {
        const int i = cur.q0 + row / a.gq, h = cur.kh * a.gq + row % a.gq;
        const size_t at = (size_t)(i * a.out.row_stride + h * a.out.head_stride);
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const float v[2] = {o[x][0] * inv, o[x][1] * inv};
          st_run<2>(a.out.ptr, at + 8 * x + 2 * t, a.dtype, v);
        }
        if (a.lse && t == 0) a.lse[(size_t)i * a.hq + h] = lt == 0.f ? ninf : (mt + log2f(lt)) * kLn2;
      }
      return true;
    }
    // the last segment of the warp goes to shared memory (once every ring is idle), an earlier one to the warp's slot
    if (last) {
      drain();
      __syncthreads();
    }
    float* dst = last ? reinterpret_cast<float*>(smem) + warp * T::kPart : a.warp_parts + gw * T::kPart;
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      *reinterpret_cast<float2*>(dst + g * D + 8 * x + 2 * t) = make_float2(o[x][0], o[x][1]);
    if (t == 0) {
      dst[kRows * D + g] = mt;
      dst[kRows * D + kRows + g] = lt;
    }
    if (lane == 0) {
      Entry& e = s_entry[2 * warp + (last ? 1 : 0)];
      e.item_start = item_start, e.item_end = item_end;
      e.q0 = cur.q0, e.n = cur.n, e.kh = cur.kh, e.tile = cur.tile;
      e.where = last ? 1 : 2;
    }
    return false;
  };

  bool at_barrier = false;
  for (long long uu = u0; uu < u1; ++uu) {
    if (fresh) {   // first unit of the warp in this item: query rows
      fresh = false;
      item_start = uu - cur.u;
      const int rows = cur.n * a.gq, row = cur.tile * kRows + g, r = min(row, rows - 1);
      pos = cur.len - cur.n + r / a.gq;
      lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      pos_min = cur.first;
      lo_max = a.window > 0 ? max(0, cur.last - a.window + 1) : 0;
      const size_t at = (size_t)((cur.q0 + r / a.gq) * a.q.row_stride + (cur.kh * a.gq + r % a.gq) * a.q.head_stride);
      const float sc = row < rows ? a.scale * kLog2e : 0.f;
      float big = 0.f;
      // two passes over the row: its largest element, then the split
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        float x[8];
        ld_run<8>(a.q.ptr, at + 32 * j + 8 * t, a.dtype, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e] * sc));
      }
      float up;
      scale_to_half_range(quad_max(big), up, f);
#pragma unroll
      for (int n = 0; n < NG; ++n) qs[n] = mv[n] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        float x[8];
        ld_run<8>(a.q.ptr, at + 32 * j + 8 * t, a.dtype, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = row < rows ? x[e] * sc * up : 0.f;
          qs[j * 32 / G] += x[e];
        }
        split_f16(x[0], x[1], q[2 * j][0], q[2 * j][1]);
        split_f16(x[2], x[3], q[2 * j][2], q[2 * j][3]);
        split_f16(x[4], x[5], q[2 * j + 1][0], q[2 * j + 1][1]);
        split_f16(x[6], x[7], q[2 * j + 1][2], q[2 * j + 1][3]);
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) qs[n] = quad_sum(qs[n]);
#pragma unroll
      for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = 0.f;
      m = ninf;
      l = 0.f;
    }
    if (!cur.empty(U) && !dead) {
      issue();
      const int st = taken % T::kStages;
      if (!mbar_wait_bounded(&s_bar[warp][st], (taken / T::kStages) & 1)) {
        set_device_error(a.err, SFFN_ERR_TIMEOUT);
        dead = true;
      }
      ++taken;
      const uint8_t* sk = ring + st * T::kStage;
      const uint8_t* sv = sk + U * (D / 2);
      const uint8_t* sp = sk + U * D;
      const int base = cur.base(U);
      const bool masked = base < lo_max || base + U - 1 > pos_min;

      // ---- scores of U positions
      float s[U / 8][2];
      const int kt = kv_pos_of_col(g);   // the position, of eight, that this lane's key words belong to
#pragma unroll
      for (int i = 0; i < U / 8; ++i) {
        const uint8_t* row = sk + (8 * i + kt) * (D / 2);
        uint32_t w[D / 32];
        if (D == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(row + key_word_off<D>(kt, t, 0));
          w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; j += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + key_word_off<D>(kt, t, j));
            w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
          }
        }
        s[i][0] = s[i][1] = 0.f;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = n * G / 32; j < (n + 1) * G / 32; ++j) {
            uint32_t p[4];
            key_halves(w[j], p);
            mma_f16(c, q[2 * j], p[0], p[1]);
            mma_f16(c, q[2 * j + 1], p[2], p[3]);
          }
          const uint2 kp = *reinterpret_cast<const uint2*>(sp + ((i * NG + n) * 4 + t) * 16);
          const float2 pa = __half22float2(u32_h2(kp.x)), pb = __half22float2(u32_h2(kp.y));
          s[i][0] = fmaf(pa.x, c[0] + c[2], fmaf(pa.y, qs[n], s[i][0]));
          s[i][1] = fmaf(pb.x, c[1] + c[3], fmaf(pb.y, qs[n], s[i][1]));
        }
      }
      const int ta = kv_pos_of_col(2 * t), tb = kv_pos_of_col(2 * t + 1);  // positions of the lane's two columns
      float mu = ninf;
#pragma unroll
      for (int i = 0; i < U / 8; ++i) {
        if (masked) {
          const int ja = base + 8 * i + ta, jb = base + 8 * i + tb;
          if (ja > pos || ja < lo) s[i][0] = ninf;
          if (jb > pos || jb < lo) s[i][1] = ninf;
        }
        mu = fmaxf(mu, fmaxf(s[i][0], s[i][1]));
      }
      mu = fmaxf(m, quad_max(mu));
      if (__any_sync(SFFN_FULL_MASK, mu > m)) {
        const float back = mu == m ? 1.f : ex2((m - mu) * f);   // m = -inf: 0
        l *= back;
#pragma unroll
        for (int n = 0; n < NG; ++n) mv[n] *= back;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[x][0] *= back, o[x][1] *= back;
        m = mu;
      }
      const float mf = m == ninf ? 0.f : m * f;
#pragma unroll
      for (int i = 0; i < U / 8; ++i) {
        s[i][0] = ex2(fmaf(s[i][0], f, -mf));
        s[i][1] = ex2(fmaf(s[i][1], f, -mf));
        l += s[i][0] + s[i][1];
      }

      // ---- weights times steps, and the sum over positions
      auto value_params = [&](int i, int n, float2& va, float2& vb) {
        const uint2 vp = *reinterpret_cast<const uint2*>(sp + ((i * NG + n) * 4 + t) * 16 + 8);
        va = __half22float2(u32_h2(vp.x)), vb = __half22float2(u32_h2(vp.y));
        if (masked) {   // what is not seen may be anything, NaN too
          const int ja = base + 8 * i + ta, jb = base + 8 * i + tb;
          if (ja > pos || ja < lo) va = make_float2(0.f, 0.f);
          if (jb > pos || jb < lo) vb = make_float2(0.f, 0.f);
        }
      };
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < U / 8; ++i)
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          float2 va, vb;
          value_params(i, n, va, vb);
          top = fmaxf(top, fmaxf(va.x, vb.x));
          mv[n] = fmaf(s[i][0], va.y, fmaf(s[i][1], vb.y, mv[n]));
        }
      float up, down;
      scale_to_half_range(quad_max(top), up, down);
      uint32_t vw[U / 16][4][D / 64];   // the lane's words of four positions per 16
#pragma unroll
      for (int k = 0; k < U / 16; ++k)
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
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        constexpr int GW = G >= 64 ? 1 : 64 / G;   // groups that the word's 64 channels lie in
        float acc[8][4];
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
#pragma unroll
        for (int k = 0; k < U / 16; ++k) {
          uint32_t pa[GW][4];
#pragma unroll
          for (int n = 0; n < GW; ++n) {
            float2 va, vb;
            value_params(2 * k, w * 64 / G + n, va, vb);
            split_f16(s[2 * k][0] * (va.x * up), s[2 * k][1] * (vb.x * up), pa[n][0], pa[n][1]);
            value_params(2 * k + 1, w * 64 / G + n, va, vb);
            split_f16(s[2 * k + 1][0] * (va.x * up), s[2 * k + 1][1] * (vb.x * up), pa[n][2], pa[n][3]);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t x0 = __byte_perm(vw[k][0][w], vw[k][1][w], hh ? 0x7632 : 0x5410);
            const uint32_t x1 = __byte_perm(vw[k][2][w], vw[k][3][w], hh ? 0x7632 : 0x5410);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t y0 = e == 0 ? x0 << 4 : x0 >> (4 * e - 4), y1 = e == 0 ? x1 << 4 : x1 >> (4 * e - 4);
              mma_f16(acc[4 * hh + e], pa[(4 * hh + e) * 8 / G % GW], value_halves(y0), value_halves(y1));
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          o[8 * w + x][0] = fmaf(acc[x][0] + acc[x][2], down, o[8 * w + x][0]);
          o[8 * w + x][1] = fmaf(acc[x][1] + acc[x][3], down, o[8 * w + x][1]);
        }
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

  // ---- partial results of the block: warp w merges row w of each item
  const float* sm = reinterpret_cast<const float*>(smem);
  for (int e0 = 0; e0 < 2 * kAttWarps;) {
    if (s_entry[e0].where == 0) {
      ++e0;
      continue;
    }
    int e1 = e0 + 1;
    while (e1 < 2 * kAttWarps && (s_entry[e1].where == 0 || s_entry[e1].item_start == s_entry[e0].item_start)) ++e1;
    const Entry& it = s_entry[e0];
    float mt = ninf;
    for (int e = e0; e < e1; ++e) {
      if (s_entry[e].where == 0) continue;
      const float* p = s_entry[e].where == 1 ? sm + (e >> 1) * T::kPart
                                             : a.warp_parts + ((long long)blockIdx.x * kAttWarps + (e >> 1)) * T::kPart;
      mt = fmaxf(mt, s_entry[e].where == 1 ? p[kRows * D + warp] : __ldcg(p + kRows * D + warp));
    }
    float lt = 0.f, ot[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) ot[c] = 0.f;
    for (int e = e0; e < e1; ++e) {
      if (s_entry[e].where == 0) continue;
      const bool in_smem = s_entry[e].where == 1;
      const float* p = in_smem ? sm + (e >> 1) * T::kPart
                               : a.warp_parts + ((long long)blockIdx.x * kAttWarps + (e >> 1)) * T::kPart;
      const float me = in_smem ? p[kRows * D + warp] : __ldcg(p + kRows * D + warp);
      const float le = in_smem ? p[kRows * D + kRows + warp] : __ldcg(p + kRows * D + kRows + warp);
      const float w = me == mt ? 1.f : ex2(me - mt);
      lt = fmaf(le, w, lt);
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float* x = p + warp * D + lane * CPL + c;
        ot[c] = fmaf(in_smem ? *x : __ldcg(x), w, ot[c]);
      }
    }
    if (it.item_start >= block_u0 && it.item_end <= block_u1) {
      write_row<D, G>(a, it.q0, it.n, it.kh, it.tile * kRows + warp, lane, ot, mt, lt);
    } else {
      float* dst = a.block_parts + ((long long)blockIdx.x * 2 + (it.item_start <= block_u0 ? 0 : 1)) * T::kPart;
#pragma unroll
      for (int c = 0; c < CPL; ++c) dst[warp * D + lane * CPL + c] = ot[c];
      if (lane == 0) {
        dst[kRows * D + warp] = mt;
        dst[kRows * D + kRows + warp] = lt;
      }
    }
    e0 = e1;
  }
}

// Rows cut by a block border: block c handles the item that the first unit of
// attention block c + 1 lies in, if that item began before it and no earlier
// border lies in it; warp w takes row w.
template <int D, int G>
__global__ void __launch_bounds__(kAttThreads) k_attend_join(const AttendArgs a, int blocks) {
  using T = Att<D, G>;
  constexpr int CPL = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto start_at = [&](int k) { return __ldcg(&a.borders[k].start); };
  const long long start = start_at(c), item_start = __ldcg(&a.borders[c].item_start),
                  item_end = __ldcg(&a.borders[c].item_end), prev = start_at(c - 1);
  if (item_end == 0 || item_start >= start || item_start < prev) return;
  const float ninf = __int_as_float(0xff800000);
  int last = c;   // blocks c - 1 .. last hold a part
  while (last + 1 < blocks && start_at(last + 1) < item_end) ++last;
  auto part = [&](int k) { return a.block_parts + ((long long)k * 2 + (k == c - 1 && prev < item_start ? 1 : 0)) * T::kPart; };
  auto has = [&](int k) { return k == c - 1 || (k + 1 < blocks ? start_at(k + 1) : item_end) > start_at(k); };
  float mt = ninf;
  for (int k = c - 1; k <= last; ++k)
    if (has(k)) mt = fmaxf(mt, __ldcg(part(k) + kRows * D + warp));
  float lt = 0.f, ot[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) ot[e] = 0.f;
  for (int k = c - 1; k <= last; ++k) {
    if (!has(k)) continue;
    const float* p = part(k);
    const float me = __ldcg(p + kRows * D + warp), le = __ldcg(p + kRows * D + kRows + warp);
    const float w = me == mt ? 1.f : ex2(me - mt);
    lt = fmaf(le, w, lt);
#pragma unroll
    for (int e = 0; e < CPL; ++e) ot[e] = fmaf(__ldcg(p + warp * D + lane * CPL + e), w, ot[e]);
  }
  const int q0 = __ldcg(&a.borders[c].q0), n = __ldcg(&a.borders[c].n), kh = __ldcg(&a.borders[c].kh),
            tile = __ldcg(&a.borders[c].tile);
  write_row<D, G>(a, q0, n, kh, tile * kRows + warp, lane, ot, mt, lt);
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
  const size_t part = (size_t)(kRows * C.desc.head_dim + 2 * kRows) * 4, blocks = C.num_sms;
  AttWs w;
  w.warp_parts = up256(blocks * sizeof(Border));
  w.block_parts = up256(w.warp_parts + blocks * kAttWarps * part);
  w.total = up256(w.block_parts + blocks * 2 * part);
  return w;
}

}  // namespace

cudaError_t configure_attend_kernels(const sffn_kv& C) {
  return by_shape(C, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    return cudaFuncSetAttribute(k_attend<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, Att<D, G>::kSmem);
  });
}

size_t attend_ws_bytes(const sffn_kv& C, int, int, int) { return att_ws(C).total; }

cudaError_t launch_attend(const sffn_kv& C, const sffn_kv_batch& b, const sffn_rows& q, int n_q_heads,
                          const sffn_rows& out, float* lse, float scale, int window, int dtype, void* ws,
                          cudaStream_t st) {
  if ((long long)window >= (long long)b.table_stride * C.desc.page_size) window = 0;   // no position is that far back
  const AttWs w = att_ws(C);
  uint8_t* p = static_cast<uint8_t*>(ws);
  const AttendArgs a{C.pages, C.page_bytes, C.head_bytes, C.desc.n_pages, C.desc.page_size, C.desc.n_kv_heads, C.err,
                     b, q, out, lse, n_q_heads, n_q_heads / C.desc.n_kv_heads, dtype, window, scale,
                     reinterpret_cast<Border*>(p), reinterpret_cast<float*>(p + w.warp_parts),
                     reinterpret_cast<float*>(p + w.block_parts)};
  const int blocks = C.num_sms;
  return by_shape(C, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    cudaError_t e = launch_ex(k_attend<D, G>, dim3(blocks), dim3(kAttThreads), Att<D, G>::kSmem, st, true, 1, a);
    if (e != cudaSuccess || blocks < 2) return e;
    return launch_ex(k_attend_join<D, G>, dim3(blocks - 1), dim3(kAttThreads), 0, st, true, 1, a, blocks);
  });
}

}  // namespace sffn
