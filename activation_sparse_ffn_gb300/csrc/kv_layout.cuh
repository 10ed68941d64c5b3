// Where the codes of a cached page stand, and how the codes of one word become
// half-precision numbers.
//
// One page of one head is a contiguous block of P positions:
//   key codes [P][D/2 bytes] | value codes [P][D/2 bytes] | params [P/8][D/G][4][16 bytes]
// so that any run of positions that starts at a multiple of eight is three
// contiguous byte ranges. The order inside a row is the order in which a warp
// of the attention kernel needs it as matrix operands (lane = 4 g + t):
//
// Keys (contraction over channels): word t * D/32 + j of a row holds channels
// 32 j + 8 t + (0..7), so that lane t of the four lanes of a position takes
// one contiguous run of D/32 words, and the words j of all four lanes make up
// 32 consecutive channels: a quantization group is never split across a
// matrix step. Rows of 128 bytes (D = 256) swap the two 16-byte halves of a
// lane's run at odd positions, so that two neighbouring positions use
// different banks.
//
// Values (contraction over positions): chunk g (D/64 words) of a row holds the
// channels c with c % 8 = g, ascending; its place in the row is rotated by
// the position so that the four positions a warp reads together use different
// banks.
//
// Params: for eight positions, the (step, mid) pairs of the keys, then those of
// the values, each position by position in the order T(0) .. T(7) with its D/G
// groups beside each other; T(i) = i for i < 4 and i ^ 1 above is the order in
// which the eight rows (keys) or columns (values) of a matrix operand are
// assigned to positions. A group with a non-finite value has step = NaN and mid = 0: a
// weight can be cleared before it meets a step, but not before it meets a mid.
#pragma once

#include "common.cuh"

namespace sffn {

// Row or column of a matrix operand <-> position within eight (its own inverse).
__host__ __device__ constexpr int kv_pos_of_col(int c) { return c ^ (c >> 2); }

__host__ __device__ constexpr size_t kv_head_bytes(int P, int D, int G) {
  return (size_t)P * D + (size_t)P * (D / G) * 8;
}
__host__ __device__ constexpr int kv_value_off(int P, int D) { return P * (D / 2); }
__host__ __device__ constexpr int kv_param_off(int P, int D) { return P * D; }

// Byte offset, within a row of keys, of the word with channels 32 j + 8 t + (0..7).
template <int D>
__host__ __device__ constexpr int key_word_off(int pos, int t, int j) {
  if (D == 256) return t * 32 + (((j >> 2) ^ (pos & 1)) * 16) + (j & 3) * 4;
  return (t * (D / 32) + j) * 4;
}

// Place of chunk g in a row of values (chunks of D/64 words).
template <int D>
__host__ __device__ constexpr int value_chunk(int pos, int g) {
  if (D == 256) return g ^ (pos & 6);
  if (D == 128) return g ^ ((pos & 2) << 1);
  return g;
}
// Byte offset, within a row of values, of word w of chunk g: channels 64 w + 8 i + g, i = 0..7.
template <int D>
__host__ __device__ constexpr int value_word_off(int pos, int g, int w) {
  return (value_chunk<D>(pos, g) * (D / 64) + w) * 4;
}

// Byte offset, within the params, of the key (which = 0) or value (1) pair of a position and group.
__host__ __device__ constexpr int param_off(int pos, int grp, int n_groups, int which) {
  return (pos >> 3) * n_groups * 64 + which * n_groups * 32 + (kv_pos_of_col(pos & 7) * n_groups + grp) * 4;
}

// Key word: the codes of channel pairs e = 0..3 (channels 2e and 2e + 1 of the
// eight) stand at bits 4 e of the two 16-bit halves; the whole word is then
// rotated left by one bit. A code lies at bits 1-4 or 5-8 of a half (after a
// rotation by 8 for e = 2, 3), where the exponent of 1024 above it makes it a
// half-precision number, as for value words below.
// From the codes, that of channel e at bits key_field(e), and back:
__host__ __device__ constexpr int key_field(int e) { return 4 * (e >> 1) + 16 * (e & 1); }
__host__ __device__ __forceinline__ uint32_t key_word(uint32_t fields) { return fields << 1 | fields >> 31; }
__host__ __device__ __forceinline__ uint32_t key_fields(uint32_t w) { return w >> 1 | w << 31; }

// Value word: codes i = 0..3 (channels 64 w + 8 i + g) at bits 4 i of the low
// half, i = 4..7 likewise of the high half, each half then rotated left by one
// bit. A code lies at bits 1-4 or 5-8 of a half, or does so once its two bytes
// are swapped, which the byte selection that pairs two positions does on the
// way: with the exponent of 1024 put above it, it is the half-precision number
// 1024 + 2u (or 1024 + 32u), and one operation makes that 2u - 15 exactly.
// From the codes in order, four bits each, and back.
__host__ __device__ __forceinline__ uint32_t value_word(uint32_t nat) {
  return ((nat << 1) & 0xfffefffeu) | ((nat >> 15) & 0x00010001u);
}
__host__ __device__ __forceinline__ uint32_t value_codes(uint32_t w) {
  return ((w >> 1) & 0x7fff7fffu) | ((w << 15) & 0x80008000u);
}

// Eight lanes hold eight 4-bit codes each; afterwards code i of lane g is what
// code g of lane i was. Its own inverse: it turns eight channels of a lane into
// the codes of a value word and back.
__device__ __forceinline__ uint32_t transpose_codes(uint32_t w, int lane) {
#pragma unroll
  for (int s = 4; s; s >>= 1) {
    const uint32_t m = s == 4 ? 0x0000ffffu : s == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;   // codes whose index has bit s clear
    const uint32_t p = __shfl_xor_sync(SFFN_FULL_MASK, w, s);
    w = (lane & s) ? (w & ~m) | ((p & ~m) >> (4 * s)) : (w & m) | ((p & m) << (4 * s));
  }
  return w;
}

// ----------------------------------------------------------------- places

// The cached position of row i of a call, found by one warp together.
struct KvPlace {
  int seq;   // -1: the row belongs to no sequence
  int pos;   // may be negative: no place in the cache
};

__device__ __forceinline__ int kv_len_in_table(const sffn_kv_batch& b, int n, int P, uint32_t* err) {
  const long long most = (long long)b.table_stride * P;
  if (n < 0 || n > most) {
    set_device_error(err, SFFN_ERR_DEVICE);
    return n < 0 ? 0 : (int)most;
  }
  return n;
}
__device__ __forceinline__ int kv_len_of(const sffn_kv_batch& b, int s, int P, uint32_t* err) {
  return kv_len_in_table(b, ld_dep(b.kv_len + s), P, err);
}

// The rows of sequence s: q_start[s] .. q_start[s + 1] - 1. False if they do not ascend within the call's rows.
struct KvSpan {
  int from, to;
};
__device__ __forceinline__ bool kv_span(const sffn_kv_batch& b, int s, KvSpan& r) {
  r.from = ld_dep(b.q_start + s), r.to = ld_dep(b.q_start + s + 1);
  return r.from >= 0 && r.to >= r.from && r.to <= b.n_tokens;
}

// Every sequence is looked at, not only those up to the row's: where starts are out of order no row has a place. Up to
// kPlaceLanes sequences a warp does that on its own, lane s for sequence s; more, the block does for its rows together
// (kv_places), which reads them once a block (one token each of sequences with 8 + 2 x 8 heads of 128, append and
// read-back: 1024 of them 30 us, 118 with each warp on its own; 64 7.6 and 7.8; 32 6.6 either way).
constexpr int kPlaceLanes = 32;
__device__ __forceinline__ bool kv_many(const sffn_kv_batch& b) { return b.q_start && b.n_seq > kPlaceLanes; }

__device__ __forceinline__ KvPlace kv_place(const sffn_kv_batch& b, int i, int lane, int P, uint32_t* err) {
  KvPlace r{-1, -1};
  if (!b.q_start) {
    r.seq = i;
    r.pos = kv_len_of(b, i, P, err) - 1;
    return r;
  }
  KvSpan rows{0, 0};
  int n = 0;
  bool bad = false;
  if (lane < b.n_seq) {
    n = ld_dep(b.kv_len + lane);
    bad = !kv_span(b, lane, rows);
  }
  const unsigned here = __ballot_sync(SFFN_FULL_MASK, rows.from <= i && i < rows.to);
  if (__any_sync(SFFN_FULL_MASK, bad)) {
    set_device_error(err, SFFN_ERR_DEVICE);
  } else if (here) {
    r.seq = __ffs(here) - 1;
    const int left = __shfl_sync(SFFN_FULL_MASK, rows.to, r.seq) - i;   // rows from this one to the sequence's last
    r.pos = max(kv_len_in_table(b, __shfl_sync(SFFN_FULL_MASK, n, r.seq), P, err) - left, -1);
  }
  return r;
}

// The places of rows i0 .. i0 + N - 1, left at places by the threads of the block together.
template <int N>
__device__ __forceinline__ void kv_places(const sffn_kv_batch& b, int i0, int threads, int P, uint32_t* err, KvPlace* places) {
  if (threadIdx.x < N) places[threadIdx.x] = KvPlace{-1, -1};
  __syncthreads();
  bool bad = false;
#pragma unroll 4
  for (int s = threadIdx.x; s < b.n_seq; s += threads) {
    KvSpan rows;
    bad |= !kv_span(b, s, rows);
    for (int i = max(rows.from, i0); i < min(rows.to, i0 + N); ++i) places[i - i0] = KvPlace{s, rows.to - i};
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x < N) {   // what was found, or nothing
    KvPlace r = places[threadIdx.x];
    if (bad) {
      set_device_error(err, SFFN_ERR_DEVICE);
      r.seq = -1;
    } else if (r.seq >= 0) {
      r.pos = max(kv_len_of(b, r.seq, P, err) - r.pos, -1);
    }
    places[threadIdx.x] = r;
  }
  __syncthreads();
}

// Page of a position, or -1 (and the device error word) if its id is out of range.
__device__ __forceinline__ int kv_page(const sffn_kv_batch& b, int seq, int page_index, int n_pages, uint32_t* err) {
  const int id = ld_dep(b.table + (size_t)seq * b.table_stride + page_index);
  if (id < 0 || id >= n_pages) {
    set_device_error(err, SFFN_ERR_DEVICE);
    return -1;
  }
  return id;
}

}  // namespace sffn
