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
// groups beside each other; T(i) = i for i < 4 and i ^ 1 above is the order in which the eight
// rows (keys) or columns (values) of a matrix operand are assigned to
// positions. A group with a non-finite value has step = NaN and mid = 0: a
// weight can be cleared before it meets a step, but not before it meets a mid.
#pragma once

#include "common.cuh"

namespace sffn {

// Row or column of a matrix operand <-> position within eight (its own inverse).
__host__ __device__ constexpr int kv_pos_of_col(int c) { return c ^ (c >> 2); }

template <int D>
__host__ __device__ constexpr int kv_row_bytes() {
  return D / 2;
}

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
// rotation by 8 for e = 2, 3): as a half-precision number the masked bits are
// u * 2^-23 (or u * 2^-19), exactly.
__host__ __device__ __forceinline__ uint32_t key_word(const uint8_t* u) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) w |= (uint32_t)u[2 * e] << (4 * e) | (uint32_t)u[2 * e + 1] << (16 + 4 * e);
  return w << 1 | w >> 31;
}
__host__ __device__ __forceinline__ int key_code(uint32_t w, int i) {
  w = w >> 1 | w << 31;
  return (w >> ((i & 1) * 16 + (i >> 1) * 4)) & 15;
}

// Value word: codes i = 0..3 (channels 64 w + 8 i + g) at bits 4 i of the low
// half, i = 4..7 likewise of the high half, each half then rotated left by one
// bit. A code lies at bits 1-4 or 5-8 of a half, or does so once its two bytes
// are swapped, which the byte selection that pairs two positions does on the
// way: with the exponent of 1024 put above it, it is the half-precision number
// 1024 + 2u (or 1024 + 32u), and one operation makes that 2u - 15 exactly.
__host__ __device__ __forceinline__ uint32_t value_word(const uint8_t* u) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= (uint32_t)u[i] << (4 * i);
  return ((w << 1) & 0xfffefffeu) | ((w >> 15) & 0x00010001u);
}
__host__ __device__ __forceinline__ int value_code(uint32_t w, int i) {
  w = ((w >> 1) & 0x7fff7fffu) | ((w << 15) & 0x80008000u);
  return (w >> (4 * i)) & 15;
}

// One stored value, decoded on its own: (2u - 15) * step + mid, the product
// exact in fp32 (an 11-bit by a 4-bit number).
template <int D>
__device__ __forceinline__ float kv_value(const uint8_t* block, int P, int n_groups, int pos, int c, int which) {
  const uint8_t* row = block + (which ? kv_value_off(P, D) : 0) + pos * (D / 2);
  int u;
  if (which == 0)
    u = key_code(__ldcg(reinterpret_cast<const uint32_t*>(row + key_word_off<D>(pos, (c & 31) >> 3, c >> 5))), c & 7);
  else
    u = value_code(__ldcg(reinterpret_cast<const uint32_t*>(row + value_word_off<D>(pos, c & 7, c >> 6))), (c & 63) >> 3);
  const uint32_t pw = __ldcg(reinterpret_cast<const uint32_t*>(
      block + kv_param_off(P, D) + param_off(pos, c / (D / n_groups), n_groups, which)));
  const float2 pm = __half22float2(*reinterpret_cast<const __half2*>(&pw));
  return __fmaf_rn((float)(2 * u - 15), pm.x, pm.y);
}

// ----------------------------------------------------------------- places

// The cached position of row i of a call, found by one warp together.
struct KvPlace {
  int seq;   // -1: the row belongs to no sequence
  int pos;   // may be negative: no place in the cache
  int len;   // cached positions of the sequence
};

__device__ __forceinline__ int kv_len_of(const sffn_kv_batch& b, int s, int P, uint32_t* err) {
  const int n = ld_dep(b.kv_len + s);
  const long long most = (long long)b.table_stride * P;
  if (n < 0 || n > most) {
    set_device_error(err, SFFN_ERR_DEVICE);
    return n < 0 ? 0 : (int)most;
  }
  return n;
}

__device__ __forceinline__ KvPlace kv_place(const sffn_kv_batch& b, int i, int lane, int P, uint32_t* err) {
  KvPlace r{-1, -1, 0};
  if (!b.q_start) {
    r.seq = i;
    r.len = kv_len_of(b, i, P, err);
    r.pos = r.len - 1;
    return r;
  }
  for (int s0 = 0; s0 < b.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < b.n_seq;
    const int end = in ? ld_dep(b.q_start + s + 1) : 0x7fffffff;
    const int n = in ? ld_dep(b.kv_len + s) : 0;
    const unsigned past = __ballot_sync(SFFN_FULL_MASK, in && end > i);
    if (past) {
      const int src = __ffs(past) - 1;
      r.seq = s0 + src;
      r.len = __shfl_sync(SFFN_FULL_MASK, n, src);
      const int e = __shfl_sync(SFFN_FULL_MASK, end, src);
      const long long most = (long long)b.table_stride * P;
      if (r.len < 0 || r.len > most) {
        set_device_error(err, SFFN_ERR_DEVICE);
        r.len = r.len < 0 ? 0 : (int)most;
      }
      const long long pos = (long long)r.len - ((long long)e - i);
      r.pos = pos < 0 ? -1 : (int)pos;
      return r;
    }
  }
  return r;
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
