// The cache of sequences that go on as copies of others (beam search).
//
// Full pages change hands by their ids alone. Of the page that is not full, the
// filled positions are copied: per head three runs of bytes (keys, values,
// params of every eight positions). Sequences of a group may swap pages, so all
// that is written has been read before: a thread takes the same 16 bytes of the
// last page of every sequence of a group, through shared memory of its own.
//
// Measured: 64 x 8 sequences with pages of 64, half filled: 32 caches (570 MB read and as
// much written) 193 us, 5.9 TB/s; one cache 12 us, of which the bytes are 5 and the
// dependent reads (lengths, tables, pages) 3.5, as for one group of four.
#include <algorithm>
#include <climits>

#include "kv_layout.cuh"
#include "step.h"

namespace sffn {

namespace {

constexpr int kThreads = 256;
constexpr int kStage = 32 * 1024;     // shared memory of a block's copies
constexpr int kMaxBeams = 64;
constexpr int kTableBlock = 1024;     // columns of the page tables that a block reorders

struct ReorderArgs {
  uint8_t* pages[kMaxCaches];
  int32_t n_pages[kMaxCaches];
  sffn_kv_batch b;
  const int32_t* parents;
  int32_t* table_out;
  uint32_t* err;
  size_t page_bytes;
  int head_bytes, page_size, row_bytes, param_bytes;   // of a head: page, keys of a position, params of eight positions
  int heads, beams, out_stride;
  int chunk, copies;   // bytes of each page that a block copies, blocks of a group for that
  int cols, tables;    // columns of the page tables at a time, blocks of a group for them
};

// Byte of a head's page at byte i of what its first n positions fill, 16 bytes at a time (every run is a multiple of 16).
__device__ __forceinline__ int filled_byte(const ReorderArgs& a, int n, int i) {
  const int rows = n * a.row_bytes;
  if (i < rows) return i;
  if (i < 2 * rows) return a.page_size * a.row_bytes + i - rows;
  return 2 * a.page_size * a.row_bytes + i - 2 * rows;
}

__global__ void __launch_bounds__(kThreads) k_reorder(const ReorderArgs a) {
  extern __shared__ uint4 stage[];
  __shared__ int s_from[kMaxBeams], s_to[kMaxBeams], s_parent[kMaxBeams];
  pdl_launch_dependents();
  pdl_wait();
  const int blocks = a.copies + a.tables, group = blockIdx.x / blocks, part = blockIdx.x % blocks;
  const int first = group * a.beams, tid = threadIdx.x;
  const int n = ld_dep(a.b.kv_len + first);
  bool bad = n < 0 || n > (long long)a.b.table_stride * a.page_size;
  if (tid < a.beams) {
    const int p = ld_dep(a.parents + first + tid);
    bad |= p < 0 || p >= a.beams || ld_dep(a.b.kv_len + first + tid) != n;
    s_parent[tid] = p;
  }
  if (__syncthreads_or(bad)) {   // the group stays as it was
    if (tid == 0) set_device_error(a.err, SFFN_ERR_DEVICE);
    return;
  }
  const int full = n / a.page_size, tail = n % a.page_size;

  if (part >= a.copies) {
    // ids of full pages: a thread reads a column of every sequence before it writes it
    if (blockIdx.z) return;   // the caches share their tables
    int32_t* ids = reinterpret_cast<int32_t*>(stage);
    const int from = (part - a.copies) * kTableBlock, to = min(from + kTableBlock, full);
    for (int c = from + tid; tid < a.cols && c < to; c += a.cols) {
      for (int s = 0; s < a.beams; ++s) ids[s * a.cols + tid] = ld_dep(a.b.table + (size_t)(first + s) * a.b.table_stride + c);
      for (int s = 0; s < a.beams; ++s) a.table_out[(size_t)(first + s) * a.out_stride + c] = ids[s_parent[s] * a.cols + tid];
    }
    return;
  }
  if (tail == 0) return;
  const int layer = blockIdx.z, pages = a.n_pages[layer];
  if (tid < a.beams) {
    int from = ld_dep(a.b.table + (size_t)(first + tid) * a.b.table_stride + full);
    int to = ld_dep(a.table_out + (size_t)(first + tid) * a.out_stride + full);
    if (from < 0 || from >= pages) from = -1;
    if (to < 0 || to >= pages) to = -1;
    s_from[tid] = from, s_to[tid] = to;
  }
  __syncthreads();
  if (tid < a.beams && (s_from[s_parent[tid]] < 0 || s_to[tid] < 0)) set_device_error(a.err, SFFN_ERR_DEVICE);
  // a thread takes the same 16 bytes of every page, reads all that go on and writes them after that
  const int per_head = 2 * tail * a.row_bytes + (tail + 7) / 8 * a.param_bytes;   // filled bytes
  const int at = part * a.chunk + tid * 16, head = at / per_head;
  if (tid * 16 >= a.chunk || head >= a.heads) return;
  uint8_t* base = a.pages[layer] + (size_t)head * a.head_bytes + filled_byte(a, tail, at - head * per_head);
  uint4* own = stage + tid;
  const int step = a.chunk / 16;
  uint4 v[8];
  for (int s0 = 0; s0 < a.beams; s0 += 8) {
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < a.beams && s_from[s0 + s] >= 0)
        v[s] = __ldcg(reinterpret_cast<const uint4*>(base + s_from[s0 + s] * a.page_bytes));
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < a.beams && s_from[s0 + s] >= 0) own[(s0 + s) * step] = v[s];
  }
  for (int s = 0; s < a.beams; ++s) {
    const int from = s_from[s_parent[s]], to = s_to[s];
    if (from >= 0 && to >= 0 && to != from) *reinterpret_cast<uint4*>(base + to * a.page_bytes) = own[s_parent[s] * step];
  }
}

}  // namespace

cudaError_t launch_kv_reorder(const sffn_kv* const* kvs, int n_kv, const sffn_kv_batch& b, const int32_t* parents,
                              int beams, int32_t* table_out, int out_stride, cudaStream_t st) {
  const sffn_kv& C = *kvs[0];
  ReorderArgs a = {};
  for (int i = 0; i < n_kv; ++i) a.pages[i] = kvs[i]->pages, a.n_pages[i] = kvs[i]->desc.n_pages;
  a.b = b, a.parents = parents, a.table_out = table_out, a.err = C.err;
  a.page_bytes = C.page_bytes, a.head_bytes = (int)C.head_bytes, a.page_size = C.desc.page_size;
  a.row_bytes = C.desc.head_dim / 2, a.param_bytes = C.desc.head_dim / C.desc.group * 64;
  a.beams = beams, a.out_stride = out_stride;
  a.heads = C.desc.n_kv_heads;
  a.chunk = std::min(kStage / beams, kThreads * 16) / 16 * 16;
  a.copies = (int)((C.page_bytes + a.chunk - 1) / a.chunk);
  a.cols = std::min(kThreads, kStage / 4 / beams);
  a.tables = (b.table_stride + kTableBlock - 1) / kTableBlock;
  const int smem = std::max(a.chunk, a.cols * 4) * beams;
  const long long blocks = (long long)(a.copies + a.tables) * (b.n_seq / beams);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_ex(k_reorder, dim3((unsigned)blocks, 1, n_kv), dim3(kThreads), smem, st,
                   true, 1, a);
}

}  // namespace sffn
