// The extern "C" entry points of the attention half of a decode step: argument
// checks, handles, and the launches.
#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "attn.h"
#include "kv_layout.cuh"

using namespace sffn;

namespace {

sffn_status invalid(const char* msg) {
  set_error(msg);
  return SFFN_ERR_INVALID_ARG;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_dtype(int d) { return d == SFFN_F32 || d == SFFN_F16 || d == SFFN_BF16; }
int elem_bytes(int d) { return d == SFFN_F32 ? 4 : 2; }

sffn_status check_device(int want) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != want) return invalid("the current CUDA device is not the one the handle was created on");
  return SFFN_OK;
}

sffn_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? SFFN_OK : cuda_fail(e, what); }

// Rows that are read or written in 16-byte pieces.
bool rows_ok(const sffn_rows& r, int64_t n, int heads, int width, int dtype) {
  const int64_t per16 = 16 / elem_bytes(dtype);
  if (!r.ptr || !aligned(r.ptr, 16)) return false;
  if (n > 1 && (r.row_stride < width || r.row_stride % per16)) return false;
  if (heads > 1 && (r.head_stride < width || r.head_stride % per16)) return false;
  return true;
}

// Rows that are read or written element by element.
bool plain_rows_ok(const sffn_rows& r, int64_t n, int width, int dtype) {
  return r.ptr && aligned(r.ptr, elem_bytes(dtype)) && (n <= 1 || r.row_stride >= width);
}

sffn_status check_ws(const void* ws, size_t have, size_t need) {
  if (!need) return SFFN_OK;
  if (!ws) return invalid("ws is NULL");
  if (!aligned(ws, 256)) return invalid("ws must be 256-byte aligned");
  if (have < need) return invalid("ws_bytes is smaller than the call's workspace");
  return SFFN_OK;
}

sffn_status check_batch(const sffn_kv_batch* b, int page_size) {
  if (!b) return invalid("batch is NULL");
  if (b->n_seq < 0 || b->n_tokens < 0) return invalid("n_seq and n_tokens must not be negative");
  if (b->n_tokens == 0) return SFFN_OK;
  if (b->n_seq < 1) return invalid("tokens without a sequence");
  if (b->table_stride < 1 || (long long)b->table_stride * page_size > (1 << 30))
    return invalid("table_stride must be positive, and table_stride * page_size at most 2^30 positions");
  if (!b->table || !b->kv_len || !aligned(b->table, 4) || !aligned(b->kv_len, 4) || !aligned(b->q_start, 4))
    return invalid("table and kv_len are required; table, kv_len and q_start must be 4-byte aligned");
  if (!b->q_start && b->n_tokens != b->n_seq) return invalid("q_start may be NULL only for one token per sequence");
  return SFFN_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- linear

sffn_status sffn_linear_validate(const sffn_linear_desc* d) {
  if (!d) return invalid("desc is NULL");
  if (d->group != 32 && d->group != 64 && d->group != 128) return invalid("group must be 32, 64 or 128");
  if (d->in_features < d->group || d->in_features > 65536 || d->in_features % d->group)
    return invalid("in_features must be a positive multiple of group, at most 65536");
  if (d->out_features < 1 || d->out_features > (1 << 20)) return invalid("out_features must be in [1, 1048576]");
  if (!is_dtype(d->scale_dtype)) return invalid("scale_dtype is not an sffn_dtype");
  if (d->max_batch < 1 || d->max_batch > 32) return invalid("max_batch must be in [1, 32]");
  return SFFN_OK;
}

sffn_status sffn_linear_create(const sffn_linear_desc* d, sffn_linear** out) {
  if (!out) return invalid("out is NULL");
  sffn_status rc = sffn_linear_validate(d);
  if (rc != SFFN_OK) return rc;
  sffn_linear* L = new (std::nothrow) sffn_linear();
  if (!L) return invalid("host allocation failed");
  L->desc = *d;
  L->kp = (d->in_features + 127) / 128 * 128;
  L->tiles = (d->out_features + 31) / 32 * 2;
  const size_t vals = (size_t)L->tiles * (L->kp / d->group) * 16 * elem_bytes(d->scale_dtype);
  cudaError_t e = cudaGetDevice(&L->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device);
  if (e == cudaSuccess) e = cudaMalloc(&L->codes, (size_t)L->tiles * 16 * L->kp / 2);
  if (e == cudaSuccess) e = cudaMalloc(&L->scales, vals);
  if (e == cudaSuccess && d->has_zero) e = cudaMalloc(&L->zeros, vals);
  if (e == cudaSuccess) e = cudaMalloc(&L->bias, (size_t)L->tiles * 16 * 4);
  if (e == cudaSuccess) e = cudaMalloc(&L->err, 256);
  if (e == cudaSuccess) e = cudaMemset(L->err, 0, 256);
  if (e == cudaSuccess) e = configure_linear_kernels(*L);
  if (e != cudaSuccess) {
    rc = cuda_fail(e, "sffn_linear_create");
    sffn_linear_destroy(L);
    return rc;
  }
  *out = L;
  return SFFN_OK;
}

sffn_status sffn_linear_pack(sffn_linear* L, const int8_t* codes, const void* scales, const void* zeros,
                             const float* bias, sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  if (!codes || !scales) return invalid("codes and scales are required");
  if ((zeros != nullptr) != (L->desc.has_zero != 0)) return invalid("zeros are required exactly if the layer has_zero");
  const void* ptrs[] = {codes, scales, zeros, bias};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return invalid("codes, scales, zeros and bias must be 16-byte aligned");
  sffn_status rc = check_device(L->device);
  if (rc != SFFN_OK) return rc;
  return pack_linear(*L, codes, scales, zeros, bias, (cudaStream_t)stream);
}

sffn_status sffn_linear_get_desc(const sffn_linear* L, sffn_linear_desc* out) {
  if (!L || !out) return invalid("linear or out is NULL");
  *out = L->desc;
  return SFFN_OK;
}

size_t sffn_linear_workspace_bytes(const sffn_linear* L, int32_t B) {
  if (!L || B < 1 || B > L->desc.max_batch) return 0;
  return linear_ws_bytes(*L, B);
}

sffn_status sffn_linear_forward(const sffn_linear* L, sffn_rows x, int32_t B, sffn_rows residual, sffn_rows y,
                                int32_t dtype, void* ws, size_t ws_bytes, sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  if (!L->packed) return invalid("sffn_linear_forward: the layer holds no weights (sffn_linear_pack)");
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (B < 1 || B > L->desc.max_batch) return invalid("B must be in [1, max_batch]");
  if (!rows_ok(x, B, 1, L->desc.in_features, dtype))
    return invalid("x: needs a pointer and a row stride of at least in_features, both multiples of 16 bytes");
  if (!plain_rows_ok(y, B, L->desc.out_features, dtype) ||
      (residual.ptr && !plain_rows_ok(residual, B, L->desc.out_features, dtype)))
    return invalid("y, residual: need an element-aligned pointer and a row stride of at least out_features");
  sffn_status rc = check_ws(ws, ws_bytes, linear_ws_bytes(*L, B));
  if (rc != SFFN_OK) return rc;
  rc = check_device(L->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_linear(*L, x, B, residual, y, dtype, ws, (cudaStream_t)stream), "sffn_linear_forward");
}

sffn_status sffn_linear_check_error(const sffn_linear* L, sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  return read_error_word(L->err, (cudaStream_t)stream);
}

void sffn_linear_destroy(sffn_linear* L) {
  if (!L) return;
  void* ps[] = {L->codes, L->scales, L->zeros, L->bias, L->err};
  for (void* p : ps)
    if (p) cudaFree(p);
  delete L;
}

// ---------------------------------------------------------------- cache

sffn_status sffn_kv_validate(const sffn_kv_desc* d) {
  if (!d) return invalid("desc is NULL");
  if (d->n_pages < 1) return invalid("n_pages must be positive");
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64) return invalid("page_size must be 16, 32 or 64");
  if (d->n_kv_heads < 1 || d->n_kv_heads > 1024) return invalid("n_kv_heads must be in [1, 1024]");
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return invalid("head_dim must be 64, 128 or 256");
  if ((d->group != 32 && d->group != 64 && d->group != 128) || d->group > d->head_dim)
    return invalid("group must be 32, 64 or 128, at most head_dim");
  return SFFN_OK;
}

size_t sffn_kv_bytes(const sffn_kv_desc* d) {
  if (sffn_kv_validate(d) != SFFN_OK) return 0;
  return kv_head_bytes(d->page_size, d->head_dim, d->group) * d->n_kv_heads * (size_t)d->n_pages;
}

sffn_status sffn_kv_create(const sffn_kv_desc* d, sffn_kv** out) {
  if (!out) return invalid("out is NULL");
  sffn_status rc = sffn_kv_validate(d);
  if (rc != SFFN_OK) return rc;
  sffn_kv* C = new (std::nothrow) sffn_kv();
  if (!C) return invalid("host allocation failed");
  C->desc = *d;
  C->head_bytes = kv_head_bytes(d->page_size, d->head_dim, d->group);
  C->page_bytes = C->head_bytes * d->n_kv_heads;
  cudaError_t e = cudaGetDevice(&C->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&C->num_sms, cudaDevAttrMultiProcessorCount, C->device);
  if (e == cudaSuccess) e = cudaMalloc(&C->pages, sffn_kv_bytes(d));
  if (e == cudaSuccess) e = cudaMalloc(&C->err, 256);
  if (e == cudaSuccess) e = cudaMemset(C->err, 0, 256);
  if (e == cudaSuccess) e = configure_attend_kernels(*C);
  if (e != cudaSuccess) {
    rc = cuda_fail(e, "sffn_kv_create");
    sffn_kv_destroy(C);
    return rc;
  }
  *out = C;
  return SFFN_OK;
}

sffn_status sffn_kv_get_desc(const sffn_kv* C, sffn_kv_desc* out) {
  if (!C || !out) return invalid("kv or out is NULL");
  *out = C->desc;
  return SFFN_OK;
}

sffn_status sffn_kv_check_error(const sffn_kv* C, sffn_stream stream) {
  if (!C) return invalid("kv is NULL");
  return read_error_word(C->err, (cudaStream_t)stream);
}

void sffn_kv_destroy(sffn_kv* C) {
  if (!C) return;
  if (C->pages) cudaFree(C->pages);
  if (C->err) cudaFree(C->err);
  delete C;
}

sffn_status sffn_kv_append(const sffn_kv* C, const sffn_kv_batch* b, sffn_rows q, int32_t n_q_heads, sffn_rows k,
                           sffn_rows v, sffn_rows q_out, const sffn_rope* rope, int32_t dtype, sffn_stream stream) {
  if (!C) return invalid("kv is NULL");
  sffn_status rc = check_batch(b, C->desc.page_size);
  if (rc != SFFN_OK) return rc;
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  const int D = C->desc.head_dim;
  if (rope) {
    if (!rope->table || !aligned(rope->table, 8)) return invalid("rope: table must be an 8-byte aligned device pointer");
    if (rope->length < 1 || rope->dim < 2 || rope->dim > D || rope->dim % 2)
      return invalid("rope: length must be positive and dim even, in [2, head_dim]");
    if (rope->style != 0 && rope->style != 1) return invalid("rope: style must be 0 or 1");
    if (!aligned(rope->positions, 4)) return invalid("rope: positions must be 4-byte aligned");
  }
  if (b->n_tokens == 0) return SFFN_OK;
  if (!rows_ok(k, b->n_tokens, C->desc.n_kv_heads, D, dtype) || !rows_ok(v, b->n_tokens, C->desc.n_kv_heads, D, dtype))
    return invalid("k, v: need a pointer and strides of at least head_dim, multiples of 16 bytes");
  if ((long long)b->n_tokens * (2 * C->desc.n_kv_heads + (q.ptr ? std::max(n_q_heads, 0) : 0)) > (1 << 30))
    return invalid("n_tokens * (n_q_heads + 2 * n_kv_heads) must be at most 2^30");
  if (q.ptr) {
    if (n_q_heads < 1 || n_q_heads > 65536) return invalid("n_q_heads must be in [1, 65536]");
    if (!rows_ok(q, b->n_tokens, n_q_heads, D, dtype) || !rows_ok(q_out, b->n_tokens, n_q_heads, D, dtype))
      return invalid("q, q_out: need a pointer and strides of at least head_dim, multiples of 16 bytes");
  }
  rc = check_device(C->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_kv_append(*C, *b, q, n_q_heads, k, v, q_out, rope ? *rope : sffn_rope{}, dtype,
                                   (cudaStream_t)stream), "sffn_kv_append");
}

sffn_status sffn_kv_gather(const sffn_kv* C, const sffn_kv_batch* b, sffn_rows k_out, sffn_rows v_out, int32_t dtype,
                           sffn_stream stream) {
  if (!C) return invalid("kv is NULL");
  sffn_status rc = check_batch(b, C->desc.page_size);
  if (rc != SFFN_OK) return rc;
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (b->n_tokens == 0) return SFFN_OK;
  const sffn_rows* rows[] = {&k_out, &v_out};
  for (const sffn_rows* r : rows)
    if (r->ptr && !rows_ok(*r, b->n_tokens, C->desc.n_kv_heads, C->desc.head_dim, dtype))
      return invalid("k_out, v_out: need strides of at least head_dim, multiples of 16 bytes");
  if ((long long)b->n_tokens * 2 * C->desc.n_kv_heads > (1 << 30))
    return invalid("n_tokens * 2 * n_kv_heads must be at most 2^30");
  if (!k_out.ptr && !v_out.ptr) return invalid("one of k_out and v_out is required");
  rc = check_device(C->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_kv_gather(*C, *b, k_out, v_out, dtype, (cudaStream_t)stream), "sffn_kv_gather");
}

// ---------------------------------------------------------------- attention

size_t sffn_attend_workspace_bytes(const sffn_kv* C, int32_t n_q_heads, int32_t n_seq, int32_t n_tokens) {
  if (!C || n_q_heads < 1 || n_q_heads % C->desc.n_kv_heads || n_seq < 0 || n_tokens < 0) return 0;
  return attend_ws_bytes(*C, n_q_heads, n_seq, n_tokens);
}

sffn_status sffn_attend(const sffn_kv* C, const sffn_kv_batch* b, sffn_rows q, int32_t n_q_heads, sffn_rows out,
                        float* lse, float scale, int32_t window, int32_t dtype, void* ws, size_t ws_bytes,
                        sffn_stream stream) {
  if (!C) return invalid("kv is NULL");
  sffn_status rc = check_batch(b, C->desc.page_size);
  if (rc != SFFN_OK) return rc;
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (n_q_heads < 1 || n_q_heads > 65536 || n_q_heads % C->desc.n_kv_heads)
    return invalid("n_q_heads must be a positive multiple of n_kv_heads, at most 65536");
  if ((long long)b->n_tokens * n_q_heads > (1 << 30)) return invalid("n_tokens * n_q_heads must be at most 2^30");
  if (!std::isfinite(scale)) return invalid("scale must be finite");
  if (window < 0) return invalid("window must not be negative");
  if (b->n_tokens == 0) return SFFN_OK;
  const int D = C->desc.head_dim;
  // the kernel's list: blocks of at least 32 positions of every tile of eight rows, counted in 32 bits
  const double tiles = ((double)b->n_tokens * (n_q_heads / C->desc.n_kv_heads) / 8 + b->n_seq) * C->desc.n_kv_heads;
  if (tiles * ((double)b->table_stride * C->desc.page_size / 32 + 2) > 2147483647.0)
    return invalid("n_tokens * n_q_heads * table_stride * page_size is too large for one call");
  if (!rows_ok(q, b->n_tokens, n_q_heads, D, dtype) || !rows_ok(out, b->n_tokens, n_q_heads, D, dtype))
    return invalid("q, out: need a pointer and strides of at least head_dim, multiples of 16 bytes");
  if (!aligned(lse, 4)) return invalid("lse must be 4-byte aligned");
  rc = check_ws(ws, ws_bytes, attend_ws_bytes(*C, n_q_heads, b->n_seq, b->n_tokens));
  if (rc != SFFN_OK) return rc;
  rc = check_device(C->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_attend(*C, *b, q, n_q_heads, out, lse, scale, window, dtype, ws, (cudaStream_t)stream),
                  "sffn_attend");
}

}  // extern "C"
