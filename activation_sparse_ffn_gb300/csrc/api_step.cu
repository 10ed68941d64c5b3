// The extern "C" entry points of what stands around the halves of a decode
// step: argument checks, handles, and the launches.
#include <algorithm>
#include <cmath>
#include <new>

#include "step.h"

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

// Rows that are read or written element by element where they are not aligned further.
bool plain_rows_ok(const sffn_rows& r, int64_t n, int64_t width, int elem) {
  return r.ptr && aligned(r.ptr, elem) && (n <= 1 || r.row_stride >= width);
}

sffn_status check_ws(const void* ws, size_t have, size_t need) {
  if (!need) return SFFN_OK;
  if (!ws) return invalid("ws is NULL");
  if (!aligned(ws, 256)) return invalid("ws must be 256-byte aligned");
  if (have < need) return invalid("ws_bytes is smaller than the call's workspace");
  return SFFN_OK;
}

sffn_status check_codes(const sffn_rows& codes, const float* scales, int n_rows, int width) {
  if (!plain_rows_ok(codes, n_rows, width, 1)) return invalid("codes: need a pointer and a row stride of at least width");
  if (!scales || !aligned(scales, 4)) return invalid("codes need scales, 4-byte aligned");
  return SFFN_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- norm

sffn_status sffn_norm(sffn_rows x, sffn_rows residual, const float* weight, double eps, int32_t n_rows, int32_t width,
                      sffn_rows sum_out, sffn_rows y, sffn_rows codes, float* scales, int32_t dtype, int32_t y_dtype,
                      sffn_stream stream) {
  if (n_rows < 0 || n_rows > (1 << 30)) return invalid("n_rows must be in [0, 2^30]");
  if (width < 1 || width > 32768) return invalid("width must be in [1, 32768]");
  if (!std::isfinite(eps) || eps < 0) return invalid("eps must be finite and not negative");
  if (!is_dtype(dtype) || !is_dtype(y_dtype)) return invalid("dtype, y_dtype: not an sffn_dtype");
  if (n_rows == 0) return SFFN_OK;
  if (!y.ptr && !codes.ptr) return invalid("one of y and codes is required");
  const int e = elem_bytes(dtype);
  if (!plain_rows_ok(x, n_rows, width, e)) return invalid("x: needs an element-aligned pointer and a row stride of at least width");
  if ((residual.ptr && !plain_rows_ok(residual, n_rows, width, e)) || (sum_out.ptr && !plain_rows_ok(sum_out, n_rows, width, e)) ||
      (y.ptr && !plain_rows_ok(y, n_rows, width, elem_bytes(y_dtype))))
    return invalid("residual, sum_out, y: need an element-aligned pointer and a row stride of at least width");
  if (!aligned(weight, 4)) return invalid("weight must be 4-byte aligned");
  if (y.ptr && y.ptr == sum_out.ptr) return invalid("y and sum_out must not be the same rows");
  if (y.ptr && (y.ptr == x.ptr || y.ptr == residual.ptr) && (y_dtype == SFFN_F32) != (dtype == SFFN_F32))
    return invalid("y may be x or residual only with elements of the same size");
  if (codes.ptr) {
    const sffn_status rc = check_codes(codes, scales, n_rows, width);
    if (rc != SFFN_OK) return rc;
  }
  NormArgs a = {};
  a.x = x, a.residual = residual, a.sum = sum_out, a.y = y, a.codes = codes, a.weight = weight, a.scales = scales;
  a.eps = eps, a.rows = n_rows, a.width = width, a.dtype = dtype, a.y_dtype = y_dtype, a.norm = true;
  return launched(launch_norm(a, (cudaStream_t)stream), "sffn_norm");
}

sffn_status sffn_quantize(sffn_rows x, int32_t n_rows, int32_t width, sffn_rows codes, float* scales, int32_t dtype,
                          sffn_stream stream) {
  if (n_rows < 0 || n_rows > (1 << 30)) return invalid("n_rows must be in [0, 2^30]");
  if (width < 1 || width > 65536) return invalid("width must be in [1, 65536]");
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (n_rows == 0) return SFFN_OK;
  if (!plain_rows_ok(x, n_rows, width, elem_bytes(dtype)))
    return invalid("x: needs an element-aligned pointer and a row stride of at least width");
  const sffn_status rc = check_codes(codes, scales, n_rows, width);
  if (rc != SFFN_OK) return rc;
  NormArgs a = {};
  a.x = x, a.codes = codes, a.scales = scales, a.rows = n_rows, a.width = width, a.dtype = a.y_dtype = dtype;
  return launched(launch_norm(a, (cudaStream_t)stream), "sffn_quantize");
}

// ---------------------------------------------------------------- 8-bit linear layer

sffn_status sffn_linear8_validate(const sffn_linear8_desc* d) {
  if (!d) return invalid("desc is NULL");
  if (d->in_features < 16 || d->in_features > 65536 || d->in_features % 16)
    return invalid("in_features must be a positive multiple of 16, at most 65536");
  if (d->out_features < 1 || d->out_features > (1 << 20)) return invalid("out_features must be in [1, 1048576]");
  if (d->max_batch < 1 || d->max_batch > 65536) return invalid("max_batch must be in [1, 65536]");
  return SFFN_OK;
}

sffn_status sffn_linear8_create(const sffn_linear8_desc* d, sffn_linear8** out) {
  if (!out) return invalid("out is NULL");
  sffn_status rc = sffn_linear8_validate(d);
  if (rc != SFFN_OK) return rc;
  sffn_linear8* L = new (std::nothrow) sffn_linear8();
  if (!L) return invalid("host allocation failed");
  L->desc = *d;
  L->kp = (d->in_features + 127) / 128 * 128;   // steps of 128
  L->tiles = (d->out_features + 255) / 256 * 2;   // blocks work on them in pairs
  const size_t np = (size_t)L->tiles * 128;
  cudaError_t e = cudaGetDevice(&L->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device);
  if (e == cudaSuccess) e = cudaMalloc(&L->codes, np * L->kp);
  if (e == cudaSuccess) e = cudaMalloc(&L->scales, np * 4);
  if (e == cudaSuccess) e = cudaMalloc(&L->bias, np * 4);
  if (e == cudaSuccess) e = cudaMalloc(&L->err, 256);
  if (e == cudaSuccess) e = cudaMemset(L->err, 0, 256);
  if (e == cudaSuccess) e = configure_linear8_kernels(*L);
  if (e != cudaSuccess) {
    rc = cuda_fail(e, "sffn_linear8_create");
    sffn_linear8_destroy(L);
    return rc;
  }
  *out = L;
  return SFFN_OK;
}

sffn_status sffn_linear8_pack(sffn_linear8* L, const int8_t* codes, const float* scales, const float* bias,
                              sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  if (!codes || !scales) return invalid("codes and scales are required");
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(bias, 16))
    return invalid("codes, scales and bias must be 16-byte aligned");
  sffn_status rc = check_device(L->device);
  if (rc != SFFN_OK) return rc;
  return pack_linear8(*L, codes, scales, bias, (cudaStream_t)stream);
}

sffn_status sffn_linear8_get_desc(const sffn_linear8* L, sffn_linear8_desc* out) {
  if (!L || !out) return invalid("linear or out is NULL");
  *out = L->desc;
  return SFFN_OK;
}

size_t sffn_linear8_workspace_bytes(const sffn_linear8* L, int32_t B) {
  if (!L || B < 1 || B > L->desc.max_batch) return 0;
  return linear8_ws_bytes(*L, B);
}

sffn_status sffn_linear8_forward(const sffn_linear8* L, sffn_rows x, const float* x_scales, int32_t B,
                                 sffn_rows residual, sffn_rows y, int32_t dtype, void* ws, size_t ws_bytes,
                                 sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  if (!L->packed) return invalid("sffn_linear8_forward: the layer holds no weights (sffn_linear8_pack)");
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (B < 1 || B > L->desc.max_batch) return invalid("B must be in [1, max_batch]");
  if (!x.ptr || !aligned(x.ptr, 16) || (B > 1 && (x.row_stride < L->desc.in_features || x.row_stride % 16)))
    return invalid("x: needs a pointer and a row stride of at least in_features, both multiples of 16 bytes");
  if (!x_scales || !aligned(x_scales, 4)) return invalid("x_scales are required, 4-byte aligned");
  const int e = elem_bytes(dtype);
  if (!plain_rows_ok(y, B, L->desc.out_features, e) ||
      (residual.ptr && !plain_rows_ok(residual, B, L->desc.out_features, e)))
    return invalid("y, residual: need an element-aligned pointer and a row stride of at least out_features");
  sffn_status rc = check_ws(ws, ws_bytes, linear8_ws_bytes(*L, B));
  if (rc != SFFN_OK) return rc;
  rc = check_device(L->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_linear8(*L, x, x_scales, B, residual, y, dtype, ws, (cudaStream_t)stream),
                  "sffn_linear8_forward");
}

sffn_status sffn_linear8_check_error(const sffn_linear8* L, sffn_stream stream) {
  if (!L) return invalid("linear is NULL");
  return read_error_word(L->err, (cudaStream_t)stream);
}

void sffn_linear8_destroy(sffn_linear8* L) {
  if (!L) return;
  void* ps[] = {L->codes, L->scales, L->bias, L->err};
  for (void* p : ps)
    if (p) cudaFree(p);
  delete L;
}

// ---------------------------------------------------------------- continuations

sffn_status sffn_beam_validate(const sffn_beam_desc* d) {
  if (!d) return invalid("desc is NULL");
  if (d->vocab < 1 || d->vocab > (1 << 24)) return invalid("vocab must be in [1, 2^24]");
  if (d->beams < 1 || d->beams > 64) return invalid("beams must be in [1, 64]");
  if (d->n_out < 1 || d->n_out > 64) return invalid("n_out must be in [1, 64]");
  if (d->max_batch < 1 || (long long)d->max_batch * d->beams > 65535)
    return invalid("max_batch must be positive, and max_batch * beams at most 65535");
  return SFFN_OK;
}

sffn_status sffn_beam_create(const sffn_beam_desc* d, sffn_beam** out) {
  if (!out) return invalid("out is NULL");
  sffn_status rc = sffn_beam_validate(d);
  if (rc != SFFN_OK) return rc;
  sffn_beam* H = new (std::nothrow) sffn_beam();
  if (!H) return invalid("host allocation failed");
  H->desc = *d;
  cudaError_t e = cudaGetDevice(&H->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&H->num_sms, cudaDevAttrMultiProcessorCount, H->device);
  if (e == cudaSuccess) e = cudaMalloc(&H->err, 256);
  if (e == cudaSuccess) e = cudaMemset(H->err, 0, 256);
  if (e != cudaSuccess) {
    rc = cuda_fail(e, "sffn_beam_create");
    sffn_beam_destroy(H);
    return rc;
  }
  *out = H;
  return SFFN_OK;
}

sffn_status sffn_beam_get_desc(const sffn_beam* H, sffn_beam_desc* out) {
  if (!H || !out) return invalid("beam or out is NULL");
  *out = H->desc;
  return SFFN_OK;
}

size_t sffn_beam_workspace_bytes(const sffn_beam* H, int32_t batch) {
  if (!H || batch < 1 || batch > H->desc.max_batch) return 0;
  return beam_ws_bytes(*H, batch);
}

sffn_status sffn_beam_select(const sffn_beam* H, sffn_rows logits, const float* scores, const uint8_t* done,
                             int32_t end_token, int32_t batch, float* out_scores, int32_t* out_parents,
                             int32_t* out_tokens, int32_t dtype, void* ws, size_t ws_bytes, sffn_stream stream) {
  if (!H) return invalid("beam is NULL");
  if (!is_dtype(dtype)) return invalid("dtype is not an sffn_dtype");
  if (batch < 0 || batch > H->desc.max_batch) return invalid("batch must be in [0, max_batch]");
  if (done && (end_token < 0 || end_token >= H->desc.vocab)) return invalid("end_token must be in [0, vocab) with done");
  if (batch == 0) return SFFN_OK;
  if (!plain_rows_ok(logits, (int64_t)batch * H->desc.beams, H->desc.vocab, elem_bytes(dtype)))
    return invalid("logits: need an element-aligned pointer and a row stride of at least vocab");
  if (!scores || !out_scores || !out_parents || !out_tokens) return invalid("scores and the three outputs are required");
  if (!aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_parents, 4) || !aligned(out_tokens, 4))
    return invalid("scores and the outputs must be 4-byte aligned");
  if (out_scores == scores && H->desc.n_out != H->desc.beams)
    return invalid("out_scores may be scores only if n_out is beams");
  sffn_status rc = check_ws(ws, ws_bytes, beam_ws_bytes(*H, batch));
  if (rc != SFFN_OK) return rc;
  rc = check_device(H->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_beam(*H, logits, scores, done, end_token, batch, out_scores, out_parents, out_tokens, dtype, ws,
                              (cudaStream_t)stream), "sffn_beam_select");
}

sffn_status sffn_beam_check_error(const sffn_beam* H, sffn_stream stream) {
  if (!H) return invalid("beam is NULL");
  return read_error_word(H->err, (cudaStream_t)stream);
}

void sffn_beam_destroy(sffn_beam* H) {
  if (!H) return;
  if (H->err) cudaFree(H->err);
  delete H;
}

// ---------------------------------------------------------------- reordering

sffn_status sffn_kv_reorder(const sffn_kv* const* kvs, int32_t n_kv, const sffn_kv_batch* b, const int32_t* parents,
                            int32_t beams, int32_t* table_out, int32_t out_stride, sffn_stream stream) {
  if (!kvs || n_kv < 1 || n_kv > kMaxCaches) return invalid("kvs: 1 to 128 caches are wanted");
  for (int i = 0; i < n_kv; ++i) {
    if (!kvs[i]) return invalid("kvs: a cache is NULL");
    const sffn_kv_desc &d = kvs[i]->desc, &f = kvs[0]->desc;
    if (d.page_size != f.page_size || d.n_kv_heads != f.n_kv_heads || d.head_dim != f.head_dim || d.group != f.group ||
        kvs[i]->device != kvs[0]->device)
      return invalid("kvs: the caches of a call differ in n_pages at most");
    for (int j = 0; j < i; ++j)
      if (kvs[j] == kvs[i]) return invalid("kvs: a cache is given twice");
  }
  if (!b) return invalid("batch is NULL");
  if (beams < 1 || beams > 64) return invalid("beams must be in [1, 64]");
  if (b->n_seq < 0 || b->n_seq % beams) return invalid("n_seq must be a multiple of beams");
  if (b->n_seq == 0) return SFFN_OK;
  if (b->table_stride < 1 || (long long)b->table_stride * kvs[0]->desc.page_size > (1 << 30))
    return invalid("table_stride must be positive, and table_stride * page_size at most 2^30 positions");
  if (!b->table || !b->kv_len || !parents || !table_out || !aligned(b->table, 4) || !aligned(b->kv_len, 4) ||
      !aligned(parents, 4) || !aligned(table_out, 4))
    return invalid("table, kv_len, parents and table_out are required, 4-byte aligned");
  if (out_stride < b->table_stride) return invalid("out_stride must be at least table_stride");
  if (table_out == b->table && out_stride != b->table_stride) return invalid("a table in place keeps its stride");
  const char* t = reinterpret_cast<const char*>(b->table);
  const char* o = reinterpret_cast<const char*>(table_out);
  const long long tb = 4ll * ((long long)(b->n_seq - 1) * b->table_stride + b->table_stride);
  const long long ob = 4ll * ((long long)(b->n_seq - 1) * out_stride + b->table_stride);
  if (t != o && t < o + ob && o < t + tb) return invalid("table_out must be the table itself or not overlap it");
  sffn_status rc = check_device(kvs[0]->device);
  if (rc != SFFN_OK) return rc;
  return launched(launch_kv_reorder(kvs, n_kv, *b, parents, beams, table_out, out_stride, (cudaStream_t)stream),
                  "sffn_kv_reorder");
}

}  // extern "C"
