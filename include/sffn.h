/*
 * sffn.h -- C ABI of libsffn.so: predictor-gated, activation-sparse FFN decode
 * on one GB300 (sm_103a), with group momentum (TAM) bookkeeping.
 *
 * Sources of the operations (page title, section):
 *   PowerInfer (SOSP'24) summary page -- §5.1 per-layer MLP predictor
 *     scores = W2 . ReLU(W1 . x); "Paper vs code": a neuron is computed iff
 *     score >= threshold (default 0.0); §5.2 neuron table mapping packed slots
 *     to the original matrix order; §5.3-§5.4 neuron-aware operators that
 *     touch only active rows (up/gate) and columns (down), each thread block on
 *     a disjoint neuron set; activation note: ReLU, ReGLU, SiLU-family.
 *   KAIROX (OSDI'26) review page -- 核心方法 item 1/3: co-activation groups
 *     stored as contiguous regions, at most 1024 groups per layer; item 4:
 *     temporal activation momentum (TAM), candidates above
 *     tau = (1 - lambda) + eps, highest scores kept within the budget;
 *     item 5: Adaptive Neuron Balancer (lambda up on I/O stall, down on compute
 *     stall); item 6: fused XOR/AND set update.
 *
 * Conventions for every call:
 *   - Device pointers are plain CUDA device addresses on the CURRENT device;
 *     host pointers are marked "host". Sizes are element counts unless named
 *     *_bytes. The caller owns every per-call buffer; handles own the packed
 *     weights and the momentum state.
 *   - Index space is packed-slot order: slot s holds original neuron perm[s].
 *     Neuron bitmask: slot i is bit (i % 32) of word (i / 32). Group bitmask:
 *     group g is bit (g % 32) of word (g / 32). Group g = slots
 *     [g*G, (g+1)*G). A group is active iff any of its slots is active.
 *   - Hot calls (sffn_predict, sffn_forward, sffn_decode_step, tam_update,
 *     tam_adapt) allocate nothing, never synchronize, only enqueue on the given
 *     stream, and may be captured in a CUDA graph. They use programmatic
 *     dependent launch between their own kernels.
 *   - Errors are returned as sffn_status, never raised: argument checks are
 *     synchronous and happen before any device work; a failed launch returns
 *     SFFN_ERR_CUDA; conditions found on the device (a bounded wait that ran
 *     out, an out-of-range index) set the handle's device error word, read by
 *     sffn_layer_check_error / tam_check_error. sffn_last_error() gives a
 *     thread-local description of the last failure.
 */
#ifndef SFFN_H_
#define SFFN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* sffn_stream;   /* == cudaStream_t; NULL = legacy default stream */

typedef enum {
  SFFN_OK = 0,
  SFFN_ERR_INVALID_ARG = 1,   /* a pointer, size, alignment or enum is not allowed */
  SFFN_ERR_UNSUPPORTED = 2,   /* valid, but not implemented by this build */
  SFFN_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
  SFFN_ERR_TIMEOUT = 4,       /* a bounded device-side wait ran out */
  SFFN_ERR_OOM = 5,           /* device allocation failed (create/pack only) */
  SFFN_ERR_DEVICE = 6         /* the device found bad data (e.g. perm not a permutation) */
} sffn_status;

/* h = ReLU(u) | ReLU(g) * u | SiLU(g) * u | ReLU(u)^2 (squared ReLU, PowerInfer's
 * "Paper vs code" list), with u = up . x and g = gate . x; only ReGLU and
 * SwiGLU read gate rows. */
typedef enum { SFFN_ACT_RELU = 0, SFFN_ACT_REGLU = 1, SFFN_ACT_SWIGLU = 2, SFFN_ACT_RELU2 = 3 } sffn_act;
typedef enum { SFFN_F32 = 0, SFFN_F16 = 1, SFFN_BF16 = 2 } sffn_dtype;

/* Storage of the FFN rows (up, gate, down): in the layer's wdtype, or as 8-bit
 * or 4-bit codes with one fp32 scale per neuron (weight = code x scale; the
 * quantized models the pages run, e.g. PowerInfer's OPT-30B-Q4). SFFN_FFN_Q4
 * stores two signed 4-bit codes per byte, element 2i in the low half of byte
 * i. The predictor (W1, W2) always uses wdtype. */
typedef enum { SFFN_FFN_ROWS = 0, SFFN_FFN_Q8 = 1, SFFN_FFN_Q4 = 2 } sffn_ffn_format;

/* Shape of one FFN layer and its predictor.
 *   d: model dimension, multiple of 8, 8 <= d <= 16384.
 *   f: FFN neurons, multiple of group_size, f / group_size <= 1024 groups.
 *   h: predictor hidden size, multiple of 8, h * element size <= 2 KB
 *      (h <= 1024 for 16-bit weights, h <= 512 for fp32).
 *   group_size: 32 or 64 (KAIROX groups).
 *   act: sffn_act. ReLU and squared ReLU read up and down; ReGLU and SwiGLU also read gate.
 *   wdtype: storage type of every weight matrix (fp32 accumulation always).
 *   max_batch: largest B the layer will be called with, 1..32. */
typedef struct {
  int32_t d, f, h, group_size;
  int32_t act;
  int32_t wdtype;
  int32_t max_batch;
  int32_t ffn_format;   /* sffn_ffn_format; SFFN_FFN_Q8 needs wdtype fp16/bf16 and d % 16 == 0,
                           SFFN_FFN_Q4 fp16/bf16 and d % 32 == 0; batched calls (B > 1)
                           are not implemented for either */
} sffn_layer_desc;

/* One token's (or a batch's) active-set views, all device buffers owned by the
 * caller. Per-token arrays are laid out [B][...] with the stated row length:
 *   nmask  [B][f/32]      neuron bitmask
 *   gmask  [B][gw]        group bitmask, gw = ceil((f/G)/32)
 *   idx    [B][f]         ascending active slots; entries past count[b] are untouched
 *   count  [B]            number of active slots
 * Batch union (only read or written when B > 1; may be NULL when B == 1):
 *   unmask [f/32], ugmask [gw], uidx [f], ucount [1]. */
typedef struct {
  uint32_t* nmask;
  uint32_t* gmask;
  int32_t* idx;
  int32_t* count;
  uint32_t* unmask;
  uint32_t* ugmask;
  int32_t* uidx;
  int32_t* ucount;
} sffn_masks;

typedef struct sffn_layer sffn_layer;
typedef struct tam_state tam_state;

/* Device addresses of a layer's packed arrays (read-only view, for tests and
 * tools): W1 [h][d], b1 [h] (fp32, zeros if none), W2 [f][h] in slot order,
 * b2 [f] (fp32, slot order, zeros if none), up/gate/downT [f][d] in slot order
 * (gate NULL for ReLU and squared ReLU; downT[s][:] is column perm[s] of down), perm [f]. */
typedef struct {
  const void* W1;
  const float* b1;
  const void* W2;
  const float* b2;
  const void* up;
  const void* gate;
  const void* downT;
  const int32_t* perm;
  /* SFFN_FFN_Q8 / SFFN_FFN_Q4 only (NULL otherwise): per-slot scales of up, gate, downT rows */
  const float* up_scale;
  const float* gate_scale;
  const float* down_scale;
} sffn_packed_view;

/* ---------------------------------------------------------------- status */

const char* sffn_status_string(sffn_status s);
/* Thread-local text of the last failure in this thread ("" if none). */
const char* sffn_last_error(void);
/* Library version string, e.g. "sffn 0.1 sm_103a". */
const char* sffn_version(void);

/* ---------------------------------------------------------------- layers */

/* Host-only check of a layer description (no CUDA call). */
sffn_status sffn_layer_validate(const sffn_layer_desc* desc);

/* Create a layer on the current device: allocates the packed weight arrays
 * (uninitialised until sffn_layer_pack) and a device error word. *out is set
 * only on success. Errors: INVALID_ARG (desc), OOM, CUDA. */
sffn_status sffn_layer_create(const sffn_layer_desc* desc, sffn_layer** out);

/* Pack row-major weights into the grouped, neuron-major layout (setup, not a
 * hot call; synchronizes the stream before returning):
 *   W1 [h][d], W2 [f][h] (row n = original neuron n), up [f][d],
 *   gate [f][d] (NULL for ReLU and squared ReLU, required otherwise), down [d][f] (column n =
 *   original neuron n), all in the layer's wdtype; b1 [h], b2 [f] fp32 or NULL
 *   (zero); perm [f] int32 with perm[slot] = original neuron id, or NULL for
 *   the identity. Slot s of the packed arrays holds neuron perm[s]; down is
 *   stored transposed so each neuron's output column is one contiguous row.
 * Device pointers; 16-byte aligned. Errors: INVALID_ARG, DEVICE (perm is not
 * a permutation of 0..f-1), OOM (temporary buffer), CUDA. */
sffn_status sffn_layer_pack(sffn_layer* layer, const void* W1, const float* b1, const void* W2,
                            const float* b2, const void* up, const void* gate, const void* down,
                            const int32_t* perm, sffn_stream stream);

/* sffn_layer_pack for an SFFN_FFN_Q8 layer: W1, b1, W2, b2, perm as there;
 * up_q, gate_q [f][d] int8 codes with up_scale, gate_scale [f] fp32 (one per
 * neuron row), down_q [d][f] int8 codes with down_scale [f] fp32 (one per
 * neuron column), all in original neuron order; gate_q and gate_scale NULL
 * for ReLU and squared ReLU. Packed like sffn_layer_pack (slot order, down
 * transposed); the scales follow their rows. Device pointers, 16-byte
 * aligned. Errors: INVALID_ARG (also: the layer is not SFFN_FFN_Q8), DEVICE,
 * OOM, CUDA. The plain sffn_layer_pack rejects SFFN_FFN_Q8 layers. */
sffn_status sffn_layer_pack_q8(sffn_layer* layer, const void* W1, const float* b1, const void* W2,
                               const float* b2, const int8_t* up_q, const float* up_scale, const int8_t* gate_q,
                               const float* gate_scale, const int8_t* down_q, const float* down_scale,
                               const int32_t* perm, sffn_stream stream);

/* sffn_layer_pack_q8 for an SFFN_FFN_Q4 layer: the same arguments, with every
 * code in [-8, 7] (one int8 per code; the library packs two per byte). A code
 * outside that range fails with DEVICE and leaves the layer unpacked.
 * Errors: INVALID_ARG (also: the layer is not SFFN_FFN_Q4), DEVICE, OOM, CUDA. */
sffn_status sffn_layer_pack_q4(sffn_layer* layer, const void* W1, const float* b1, const void* W2,
                               const float* b2, const int8_t* up_q, const float* up_scale, const int8_t* gate_q,
                               const float* gate_scale, const int8_t* down_q, const float* down_scale,
                               const int32_t* perm, sffn_stream stream);

sffn_status sffn_layer_get_desc(const sffn_layer* layer, sffn_layer_desc* out /* host */);
sffn_status sffn_layer_packed(const sffn_layer* layer, sffn_packed_view* out /* host */);

/* Bytes of device workspace that the hot calls need for batch size B
 * (0 if the arguments are invalid). The workspace is caller-owned scratch,
 * 256-byte aligned, reused across calls; its contents need no initialisation. */
size_t sffn_workspace_bytes(const sffn_layer* layer, int32_t B);

/* Synchronize the stream, then read and clear the layer's device error word:
 * OK, TIMEOUT (a bounded wait ran out) or DEVICE (bad data seen on device). */
sffn_status sffn_layer_check_error(const sffn_layer* layer, sffn_stream stream);

void sffn_layer_destroy(sffn_layer* layer);

/* Optional per-kernel timing hooks. Kernel slots for B = 1: 0 predictor
 * hidden layer, 1 predictor scores + threshold, 2 sparse FFN (gather of active
 * up/gate rows, activation, and the active downT rows into per-block partial
 * sums), 3 reduction of the partial sums into y (and x + y). For B > 1 the
 * slots time the four tensor-core products: 0 hidden, 1 scores, 2 up/gate
 * over the union rows, 3 down over the union rows. When set, every later hot call on this layer records
 * begin[k] on its stream right before launching kernel k and end[k] right
 * after it (NULL entries are skipped). The handles are cudaEvent_t values owned
 * by the caller, which must keep them alive while tracing is on. Recording
 * between two kernels removes their launch overlap, so traced timings bound
 * each kernel alone. Pass NULL to turn tracing off. Host only; not
 * thread-safe against hot calls on the same layer from other threads. */
typedef struct {
  void* begin[4];
  void* end[4];
} sffn_trace;

sffn_status sffn_layer_set_trace(sffn_layer* layer, const sffn_trace* trace /* host, or NULL */);

/* Optional L2 hint for a layer stack at B = 1. `next` names the layer whose
 * hot call follows this layer's on the same stream (in a stack: layer l + 1,
 * and for the last layer layer 0 of the next token), or NULL to turn the hint
 * off. Each block of this layer's sparse-FFN kernel then asks L2 to fetch its
 * share of next's predictor hidden-layer weights (W1, PowerInfer §5.1) once
 * it has issued the copies of its own rows, so that those bytes move while
 * other blocks finish and while the reduction runs; the next predictor then
 * reads them from L2. Results are unchanged (the
 * prefetch only warms the cache). The library does not own `next`: the caller
 * keeps it alive while the hint is set, or unsets it first. `next` must live
 * on the same device; it may equal `layer`. Host only.
 * Errors: INVALID_ARG (layer NULL, or next on another device). */
sffn_status sffn_layer_set_next(sffn_layer* layer, const sffn_layer* next /* or NULL */);

/* Optional hot-group residency in L2 (the single-GPU analogue of PowerInfer's
 * hot/cold neuron split, §3-§4, with L2 in place of the GPU and HBM in place of
 * the CPU; KAIROX's momentum picks the hot groups, 核心方法 item 4). resident is
 * a device bitset of the layer's groups, [ceil(n_groups / 32)] uint32 (for
 * instance one layer's row of tam_outputs.resident from tam_update with a
 * capacity sized to the L2 share it may hold), or NULL to turn the hint off.
 * The B = 1 sparse-FFN kernel reads it at every launch (so tam_update may
 * rewrite it on the same stream between calls) and reads the up/gate/downT
 * rows of predicted-active neurons in those groups with the L2 evict-last
 * priority, all other rows with evict-first, so that hot rows tend to be
 * served from L2 on the next tokens. Results are unchanged (cache priorities
 * only). The caller keeps the buffer alive while it is set. Host only.
 * Errors: INVALID_ARG (layer NULL, resident not 4-byte aligned). */
sffn_status sffn_layer_set_l2_resident(sffn_layer* layer, const uint32_t* resident /* device, or NULL */);

/* Optional actual-activation zero-skip (PowerInfer §5.4: a neuron-aware
 * operator checks whether a neuron is active and computes only the active
 * ones, here applied to the activation itself). With enable != 0, the B = 1
 * sparse FFN (sffn_forward, sffn_decode_step) reads the transposed-down row of
 * a predicted-active neuron only if its activation h is non-zero (ReLU or a
 * ReGLU gate that clamps to 0 gives h = 0, and h * downT_i adds nothing to y).
 * The up (and gate) rows of every predicted-active neuron are still read: h is
 * known only after them. y is unchanged up to the sign of a zero sum;
 * idx / count / gmask still describe the predicted mask. rows_read: optional
 * device int32, or NULL; each B = 1 FFN call then writes the number of
 * transposed-down rows it read (stream-ordered with the call). Off by default;
 * calls with B > 1 ignore it. The caller keeps rows_read alive while it is
 * set. Host only. Errors: INVALID_ARG (layer NULL, rows_read not 4-byte
 * aligned). */
sffn_status sffn_layer_set_zero_skip(sffn_layer* layer, int32_t enable, int32_t* rows_read /* device, or NULL */);

/* Optional B = 1 grid sizes, for running one layer's predictor and another
 * layer's sparse FFN at the same time on two streams (one-layer-ahead
 * prediction: KAIROX observes that adjacent layers see near-identical inputs,
 * so layer l + 1's active set can be predicted from layer l's input while
 * layer l's FFN runs). The sparse-FFN kernel holds one large-shared-memory
 * block per SM and the predictor-scores kernel likewise, so they can only
 * overlap on disjoint SMs: ffn_blocks limits the FFN kernel and score_blocks
 * the scores kernel of this layer to that many blocks (0 = one per SM, the
 * default). The predictor's hidden-layer kernel needs no limit (it shares
 * SMs). Masks do not depend on the grid; y may differ by fp32 rounding,
 * because the FFN's per-block partial sums change with the block count.
 * Host only; the workspace size (sffn_workspace_bytes) never grows.
 * Errors: INVALID_ARG (layer NULL, a count outside [0, number of SMs], or
 * too few FFN blocks for the layer's shared-memory ring). */
sffn_status sffn_layer_set_grid(sffn_layer* layer, int32_t ffn_blocks, int32_t score_blocks);

/* Which arithmetic serves batched calls (B > 1) on this layer. The batch
 * reads each row of the union of its tokens' active sets once (KAIROX 问题与
 * 动机: a batch activates the union of its tokens' neurons; PowerInfer §3.2
 * on batches below 32):
 *   SFFN_BATCH_TENSOR      every product on the tensor cores (tcgen05.mma over
 *                          the union rows, activations as 16-bit hi/lo parts);
 *   SFFN_BATCH_CUDA_CORES  for 2 <= B <= 4: fp32 FFMA on the CUDA cores, the
 *                          B = 1 kernels' structure with every token's x in
 *                          registers (16-bit SFFN_FFN_ROWS weights, d <= 8192;
 *                          otherwise UNSUPPORTED); B > 4 takes the tensor cores;
 *   SFFN_BATCH_AUTO        the default: the CUDA cores for B = 2 where they
 *                          apply, the tensor cores otherwise (measured on
 *                          GB300: the CUDA-core arm is faster at B = 2 and
 *                          slower from B = 3 on).
 * Results agree within the parity tolerances either way; both arms write the
 * same views. Host only. Errors: INVALID_ARG (layer NULL, unknown path). */
typedef enum { SFFN_BATCH_AUTO = 0, SFFN_BATCH_TENSOR = 1, SFFN_BATCH_CUDA_CORES = 2 } sffn_batch_path;
sffn_status sffn_layer_set_batch_path(sffn_layer* layer, int32_t path);

/* The arm that serves a batched call of B tokens on this layer under its
 * current setting: SFFN_BATCH_TENSOR or SFFN_BATCH_CUDA_CORES, or -1 when no
 * arm does (B outside [2, max_batch], or a layer the batched paths do not
 * take: such a call returns UNSUPPORTED). Host only. */
int32_t sffn_layer_batch_arm(const sffn_layer* layer, int32_t B);

/* ---------------------------------------------------------------- hot calls */

/* Predictor (PowerInfer §5.1 and the threshold note): for each token b,
 *   hid = ReLU(W1 . x_b + b1), s = W2 . hid + b2, slot i active iff s_i >= thres
 * (NaN is inactive), written as masks->nmask/gmask/idx/count for row b; for
 * B > 1 also the union views. x: [B][d] fp32 device, 16-byte aligned.
 * ws: workspace of at least sffn_workspace_bytes(layer, B).
 * Errors: INVALID_ARG, UNSUPPORTED (B beyond what this build implements), CUDA. */
sffn_status sffn_predict(const sffn_layer* layer, const float* x, int32_t B, float thres,
                         const sffn_masks* masks, void* ws, size_t ws_bytes, sffn_stream stream);

/* Sparse FFN over the active set given by masks->nmask (rows [B][f/32]; any
 * caller-made mask is allowed): for each token b,
 *   y_b = sum_{slot i active for b} act(gate_i . x_b, up_i . x_b) * downT_i
 * with act = ReLU(u) | ReLU(g)*u | SiLU(g)*u, fp32 accumulation, fixed
 * summation order (run-to-run bit-identical). Only active rows are read
 * (PowerInfer §5.4). y: [B][d] fp32. x_out: NULL, or [B][d] fp32 that receives
 * x + y (the residual stream of a layer stack). Other mask fields are ignored.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
sffn_status sffn_forward(const sffn_layer* layer, const float* x, int32_t B, const sffn_masks* masks,
                         float* y, float* x_out, void* ws, size_t ws_bytes, sffn_stream stream);

/* sffn_predict followed by sffn_forward on the predicted masks, as one
 * pipelined sequence of kernels. All mask views are written. */
sffn_status sffn_decode_step(const sffn_layer* layer, const float* x, int32_t B, float thres,
                             const sffn_masks* masks, float* y, float* x_out, void* ws,
                             size_t ws_bytes, sffn_stream stream);

/* sffn_decode_step for callers that cannot allocate device memory: a decode
 * loop that must never stall on an allocation (one can synchronize the whole
 * GPU), a runtime that reaches this library only through its C ABI and has no
 * CUDA allocator, or a process whose memory pool refuses new allocations once
 * serving starts. Same arguments and results as sffn_decode_step at B = 1,
 * minus the workspace: scratch comes from one 16 MiB device array inside the
 * library, which every GPU that loads the library holds until the process
 * exits. B > 1 returns UNSUPPORTED (the batched path's scratch is not held in
 * the array). The array is enough for any valid layer at B = 1 on a GPU with
 * up to about 240 SMs (the per-block partial sums take SMs x d x 4 bytes, at
 * most 10 MB on a 152-SM GB300, so no valid layer reaches the limit there); a
 * layer needing more returns INVALID_ARG. The call allocates nothing and
 * records no sffn_layer_set_trace events. Its first call on each device looks
 * up the array's device address (cudaGetSymbolAddress), so make that first
 * call before any stream capture. All calls on a device share the array:
 * calls that can overlap on the GPU race on it and must be ordered by the
 * caller; nothing in it needs clearing between calls. The pages describe no
 * counterpart of this call; it exists for callers of this library. */
sffn_status sffn_decode_step_static_ws(const sffn_layer* layer, const float* x, int32_t B, float thres,
                                       const sffn_masks* masks, float* y, float* x_out, sffn_stream stream);

/* ---------------------------------------------------------------- whole stack */

/* A stack of layers decoded one token at a time by ONE kernel launch: for
 * every layer in order, the predictor (PowerInfer §5.1), the threshold, the
 * sparse FFN over the predicted rows (§5.3-§5.4) and the residual
 * x_{l+1} = x_l + y_l -- the computation of sffn_decode_step at B = 1 with
 * x_out chaining the layers, with the same summation orders (hid, masks,
 * index lists, y and x_{l+1} are bit-identical to that chain on the same
 * inputs). One thread block per SM runs the whole token; grid-wide barriers
 * separate the phases, and each block streams the next phases' predictor
 * weights while the barriers and the other phases run. The layers must
 * share d, f, h, group_size, act and storage, use 16-bit weights in
 * SFFN_FFN_ROWS form, and keep at most 32 KB per neuron of up/gate rows
 * (d <= 8192 for ReGLU/SwiGLU, d <= 16384 for ReLU); other shapes return
 * UNSUPPORTED (use the per-layer calls). The stack keeps the layers' packed
 * arrays' addresses, not the layers: they must outlive it (re-packing a layer
 * in place is fine). Per-layer options (sffn_layer_set_next, _set_grid,
 * _set_l2_resident, _set_zero_skip) do not apply to the stack kernel.
 * Errors: INVALID_ARG (NULL, n_layers outside [1, 4096], layers that differ
 * or live on other devices), UNSUPPORTED, OOM, CUDA. */
typedef struct sffn_stack sffn_stack;
sffn_status sffn_stack_create(const sffn_layer* const* layers /* host array [n_layers] */, int32_t n_layers,
                              sffn_stack** out);

/* Bytes of caller workspace sffn_stack_decode needs (0 if stack is NULL):
 * the hidden vector and one partial sum of y per SM. */
size_t sffn_stack_workspace_bytes(const sffn_stack* stack);

/* One decode token through every layer (device pointers, fp32):
 *   x0  [d]            input of layer 0 (16-byte aligned); it may be one of
 *                      xs's rows, e.g. the previous token's output
 *                      xs + (n_layers-1)*d, and is otherwise not written;
 *   xs  [n_layers][d]  written: xs[l] = x_l + y_l, the input of layer l+1
 *                      (x_0 = x0); xs[n_layers-1] is the token's output;
 *   ys  [n_layers][d]  written if not NULL: y_l;
 *   masks: each field is a per-layer array, rows [n_layers][...] as for one
 *     token: nmask [n_layers][f/32] (required), gmask [n_layers][gw],
 *     idx [n_layers][f], count [n_layers] (each optional, NULL = not
 *     written); the union fields are ignored.
 *   ws: at least sffn_stack_workspace_bytes(stack), 256-byte aligned.
 * The kernel's grid barrier state lives in the stack handle, so calls on one
 * stack must not overlap on the GPU (order them on one stream); different
 * stacks may run concurrently only if the GPU can hold both grids, which one
 * GB300 cannot (each holds every SM). The launch needs every SM: work that
 * occupies SMs at the same time only delays it. Allocates nothing, does not
 * synchronize, may be captured in a CUDA graph. A bounded wait that runs out
 * is reported by sffn_stack_check_error.
 * Errors: INVALID_ARG, CUDA. */
sffn_status sffn_stack_decode(const sffn_stack* stack, const float* x0, float* xs, float* ys, float thres,
                              const sffn_masks* masks, void* ws, size_t ws_bytes, sffn_stream stream);

/* Synchronize the stream, read and clear the stack's device error word (OK,
 * TIMEOUT or DEVICE); after an error it also resets the grid barrier so the
 * next call starts clean. */
sffn_status sffn_stack_check_error(const sffn_stack* stack, sffn_stream stream);
void sffn_stack_destroy(sffn_stack* stack);

/* ---------------------------------------------------------------- TAM */

/* Momentum state for n_layers layers of n_groups groups (1..1024): scores
 * (fp32, start 0), lambda per layer (start lambda0, in (0, 1)), resident
 * bitset (start empty), and a device error word. */
sffn_status tam_create(int32_t n_layers, int32_t n_groups, float lambda0, tam_state** out);

/* Outputs of tam_update; every pointer is optional (NULL = not written).
 * Per-layer rows, n_layers rows each: bitsets [n][gw] with gw =
 * ceil(n_groups/32); topk [n][capacity_k] group ids in rank order (score
 * descending, then group id ascending), entries past n_res are -1;
 * n_cand [n], n_res [n]. */
typedef struct {
  uint32_t* cand;
  uint32_t* resident;
  uint32_t* load;
  uint32_t* evict;
  uint32_t* changed;
  int32_t* topk;
  int32_t* n_cand;
  int32_t* n_res;
} tam_outputs;

/* One momentum step for layers [layer0, layer0 + n_layers) (KAIROX 核心方法
 * item 4), float32 with one rounding per operation and no fused multiply-add:
 *   om = 1 - lambda; tau = om + eps;
 *   s_g = lambda * s_g;  s_g = s_g + (group g active ? om : 0);
 *   cand = {g : s_g > tau};  resident = the first capacity_k of cand ranked by
 *   (s_g descending, g ascending);  load = res & ~prev;  evict = prev & ~res;
 *   changed = res ^ prev;  the state's resident set becomes res.
 * gmask: device, row l (for layer layer0 + l) starts at gmask + l*gmask_stride
 * (words), gmask_stride >= gw. lambda < 0 uses each layer's state lambda.
 * eps >= 0, capacity_k in [0, n_groups]. One thread block per layer.
 * Errors: INVALID_ARG, CUDA. */
sffn_status tam_update(tam_state* tam, int32_t layer0, int32_t n_layers, const uint32_t* gmask,
                       int32_t gmask_stride, float lambda, float eps, int32_t capacity_k,
                       const tam_outputs* out, sffn_stream stream);

/* The whole per-layer decode step as the pages order it: the predictor, the
 * sparse FFN on the predicted masks (sffn_decode_step), then one momentum
 * step of layer `layer_index` of `tam` (tam_update with layer0 = layer_index,
 * n_layers = 1) on the group bitmask this call writes: masks->gmask for B = 1, the batch
 * union masks->ugmask for B > 1 (KAIROX 核心方法 item 4: the momentum of every
 * group is updated at every token from the predicted need; PowerInfer §5.1
 * for the predictor). All three are enqueued on `stream` in that order. The
 * momentum arguments mean what they mean for tam_update; `out` may be NULL.
 * The state must have the layer's group count and live on the same device.
 * Equivalent to sffn_decode_step followed by tam_update on the same stream;
 * a caller running many layers may instead batch the momentum steps of all
 * layers into one tam_update per token on a second stream (same results).
 * Errors: as sffn_decode_step and tam_update, and INVALID_ARG when the needed
 * group bitmask pointer is NULL. */
sffn_status sffn_decode_step_tam(const sffn_layer* layer, tam_state* tam, int32_t layer_index, const float* x,
                                 int32_t B, float thres, const sffn_masks* masks, float* y, float* x_out,
                                 void* ws, size_t ws_bytes, float lambda, float eps, int32_t capacity_k,
                                 const tam_outputs* out, sffn_stream stream);

/* Adaptive Neuron Balancer step (KAIROX 核心方法 item 5) for layers
 * [layer0, layer0 + n_layers): lambda_l <- min(hi, max(lo, lambda_l + (stall[l] ?
 * +alpha : -alpha))) in float32, where stall [n_layers] uint8 device (nonzero =
 * I/O stall). Requires 0 < lo <= hi < 1, alpha >= 0. */
sffn_status tam_adapt(tam_state* tam, int32_t layer0, int32_t n_layers, const uint8_t* stall,
                      float alpha, float lo, float hi, sffn_stream stream);

/* Copy the state out of / into caller device buffers (checkpoint / resume):
 * scores [n_layers][n_groups] fp32, lambdas [n_layers] fp32,
 * resident [n_layers][gw] u32. Any pointer may be NULL (skipped). */
sffn_status tam_get_state(const tam_state* tam, float* scores, float* lambdas, uint32_t* resident,
                          sffn_stream stream);
sffn_status tam_set_state(tam_state* tam, const float* scores, const float* lambdas,
                          const uint32_t* resident, sffn_stream stream);
sffn_status tam_get_shape(const tam_state* tam, int32_t* n_layers /* host */, int32_t* n_groups /* host */);
sffn_status tam_check_error(const tam_state* tam, sffn_stream stream);
void tam_destroy(tam_state* tam);

/* ------------------------------------------- 4-bit projections (attention) */

/* The attention half of a decode step: the projections around it, the cache
 * of keys and values, and the attention over that cache. A step of one layer
 * is sffn_linear_forward (q, k and v), sffn_kv_append, sffn_attend,
 * sffn_linear_forward (output), then the sparse FFN (sffn_decode_step). Hot
 * calls: sffn_linear_forward, sffn_kv_append, sffn_kv_gather, sffn_attend
 * (same rules as above: they allocate nothing, never synchronize, and may be
 * captured in a CUDA graph). */

/* Rows of a two- or three-dimensional device array: element (i, h, c) is at
 * ptr + i*row_stride + h*head_stride + c (in elements; c contiguous, one h
 * for two dimensions). ptr and both strides must be multiples of 16 bytes
 * (a stride that is never stepped along is not looked at). */
typedef struct {
  void* ptr;
  int64_t row_stride;
  int64_t head_stride;
} sffn_rows;

/* A linear layer with 4-bit codes and group scales:
 *   y[b][n] = sum_k scale[n][k/G] * (code[n][k] - zero[n][k/G]) * x[b][k]
 *             + bias[n] + residual[b][n],
 * codes in [-8, 7], zero = 0 if the layer has none.
 *   in_features: multiple of group, at most 65536.
 *   out_features: 1 .. 1048576.
 *   group: 32, 64 or 128 consecutive inputs share a scale (and a zero).
 *   scale_dtype: type of the scales and zeros as given and stored.
 *   has_zero: nonzero if the layer has zeros.
 *   max_batch: largest B the layer will be called with, 1..32. */
typedef struct {
  int32_t in_features, out_features, group, scale_dtype, has_zero, max_batch;
} sffn_linear_desc;

typedef struct sffn_linear sffn_linear;

/* Host-only check of a description (no CUDA call). */
sffn_status sffn_linear_validate(const sffn_linear_desc* desc);
/* Allocates the packed arrays on the current device. Errors: INVALID_ARG, OOM, CUDA. */
sffn_status sffn_linear_create(const sffn_linear_desc* desc, sffn_linear** out);
/* Pack codes [out][in] int8 (each in [-8, 7]; another value fails with
 * DEVICE and leaves the layer unpacked), scales and zeros [out][in/group] in
 * scale_dtype (zeros NULL exactly if has_zero is 0) and bias [out] fp32 or
 * NULL. Setup call: synchronizes the stream. Device pointers, 16-byte
 * aligned. Errors: INVALID_ARG, DEVICE, CUDA. */
sffn_status sffn_linear_pack(sffn_linear* linear, const int8_t* codes, const void* scales, const void* zeros,
                             const float* bias, sffn_stream stream);
sffn_status sffn_linear_get_desc(const sffn_linear* linear, sffn_linear_desc* out /* host */);
/* Bytes of caller workspace for batch B (256-byte aligned, contents need no
 * initialisation; 0 if the arguments are invalid or none is needed). */
size_t sffn_linear_workspace_bytes(const sffn_linear* linear, int32_t B);
/* x [B][in], y [B][out] and residual [B][out] (ptr NULL = none) in `dtype`;
 * sums in fp32, y rounded once. fp16 x is taken as it is; of bf16 and fp32 x,
 * what lies below 2^-38 of a token's largest element does not count (a bf16
 * element loses nothing down to 2^-30 of it; fp32 elements keep 22 bits).
 * residual may be y itself; x must not overlap y. A token with a non-finite x
 * gives non-finite values in its own outputs only. y and residual need only be
 * aligned to their elements, with any stride >= out.
 * Errors: INVALID_ARG (also: not packed), CUDA. */
sffn_status sffn_linear_forward(const sffn_linear* linear, sffn_rows x, int32_t B, sffn_rows residual, sffn_rows y,
                                int32_t dtype, void* ws, size_t ws_bytes, sffn_stream stream);
/* Synchronize the stream, then read and clear the layer's device error word
 * (TIMEOUT: a bounded wait ran out). */
sffn_status sffn_linear_check_error(const sffn_linear* linear, sffn_stream stream);
void sffn_linear_destroy(sffn_linear* linear);

/* ------------------------------------------------- paged 4-bit key/value cache */

/* Pages of cached keys and values of one layer. A page holds page_size
 * consecutive positions of one sequence for every key head. Keys and values
 * are rounded per (position, head, group of channels) to sixteen levels
 *   value = mid + step * (2u - 15),  u in 0..15,
 * in fp32 arithmetic, one rounding per operation: lo, hi = least and largest
 * value of the group, mid = f16(lo/2 + hi/2), step = f16(max(hi - mid,
 * mid - lo) * f32(1/15)) (both limited to +-65504), u = floor((x - mid) *
 * (1 / (2 step)) + 8) limited to 0..15, and u = 8 if step is 0. A group with
 * a non-finite value is stored as NaN (step = NaN).
 *   n_pages: 1 .. 2^31 - 1.  page_size: 16, 32 or 64.  n_kv_heads: 1 .. 1024.
 *   head_dim: 64, 128 or 256.  group: 32, 64 or 128, at most head_dim. */
typedef struct {
  int32_t n_pages, page_size, n_kv_heads, head_dim, group;
} sffn_kv_desc;

typedef struct sffn_kv sffn_kv;

sffn_status sffn_kv_validate(const sffn_kv_desc* desc);
/* Bytes of device memory the pages of a cache take (0 if desc is invalid). */
size_t sffn_kv_bytes(const sffn_kv_desc* desc);
/* Allocates the pages on the current device (contents undefined: a position
 * is read only after a call appended it). Errors: INVALID_ARG, OOM, CUDA. */
sffn_status sffn_kv_create(const sffn_kv_desc* desc, sffn_kv** out);
sffn_status sffn_kv_get_desc(const sffn_kv* kv, sffn_kv_desc* out /* host */);
/* Synchronize the stream, then read and clear the cache's device error word
 * (DEVICE: a page id, length, row start or rotation position out of range was
 * seen). */
sffn_status sffn_kv_check_error(const sffn_kv* kv, sffn_stream stream);
void sffn_kv_destroy(sffn_kv* kv);

/* The tokens of a call. Sequence s has the n_s = q_start[s+1] - q_start[s]
 * rows q_start[s] .. q_start[s+1] - 1 of the call's arrays, and kv_len[s]
 * cached positions, these tokens included: its row q_start[s] + i is at
 * position kv_len[s] - n_s + i. Position p lives in page table[s][p /
 * page_size], slot p % page_size. A row whose position is negative has no
 * place in the cache (a sequence that is padded at its front).
 *   table   [n_seq][table_stride] page ids, device
 *   kv_len  [n_seq] device
 *   q_start [n_seq + 1] device, ascending from at least 0 to at most
 *           n_tokens; or NULL: one token per sequence (n_tokens == n_seq)
 * A length above table_stride * page_size is taken as that, and a page id
 * outside [0, n_pages) as page 0 in reads and nowhere in writes; both set
 * the cache's device error word. Rows outside every sequence (before
 * q_start[0] or from q_start[n_seq] on) are ignored: nothing is read from or
 * written to their places. Starts that descend or lie outside 0 .. n_tokens
 * set the error word too, and the call then writes nothing.
 * table_stride * page_size: at most 2^30. */
typedef struct {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t n_seq, n_tokens, table_stride;
} sffn_kv_batch;

/* Position rotation: channel pairs (a, b) of the first `dim` channels of a
 * query or key head become (a cos - b sin, b cos + a sin) with (cos, sin) =
 * table[position][pair], fp32, each product and sum rounded once. style 0:
 * pair j is channels (j, j + dim/2); style 1: channels (2j, 2j + 1). dim is
 * even, 0 < dim <= head_dim; table is 8-byte aligned. A position outside
 * [0, length) is not rotated and sets the cache's device error word. */
typedef struct {
  const float* table;           /* [length][dim / 2][2], device */
  const int32_t* positions;     /* [n_tokens] device, or NULL: the position in the cache */
  int32_t length, dim, style;
} sffn_rope;

/* Append keys and values of the batch's tokens: k, v [n_tokens][n_kv_heads]
 * [head_dim], rotating the keys on the way if `rope` is not NULL; and, if
 * q.ptr is not NULL, write the rotated queries q [n_tokens][n_q_heads]
 * [head_dim] to q_out (q_out may be q itself). All in `dtype`. Rows without a
 * place in the cache only have their queries written. Two rows of one call
 * must not share a place. n_tokens * (n_q_heads + 2 n_kv_heads) is at most
 * 2^30. Errors: INVALID_ARG, CUDA. */
sffn_status sffn_kv_append(const sffn_kv* kv, const sffn_kv_batch* batch /* host */, sffn_rows q, int32_t n_q_heads,
                           sffn_rows k, sffn_rows v, sffn_rows q_out, const sffn_rope* rope /* host, or NULL */,
                           int32_t dtype, sffn_stream stream);

/* Read back what the cache holds for the batch's tokens: k_out, v_out
 * [n_tokens][n_kv_heads][head_dim] in `dtype` (either ptr may be NULL). Rows
 * without a place in the cache give 0. Errors: INVALID_ARG, CUDA. */
sffn_status sffn_kv_gather(const sffn_kv* kv, const sffn_kv_batch* batch /* host */, sffn_rows k_out, sffn_rows v_out,
                           int32_t dtype, sffn_stream stream);

/* Attention of the batch's tokens over the cache, after their keys and values
 * were appended. Query head h reads key head h / (n_q_heads / n_kv_heads). The
 * token at position p sees positions max(0, p - window + 1) .. p (window 0:
 * all up to p):
 *   out[i][h] = sum_j softmax_j(scale * q[i][h] . K[j]) V[j],
 *   lse[i][h] = log sum_j exp(scale * q[i][h] . K[j])  (fp32, or NULL),
 * softmax statistics and sums in fp32. A token that sees nothing gives out =
 * 0 and lse = -infinity. Positions a token does not see never reach its
 * result, whatever is stored there, and the ids of pages that no token of the
 * call sees are not looked at: those before a window may have been retired.
 * q, out in `dtype`; q and out must not overlap. fp16 q is taken as it is; of
 * bf16 and fp32 q, what lies below 2^-38 of the largest element of a row and
 * group of channels does not count (a bf16 element loses nothing down to 2^-30
 * of it; fp32 elements keep 22 bits). The same arguments give the same bits at
 * every call.
 * n_q_heads: a multiple of n_kv_heads, n_q_heads * n_tokens at most 2^30, and
 * (n_q_heads * n_tokens / 8 + n_kv_heads * n_seq) * (table_stride * page_size
 * / 32 + 2) below 2^31. scale: finite.
 * ws: at least sffn_attend_workspace_bytes, 256-byte aligned. */
size_t sffn_attend_workspace_bytes(const sffn_kv* kv, int32_t n_q_heads, int32_t n_seq, int32_t n_tokens);
sffn_status sffn_attend(const sffn_kv* kv, const sffn_kv_batch* batch /* host */, sffn_rows q, int32_t n_q_heads,
                        sffn_rows out, float* lse /* [n_tokens][n_q_heads] */, float scale, int32_t window,
                        int32_t dtype, void* ws, size_t ws_bytes, sffn_stream stream);

/* ------------------------------------- around the halves: norm and 8-bit rows */

/* What a decode step needs before, between and after its two halves: the
 * norm with the residual's addition, rows rounded to 8 bits and the
 * projections that take them, the choice of the best continuations, and the
 * reordering of the cache by the sequences that go on. Hot calls: sffn_norm,
 * sffn_quantize, sffn_linear8_forward, sffn_beam_select, sffn_kv_reorder
 * (same rules as above: they allocate nothing, never synchronize, and may be
 * captured in a CUDA graph). */

/* Root-mean-square norm of n_rows rows of `width` elements, with the
 * residual's addition before it and, if asked for, rows of 8-bit codes after
 * it:
 *   t = x + residual                         (t = x without one)
 *   f = f32(1 / sqrt(mean(t^2) + eps))       (mean and root in 64 bits)
 *   y = (t * f) * weight                     (y = t * f without one)
 *   scale = max |y| / 127,  code = y / scale rounded to the nearest whole
 *                                            number, ties to even
 * in fp32, one rounding per operation, so that codes and scales are defined
 * (the mean is good to 2^-44: f is its rounding but for one row in some 2^20,
 * where it may be the next number).
 *   x, residual, sum_out (t, rounded once) in `dtype`; y in `y_dtype`;
 *   weight [width] fp32; codes int8, scales [n_rows] fp32.
 * residual, weight, sum_out, y and (codes, scales) are optional (NULL), but
 * one of y and codes is required. x, residual and sum_out may be the same
 * rows; y may be x or residual if its elements have their size, but not
 * sum_out; rows must not overlap otherwise. A row whose
 * y are all 0 has scale 0 and codes 0; a row with a y that is not finite has
 * scale NaN and codes 0. Pointers and strides need only be aligned to their
 * elements (rows on 16 bytes are faster).
 * n_rows: 0 .. 2^30.  width: 1 .. 32768.  eps: finite, not negative.
 * Errors: INVALID_ARG, CUDA. */
sffn_status sffn_norm(sffn_rows x, sffn_rows residual, const float* weight, double eps, int32_t n_rows, int32_t width,
                      sffn_rows sum_out, sffn_rows y, sffn_rows codes, float* scales, int32_t dtype, int32_t y_dtype,
                      sffn_stream stream);

/* Codes and scales of rows as they are: scale = max |x| / 127 and so on, as
 * above with y = x. width: 1 .. 65536. Errors: INVALID_ARG, CUDA. */
sffn_status sffn_quantize(sffn_rows x, int32_t n_rows, int32_t width, sffn_rows codes, float* scales, int32_t dtype,
                          sffn_stream stream);

/* A linear layer with 8-bit codes, a scale for each output channel, and rows
 * of 8-bit codes with a scale each:
 *   y[b][n] = (sum_k code[n][k] * x[b][k]) * (scale[n] * x_scale[b])
 *             + bias[n] + residual[b][n].
 * The sum is exact (32-bit whole numbers), what follows is fp32 with one
 * rounding per operation, so that a token's y does not depend on the batch
 * it comes in.
 *   in_features: multiple of 16, 16 .. 65536.  out_features: 1 .. 1048576.
 *   max_batch: largest B the layer will be called with, 1 .. 65536. */
typedef struct {
  int32_t in_features, out_features, max_batch;
} sffn_linear8_desc;

typedef struct sffn_linear8 sffn_linear8;

/* Host-only check of a description (no CUDA call). */
sffn_status sffn_linear8_validate(const sffn_linear8_desc* desc);
/* Allocates the packed arrays on the current device. Errors: INVALID_ARG, OOM, CUDA. */
sffn_status sffn_linear8_create(const sffn_linear8_desc* desc, sffn_linear8** out);
/* Pack codes [out][in] int8, scales [out] fp32 and bias [out] fp32 or NULL.
 * Setup call: synchronizes the stream. Device pointers, 16-byte aligned.
 * Errors: INVALID_ARG, CUDA. */
sffn_status sffn_linear8_pack(sffn_linear8* linear, const int8_t* codes, const float* scales, const float* bias,
                              sffn_stream stream);
sffn_status sffn_linear8_get_desc(const sffn_linear8* linear, sffn_linear8_desc* out /* host */);
/* Bytes of caller workspace for batch B (256-byte aligned, contents need no
 * initialisation; 0 if the arguments are invalid or none is needed). */
size_t sffn_linear8_workspace_bytes(const sffn_linear8* linear, int32_t B);
/* x [B][in] int8 (pointer and stride multiples of 16 bytes) with x_scales [B]
 * fp32, y and residual [B][out] in `dtype` (residual.ptr NULL = none; it may
 * be y itself), element-aligned, with any stride >= out. y must not overlap
 * x. A token whose scale is NaN gives NaN in its own outputs only.
 * Errors: INVALID_ARG (also: not packed), CUDA. */
sffn_status sffn_linear8_forward(const sffn_linear8* linear, sffn_rows x, const float* x_scales, int32_t B,
                                 sffn_rows residual, sffn_rows y, int32_t dtype, void* ws, size_t ws_bytes,
                                 sffn_stream stream);
/* Synchronize the stream, then read and clear the layer's device error word
 * (TIMEOUT: a bounded wait ran out). */
sffn_status sffn_linear8_check_error(const sffn_linear8* linear, sffn_stream stream);
void sffn_linear8_destroy(sffn_linear8* linear);

/* -------------------------------------------- search over several continuations */

/* The n_out best continuations of each of `batch` searches with `beams`
 * sequences each, over a vocabulary: with z = logits[b * beams + j],
 *   total[j][v] = scores[b][j] + z[v] - log sum_u exp(z[u]),
 * the n_out largest by (total, then lowest j * vocab + v), largest first. Of
 * one sequence a larger logit goes first also where its score is so large that
 * totals in 64 bits are equal.
 *   vocab: 1 .. 2^24.  beams: 1 .. 64.  n_out: 1 .. 64.
 *   max_batch: largest batch the handle will be called with, at least 1, max_batch * beams at most 65535. */
typedef struct {
  int32_t vocab, beams, n_out, max_batch;
} sffn_beam_desc;

typedef struct sffn_beam sffn_beam;

sffn_status sffn_beam_validate(const sffn_beam_desc* desc);
/* A handle of the current device (a device error word only). Errors: INVALID_ARG, OOM, CUDA. */
sffn_status sffn_beam_create(const sffn_beam_desc* desc, sffn_beam** out);
sffn_status sffn_beam_get_desc(const sffn_beam* beam, sffn_beam_desc* out /* host */);
/* Bytes of caller workspace for `batch` searches (256-byte aligned, contents
 * need no initialisation; 0 if the arguments are invalid). */
size_t sffn_beam_workspace_bytes(const sffn_beam* beam, int32_t batch);
/* logits [batch * beams][vocab] in `dtype`, element-aligned, any stride >=
 * vocab (rows on 16 bytes are faster); scores [batch][beams] fp32.
 * done [batch][beams] bytes or NULL: a sequence whose byte is not 0 has ended,
 * its logits are not read, and its only continuation is end_token with the
 * score it has. A sequence whose score is -infinity has none, nor has one
 * whose logits are all -infinity (masked tokens are -infinity and are never
 * chosen). Logits with a NaN or +infinity, or a score that is NaN or
 * +infinity, have none either and set the handle's device error word.
 * out_scores fp32, out_parents (j) and out_tokens (v) [batch][n_out]; places
 * that nothing is left for have score -infinity, parent 0 and token 0 (a total
 * below fp32's range has score -infinity too, but its parent and token).
 * Exponentials are summed in fp32 with what additions round off (a logarithm
 * of a sum is good to about 2^-22, and to 2^-18 whatever the logits), totals
 * compared in 64 bits; the same arguments give the same bits at every call.
 * out_scores may be `scores` if n_out is `beams`. Errors: INVALID_ARG, CUDA. */
sffn_status sffn_beam_select(const sffn_beam* beam, sffn_rows logits, const float* scores, const uint8_t* done,
                             int32_t end_token, int32_t batch, float* out_scores, int32_t* out_parents,
                             int32_t* out_tokens, int32_t dtype, void* ws, size_t ws_bytes, sffn_stream stream);
/* Synchronize the stream, then read and clear the handle's device error word
 * (DEVICE: logits or a score that have no distribution were seen). */
sffn_status sffn_beam_check_error(const sffn_beam* beam, sffn_stream stream);
void sffn_beam_destroy(sffn_beam* beam);

/* Reorder the cache by the sequences that go on. The batch's sequences come
 * in groups of `beams`, all sequences of a group with the same kv_len n;
 * sequence s of group g goes on as a copy of sequence m = g * beams +
 * parents[s]:
 *   - pages that are full (the first n / page_size) are shared: their ids in
 *     row s of table_out are those of row m of batch->table. Nothing may be
 *     written to them from then on (append writes from position n on; a
 *     search that starts anew starts from a table without shared pages).
 *   - the n % page_size positions of the page that is not full are copied, in
 *     every one of the n_kv caches, from the page that row m of batch->table
 *     names to the one that row s of table_out named before the call.
 * Ids of table_out from that page on are left as they are. table_out may be
 * batch->table itself with the same stride (the usual case): every sequence
 * then keeps its own last page, whatever it is a copy of. Otherwise it must
 * not overlap it, and the last pages that it names must differ from those of
 * batch->table. The last pages of a call's sequences must differ from each
 * other in either table.
 *   kvs [n_kv] host array of caches that differ in n_pages at most (the
 *       layers of a model, which share their tables), 1 .. 128.
 *   batch: table, kv_len, n_seq and table_stride are used; n_seq is a
 *       multiple of beams.  parents [n_seq] device, each in 0 .. beams - 1.
 *   beams: 1 .. 64.  out_stride: at least table_stride.
 * A group whose lengths differ or do not fit the table, or with a parent out
 * of range, is left as it was; a last page's id out of range is not copied
 * from or to. All of these set the error word of the first cache.
 * Errors: INVALID_ARG, CUDA. */
sffn_status sffn_kv_reorder(const sffn_kv* const* kvs /* host */, int32_t n_kv, const sffn_kv_batch* batch /* host */,
                            const int32_t* parents, int32_t beams, int32_t* table_out, int32_t out_stride,
                            sffn_stream stream);

/* ---------------------------------------------------------------- self-test */

/* Exercise the bounded-wait path without any fault: one thread block waits
 * on a shared-memory barrier that nothing will complete, gives up after
 * limit_us microseconds (1..100000), records SFFN_ERR_TIMEOUT in the layer's
 * device error word and returns. sffn_layer_check_error then reports TIMEOUT
 * and the context stays usable. */
sffn_status sffn_selftest_wait_timeout(const sffn_layer* layer, int32_t limit_us, sffn_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SFFN_H_ */
