/*
 * raxlora.h - C ABI of the MI355X (gfx950) batched multi-adapter LoRA library.
 *
 * The library applies, for every token t with its own adapter slot i(t) in a
 * resident pool,
 *
 *     y[t] += s_i * B_i (A_i x[t])            (the base output W0 x[t] is the caller's)
 *
 * as a shrink (x -> rank space through lora_a = A) and an expand (rank space ->
 * output through lora_b = B), driven by per-batch routing metadata.
 *
 * Passages this interface follows (page title, then section):
 *   [llama.cpp] "llama.cpp 源码完全拆解(十六):LoRA 适配器——低秩补丁如何挂进 ggml 计算图"
 *   [TRT-LLM]   "TensorRT-LLM 源码完全拆解(二十一):LoRA 服务——adapter 池、批内多适配器与
 *               前向替换的完整链路"
 *   [vLLM-deep] "vLLM LoRA 实现深度解析"
 *   [vLLM-book] "第16章 LoRA 适配器热切换：一个引擎承载多个微调"
 *
 * Conventions for every call:
 *   - Matrices are row-major.  x is [T, k] with row stride ldx elements, y is
 *     [T, D] with D = sum of the slice widths and row stride ldy.  A adapter's
 *     A (shrink) is [rank, k] and its B (expand) is [d_n, rank] per output slice,
 *     as PEFT stores lora_a / lora_b ([vLLM-deep] §3.3).
 *   - "device pointer" means memory on the pool's GPU; "host pointer" ordinary
 *     process memory.  The library never takes ownership of caller memory.
 *   - Calls that take a hipStream_t only enqueue work on that stream (no host
 *     synchronisation) unless documented as synchronous.  The caller keeps its
 *     buffers alive until that work has completed.
 *   - Every call returns LORA_OK (0) or a negative lora_status; nothing throws
 *     across the ABI.  lora_last_error() gives a message for the calling thread.
 *     Argument checks run before any HIP call, so a rejected call has no effect.
 *   - Alignment: k and every slice width must be multiples of 8, ldx and ldy
 *     multiples of 8 elements, and x, y, u 16-byte aligned (the kernels move 16
 *     bytes per lane; [TRT-LLM] "前向替换" notes the grouped kernels assume K, N of
 *     at least 8).  Otherwise LORA_ERR_ALIGN.
 *   - Thread safety: distinct objects may be used from distinct threads.  One
 *     pool or routing object must not be mutated (register/unregister/build) while
 *     work that reads it may still run on another stream.  lora_linear and
 *     lora_shrink use a workspace owned by the pool, so two of them on one pool
 *     must not overlap in time (same stream is always safe).
 *   - Environment (read by the library; none is needed, all select among
 *     equivalent paths or launch shapes, and results stay within the tolerances
 *     the tests check):
 *       RAXLORA_MFMA_MIN_SEG  segments of at least this many tokens go to the
 *                             matrix cores (bf16 and FP8 pools; default 4; read when a
 *                             routing object is created)
 *       RAXLORA_DISABLE_MFMA  1: every segment on the vector units
 *       RAXLORA_CB1_MAX       matrix-core expand units take one 128-column block
 *                             instead of four when (column groups of four x tile
 *                             slots) is at most this (default 512)
 *       RAXLORA_XCD_GROUP     consecutive decode units kept on one XCD (default 4)
 *       RAXLORA_TILE_INTERLEAVE  matrix-core expand: 0 gives XCD x the x-th eighth
 *                             of the tile list, n > 0 deals runs of n tiles round
 *                             the XCDs (default: 1 when T < 64 S, else 0; the
 *                             results are the same either way)
 *       RAXLORA_GROUP_ORDER   0: grouped calls lay out their modules and decode units
 *                             in the order given (default 1: modules with the longest
 *                             shrink items first, decode expand units by descending
 *                             slot rank; results are the same either way)
 *       RAXLORA_LOG           1: one line on stderr per shrink or expand launch with
 *                             the launch shape chosen (path, k split, waves, units)
 *       RAXLORA_SLOT_MODE     0: never use the slot-major kernels (one unit per slot,
 *                             weight loads issued before the routing data arrives);
 *                             1: use them wherever the shape allows (T <= 256,
 *                             in_features <= 32768, bf16 or FP8 weights); default:
 *                             for 4 S <= T <= 128
 */
#ifndef RAXLORA_H
#define RAXLORA_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lora_pool lora_pool;
typedef struct lora_routing lora_routing;

/* LORA_FP8E4M3: adapter weights as OCP float8 e4m3 ("fn": 4 exponent bits, bias 7, 3
 * mantissa bits, largest finite 448), the native-FP8 adapter cache of [TRT-LLM]
 * (the FP8 special case of the weight preparation, and "前向替换").  A pool of this
 * weight type takes bf16 activations x, which the kernels clamp to [-448, 448]
 * and round to e4m3 before use, as the page converts the input; products are exact
 * and accumulate in fp32; y is bf16 or fp32.  The matrix-core shrink runs on the FP8
 * matrix cores (e4m3 x e4m3); the vector units and the expand widen the weights to
 * bf16 in registers (exact). */
typedef enum { LORA_F32 = 0, LORA_BF16 = 1, LORA_FP8E4M3 = 2 } lora_dtype;

typedef int lora_status;
#define LORA_OK                0
#define LORA_ERR_INVALID_ARG  (-1)   /* null handle or pointer, non-finite value, bad flag   */
#define LORA_ERR_SHAPE        (-2)   /* sizes or strides inconsistent                         */
#define LORA_ERR_DTYPE        (-3)   /* input dtype differs from the pool's                   */
#define LORA_ERR_RANK         (-4)   /* rank outside [1, max_lora_rank]                       */
#define LORA_ERR_SLOT         (-5)   /* slot outside [0, max_slots)                           */
#define LORA_ERR_CAPACITY     (-6)   /* more tokens than the object was created for           */
#define LORA_ERR_HIP          (-7)   /* a HIP runtime call failed                             */
#define LORA_ERR_OOM          (-8)   /* device allocation failed                              */
#define LORA_ERR_NO_DEVICE    (-9)   /* no usable GPU / device index out of range             */
#define LORA_ERR_ALIGN        (-10)  /* alignment rule above violated                         */
#define LORA_ERR_STATE        (-11)  /* object used out of order (e.g. routing never built)   */

/* register_adapter flags */
#define LORA_SRC_DEVICE   1u   /* A_slices / B_slices are device pointers (else host)          */
#define LORA_PREMULTIPLY  2u   /* fold the scale into B at registration                        */

/* Limits fixed at build time. */
#define LORA_MAX_SLICES    8
#define LORA_MAX_SLOTS     1024
#define LORA_MAX_RANK      256
#define LORA_MAX_IN_FEATURES 65536
#define LORA_MAX_GROUP     8      /* target modules of one grouped call */
#define LORA_NOALLOC_SCRATCH_BYTES (16u << 20)   /* scratch of lora_linear_noalloc, per GPU */

/* Message for the last failing call on this thread ("" if none). Never NULL. */
const char* lora_last_error(void);
/* Static name of a status code. */
const char* lora_status_string(lora_status status);

/*
 * Scale of the low-rank branch ([llama.cpp] "缩放系数到底乘在哪": adapter_scale *
 * alpha / rank, or adapter_scale alone when alpha is 0, i.e. absent; [TRT-LLM]
 * "LoraManager 的加载流水线" step 4 and [vLLM-deep] §1 "rsLoRA 变体": alpha/sqrt(rank)
 * when rslora is set).  Computed in double as adapter_scale*alpha, divided by rank
 * or sqrt(rank), and rounded once to float.  Pure host function, no device needed.
 * Errors: out_scale NULL -> INVALID_ARG; rank < 1 -> RANK; alpha or adapter_scale
 * not finite, or a non-finite result -> INVALID_ARG.
 */
lora_status lora_compute_scale(float alpha, int rank, int rslora, float adapter_scale,
                               float* out_scale);

/*
 * Create a pool of max_slots adapter slots for one target module (one linear
 * layer, or a packed group such as q/k/v or gate/up with num_slices output
 * slices of widths slice_out[0..num_slices)), like one layer's stacked LoRA
 * buffers ([vLLM-deep] §9: lora_a_stacked [max_loras, max_lora_rank, in],
 * lora_b_stacked [max_loras, out, max_lora_rank]).  max_lora_rank fixes the
 * padding of every slot ([TRT-LLM] "LoraConfig": a workspace bound, not
 * enlargeable later).  max_tokens bounds T for lora_linear / lora_shrink (it
 * sizes the pool-owned rank-space workspace: k-split partial sums, up to 16 x
 * num_slices x max_tokens x max_lora_rank fp32, and for pools of at most 32 slots
 * 16 more rows per slot, where a small decode batch's partial sums of each segment's
 * first 16 tokens go).  All slots start empty (rank 0).
 * slice_out is a host array, read during the call.  The pool owns its device
 * memory (allocated on `device` here) until lora_pool_destroy.
 * Errors: out/slice_out NULL -> INVALID_ARG; max_slots outside [1, LORA_MAX_SLOTS],
 * max_lora_rank outside [1, LORA_MAX_RANK], in_features < 1, num_slices outside
 * [1, LORA_MAX_SLICES], a slice width < 1, max_tokens < 1, in_features above
 * LORA_MAX_IN_FEATURES -> SHAPE; bad wdtype ->
 * DTYPE; in_features or a width not a multiple of 8 -> ALIGN; device missing ->
 * NO_DEVICE; allocation -> OOM.
 */
lora_status lora_pool_create(lora_pool** out, int device, int max_slots, int max_lora_rank,
                             int in_features, const int* slice_out, int num_slices,
                             lora_dtype wdtype, int max_tokens);

/*
 * A pool for the token embedding ([llama.cpp] "嵌入层:查表后再加增量": the lookup gets
 * a low-rank delta, get_rows of A by token id lifted by B; "token_embd" shape
 * contract: A is [r, V], B is [d, r]).  One slice of width d; vocab = V.  Adapters
 * are registered with lora_register_adapter as for other pools (A_slices[0] is
 * [rank, vocab], B_slices[0] is [d, rank]); the pool stores A transposed, one
 * contiguous row of max_lora_rank values per vocabulary id, so
 * lora_pool_read_slot returns A_host as [vocab, max_lora_rank].  Used only with
 * lora_embedding (and lora_expand); lora_shrink, lora_linear and lora_route_linear
 * reject it (INVALID_ARG).  Errors as lora_pool_create, except that vocab needs no
 * alignment and no upper bound (it is not a contraction length).
 */
lora_status lora_embedding_pool_create(lora_pool** out, int device, int max_slots, int max_lora_rank, int vocab,
                                       int d, lora_dtype wdtype, int max_tokens);

/* Free the pool.  All work that uses it must have completed.  NULL is a no-op. */
lora_status lora_pool_destroy(lora_pool* pool);

/*
 * Load an adapter into `slot` ([vLLM-deep] §5.3 set_lora(index, A, B): the
 * activation step writes the slot's buffers; [TRT-LLM] "AdapterSlotManager":
 * slots are fixed, their contents swapped).
 *   A_slices[n]: [rank, in_features] row-major, B_slices[n]: [slice_out[n], rank]
 *   row-major, both in the pool dtype.  A NULL pair marks a missing slice, which
 *   contributes nothing ([TRT-LLM] "LoraConfig": missing q/k/v padded with
 *   zeros); exactly one of the pair NULL is INVALID_ARG.
 *   Scale: see lora_compute_scale.  With LORA_PREMULTIPLY the pool stores
 *   round(s * B) (float32 product, one round to the pool dtype) and applies 1
 *   afterwards ([vLLM-deep] §1 "推理优化:预合并 scaling"); otherwise it stores B and
 *   multiplies the finished branch by s ([llama.cpp] "真正的核心").
 * With LORA_SRC_DEVICE the sources are device pointers and the copy is enqueued
 * on `stream`; otherwise they are host pointers and the call returns after the
 * copy has completed.  Re-registering a slot overwrites it in stream order.
 * Errors: pool NULL -> INVALID_ARG; slot -> SLOT; rank outside [1, max_lora_rank]
 * -> RANK; non-finite alpha / adapter_scale -> INVALID_ARG; unknown flag bit ->
 * INVALID_ARG; HIP failure -> HIP.
 */
lora_status lora_register_adapter(lora_pool* pool, int slot, const void* const* A_slices,
                                  const void* const* B_slices, float alpha, int rank, int rslora,
                                  float adapter_scale, unsigned flags, hipStream_t stream);

/* Empty `slot`: rank 0, so tokens still routed to it contribute nothing ([TRT-LLM]
 * "一次 decode 批次的路由": an empty slot has rank 0 and null pointers).  Enqueued on
 * `stream`.  Errors: pool NULL -> INVALID_ARG; slot -> SLOT. */
lora_status lora_unregister_adapter(lora_pool* pool, int slot, hipStream_t stream);

/* Host mirror of a slot's table entry (synchronous, no device access): rank,
 * scale still applied after the branch (1 when pre-multiplied), mask of present
 * slices, and the byte offsets of the slot's A and rank-major B blocks from the
 * pool base.  Any out pointer may be NULL. */
lora_status lora_pool_slot_info(const lora_pool* pool, int slot, int* rank, float* scale,
                                uint32_t* slice_mask, uint64_t* a_offset, uint64_t* bt_offset);

/* Copy a slot's stored slice back to host memory (synchronous; for tests):
 * A_host [max_lora_rank, in_features] (embedding pools: [vocab, max_lora_rank])
 * and Bt_host [max_lora_rank, slice_out[slice]]
 * (B transposed, rank-major), both in the pool dtype, rows >= rank zero.
 * Either pointer may be NULL. */
lora_status lora_pool_read_slot(const lora_pool* pool, int slot, int slice, void* A_host,
                                void* Bt_host);

/*
 * Routing metadata for one batch ([vLLM-book] §16.4.3 LoRAKernelMeta;
 * [TRT-LLM] "一次 decode 批次的路由": sorted_ids, per-slot counts and offsets in
 * fixed-address buffers).  The object owns fixed-address device buffers sized for
 * max_tokens tokens and max_slots slots, so the same addresses serve every batch.
 * Errors: out NULL -> INVALID_ARG; max_tokens < 1 or max_slots outside
 * [1, LORA_MAX_SLOTS] -> SHAPE; NO_DEVICE / OOM as for pools.
 */
lora_status lora_routing_create(lora_routing** out, int device, int max_tokens, int max_slots);
lora_status lora_routing_destroy(lora_routing* routing);

/*
 * Build the routing for T tokens from token_slot_ids[T] (device, int32): a slot
 * in [0, max_slots), or -1 for no LoRA.  Any other id is routed as -1 and
 * counted as invalid.  Key(t) = id, or S = max_slots for no LoRA (the sentinel
 * slot of [TRT-LLM] "AdapterSlotManager").  Produces, on the device:
 *   counts[S+1], seg_offsets[S+2] (exclusive prefix, [0] = 0, [S] = LoRA tokens,
 *   [S+1] = T), sorted_ids[T] (token indices grouped by key, ascending within a
 *   key), active slots (keys < S with tokens, ascending) and their number.
 * Enqueued on `stream`; T = 0 is allowed (ids may then be NULL).
 * Errors: routing NULL, or ids NULL with T > 0 -> INVALID_ARG; T < 0 -> SHAPE;
 * T > max_tokens -> CAPACITY.
 */
lora_status lora_build_routing(lora_routing* routing, const int32_t* token_slot_ids, int T,
                               hipStream_t stream);

/*
 * The same routing for num_seqs sequences of tokens_per_seq consecutive tokens each
 * ([TRT-LLM] "一次 decode 批次的路由": the linear-tree verification batch of speculative
 * decoding, where each sequence contributes its draft tokens plus one): seq_slot_ids
 * [num_seqs] (device, int32) holds one slot (or -1) per sequence; token t belongs to
 * sequence t / tokens_per_seq, so T = num_seqs * tokens_per_seq.  The outputs are
 * those of lora_build_routing on the per-token ids (each sequence's id repeated
 * tokens_per_seq times): the page's sequence-level sort expanded to tokens, sequence
 * q's tokens q p .. q p + p - 1 in order, counts p times the sequence counts; an
 * invalid sequence id counts its p tokens as invalid.  tokens_per_seq = 1 is
 * lora_build_routing.  Errors: NULL routing, or ids NULL with T > 0 -> INVALID_ARG;
 * num_seqs < 0 or tokens_per_seq < 1 -> SHAPE; T > max_tokens -> CAPACITY.
 */
lora_status lora_build_routing_seq(lora_routing* routing, const int32_t* seq_slot_ids, int num_seqs,
                                   int tokens_per_seq, hipStream_t stream);

/* Copy the last routing back to host memory (synchronous; for tests and
 * diagnostics).  counts[S+1], seg_offsets[S+2], sorted_ids[T], active_slots[S]
 * (entries past num_active unspecified); any pointer may be NULL.
 * Errors: STATE if the routing was never built. */
lora_status lora_routing_query(const lora_routing* routing, int32_t* counts, int32_t* seg_offsets,
                               int32_t* sorted_ids, int32_t* active_slots, int* num_active,
                               int* n_invalid);

/*
 * Shrink ([vLLM-book] §16.4.2 lora_shrink on lora_a; [vLLM-deep] §6):
 *   u[n][t][j] = sum_c A_slot(t)[n][j][c] * x[t][c]      (fp32 accumulate)
 * x: device [T, in_features] in the pool dtype (else DTYPE, [TRT-LLM] "三种输入
 * dtype": input and cache dtype must match).  u: device fp32 [num_slices, T,
 * max_lora_rank], caller-owned; written for LoRA tokens of non-empty slots and
 * j < rank (zero for a missing slice); other entries are left as they were.
 * Errors: INVALID_ARG (NULL), STATE (routing not built), SHAPE (ldx < in_features,
 * routing S != pool S), CAPACITY (T > pool max_tokens), ALIGN.
 */
lora_status lora_shrink(const lora_pool* pool, const lora_routing* routing, const void* x,
                        int ldx, float* u, hipStream_t stream);

/*
 * Expand and add ([vLLM-book] §16.4.2 lora_expand on lora_b; [TRT-LLM] "前向替换":
 * the correction is added in place onto the base output):
 *   y[t][o_n + i] = round_y( y[t][o_n + i] + s * sum_j B_slot(t)[n][i][j] * u[n][t][j] )
 * with fp32 arithmetic and one rounding to ydtype.  u as written by lora_shrink.
 * y: device [T, D], in/out, ydtype = the pool dtype or LORA_F32.  Rows of no-LoRA
 * tokens, of empty or zero-scale slots, and columns of missing slices are not
 * written.  Errors as lora_shrink, plus DTYPE for an unsupported ydtype.
 */
lora_status lora_expand(const lora_pool* pool, const lora_routing* routing, const float* u,
                        void* y, int ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * Fused shrink + expand onto the caller's base output ([TRT-LLM] "前向替换":
 * forward_with_base adds the LoRA result onto the base projection; [vLLM-book]
 * §16.4.4 add_lora_linear).  Same result as lora_shrink then lora_expand, with the
 * intermediate kept in the pool's workspace as k-split partial sums, added in
 * split order by the expand, so repeated calls are bitwise identical (and equal
 * to lora_shrink then lora_expand).  Long same-slot segments of bf16 and FP8 pools go to
 * the matrix cores (MFMA).  Two kernel launches per call.
 * Errors as lora_expand.
 */
lora_status lora_linear(const lora_pool* pool, const lora_routing* routing, const void* x, int ldx,
                        void* y, int ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * Routing and fused shrink + expand of one batch: lora_build_routing(routing,
 * token_slot_ids, T) followed by lora_linear(pool, routing, x, y), with the same
 * results (routing outputs and y bitwise identical).  For 1 <= T <= 256 tokens and
 * pools of at most 255 slots the routing is built inside the shrink launch, whose
 * units find their segments from token_slot_ids directly ([vLLM-book] §16.4.2: the
 * per-batch metadata that groups tokens by slot; [TRT-LLM] "一次 decode 批次的路由"), so
 * the call costs two launches instead of three; larger batches take the two calls.
 * The routing object then holds this batch's routing for further lora_linear calls
 * (other target modules of the same tokens).  token_slot_ids must stay unchanged
 * until the call's work has run.  Arguments and errors as lora_build_routing and
 * lora_linear (routing and pool must have the same slot count).
 */
lora_status lora_route_linear(const lora_pool* pool, lora_routing* routing, const int32_t* token_slot_ids,
                              int T, const void* x, int ldx, void* y, int ldy, lora_dtype ydtype,
                              hipStream_t stream);

/*
 * lora_linear / lora_route_linear joined to a base projection that another stream
 * is still computing ([llama.cpp] "为什么低秩增量可以「后加」" and [TRT-LLM] "前向替换": the
 * LoRA branch and the base output are independent until the final add).  The
 * routing and the shrink (which read only ids and x) are enqueued on `stream`
 * at once; then `stream` waits for y_ready (hipStreamWaitEvent), recorded by the
 * caller after the work that writes the base output into y; then the expand adds
 * onto y.  y_ready NULL: exactly lora_linear / lora_route_linear.  Results are
 * bitwise those of the base work followed by the plain call.  Arguments and errors
 * as lora_linear / lora_route_linear, plus HIP if the wait cannot be enqueued.
 */
lora_status lora_linear_join(const lora_pool* pool, const lora_routing* routing, const void* x, int ldx,
                             void* y, int ldy, lora_dtype ydtype, hipStream_t stream, hipEvent_t y_ready);
lora_status lora_route_linear_join(const lora_pool* pool, lora_routing* routing, const int32_t* token_slot_ids,
                                   int T, const void* x, int ldx, void* y, int ldy, lora_dtype ydtype,
                                   hipStream_t stream, hipEvent_t y_ready);

/*
 * lora_linear for callers that cannot allocate device memory at call time (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same shrink and expand launches with the same results bitwise, but the k-split
 * partial sums live in a fixed scratch array of LORA_NOALLOC_SCRATCH_BYTES inside the
 * library's device image instead of the pool's workspace.  The call allocates and
 * frees nothing (the array's device address is looked up once per GPU, on the first
 * call there).  The caller still passes x and y as for lora_linear.
 * Every call on one GPU shares that GPU's array and leaves its last contents there;
 * nothing in it needs to start at zero.  Calls that overlap in time on one GPU (other
 * streams, other threads) race on it: serialise them, e.g. on one stream.
 * Needs nsplit * num_slices * T * Rk * 4 bytes, where Rk is max_lora_rank rounded up
 * to 32 and nsplit at most 16 (in_features / 512 rounded up, halved for batches of at
 * least 64 tokens per slot); above the maximum the call fails with CAPACITY before any
 * work is enqueued (when 16 rows per slot more fit as well, a small decode batch uses
 * them as the pool's workspace would).  Arguments and other errors as lora_linear.
 */
lora_status lora_linear_noalloc(const lora_pool* pool, const lora_routing* routing, const void* x, int ldx, void* y,
                                int ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * Several target modules of one batch in one shrink and one expand launch: for each
 * m < num_pools, lora_linear(pools[m], routing, x[m], ldx[m], y[m], ldy[m], ydtype),
 * with the same results bitwise (every module's units compute what its own call
 * computes).  This is the grouped form of the pages' layer step: [TRT-LLM] "前向替换:
 * LoraLayer 的三条路径" sizes one intermediate buffer [num_layer_modules, batch_size,
 * max_rank] and runs one grouped product over every (module, slot) problem of the
 * layer; [vLLM-book] §16.4.4 add_shrink / add_expand take several slices in one call.
 * A layer's q/k/v/o/gate/up/down modules then cost two launches instead of two each
 * ([llama.cpp] "性能与工程取舍": in decode the extra cost of LoRA is mostly launches).
 *   pools[m]: distinct linear pools with the routing's slot count, all of one weight
 *   dtype and of max_lora_rank padding to one multiple of 32; each keeps its own
 *   workspace, so no pool may appear twice.  x[m] is [T, in_features of pools[m]]
 *   with row stride ldx[m]; y[m] is [T, D of pools[m]] with row stride ldy[m]; the y
 *   of different modules must not share elements (they may be column ranges of one
 *   buffer).  Host arrays pools, x, ldx, y, ldy are read during the call.
 * Errors: INVALID_ARG (NULL array or entry, a repeated pool, an embedding pool),
 * SHAPE (num_pools outside [1, LORA_MAX_GROUP], slot count or rank padding differing),
 * DTYPE (weight dtypes differing, or as lora_linear), plus those of lora_linear for
 * each module.
 */
lora_status lora_linear_group(const lora_pool* const* pools, int num_pools, const lora_routing* routing,
                              const void* const* x, const int* ldx, void* const* y, const int* ldy, lora_dtype ydtype,
                              hipStream_t stream);

/*
 * lora_build_routing(routing, token_slot_ids, T) followed by lora_linear_group: for
 * 1 <= T <= 256 tokens and at most 255 slots the routing is built inside the grouped
 * shrink launch (two launches for the whole layer step); larger batches take the
 * routing launch first.  Routing outputs and y bitwise those of the separate calls.
 * Arguments and errors as lora_build_routing and lora_linear_group.
 */
lora_status lora_route_linear_group(const lora_pool* const* pools, int num_pools, lora_routing* routing,
                                    const int32_t* token_slot_ids, int T, const void* const* x, const int* ldx,
                                    void* const* y, const int* ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * Embedding LoRA onto the caller's lookup result ([llama.cpp] "嵌入层:查表后再加增量"):
 *   y[t][i] = round_y( y[t][i] + s * sum_j B_slot(t)[i][j] * A_slot(t)[j][vocab_ids[t]] )
 * for LoRA tokens of the routing (built from the tokens' slot ids as usual).
 * vocab_ids: device int32 [T], the tokens' vocabulary ids; an id outside
 * [0, vocab) contributes zero (its row is rewritten as y + 0).  Two launches: a
 * gather of each token's row of A into the pool's workspace, then the expand of
 * lora_linear.  y as for lora_expand; the pool must come from
 * lora_embedding_pool_create (else INVALID_ARG).  Errors as lora_expand, plus
 * INVALID_ARG for vocab_ids NULL with T > 0.
 */
lora_status lora_embedding(const lora_pool* pool, const lora_routing* routing, const int32_t* vocab_ids, void* y,
                           int ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * lora_build_routing(routing, slot_ids, T) followed by lora_embedding(pool,
 * routing, vocab_ids, y), with the same results (routing outputs and y bitwise
 * identical): the gather reads the tokens' slot ids directly and writes each
 * token's rank row by token index, and for T <= 256 tokens and pools of at most
 * 255 slots the routing is built inside the gather launch (two launches instead of
 * three).  slot_ids, vocab_ids: device int32 [T].  Errors as lora_build_routing and
 * lora_embedding.
 */
lora_status lora_route_embedding(const lora_pool* pool, lora_routing* routing, const int32_t* slot_ids, int T,
                                 const int32_t* vocab_ids, void* y, int ldy, lora_dtype ydtype, hipStream_t stream);

/*
 * ---- Between the packed q/k/v projection and the o projection of a layer ----
 *
 * The page plan, the rotary append and the paged attention below take a step from the
 * packed q/k/v rows (base output plus lora_linear's correction) to the attention output
 * that the o projection reads.  They share one paged cache: keys and values lie in pages
 * of page_size tokens, a sequence's block table names its pages in order, and a token's
 * slot is page * page_size + offset within the page.  Conventions as above; in addition:
 *   - page_size is a power of two from 16 to 1024 and num_pages * page_size < 2^31.
 *   - Ids, lengths, positions and slots are int32 device vectors.  Page ids and slots
 *     outside the cache are never followed: a token with such a slot is not stored, the
 *     keys of such a page are left out of the attention.
 */
#define LORA_MAX_SEQS      4096   /* sequences of one step */
#define LORA_MAX_HEAD_DIM  256
#define LORA_PLAN_META     8      /* words of lora_page_plan's meta */

/*
 * One layer's paged cache, the caller's memory.  Element i of the key (value) of kv head h
 * at offset o of page p lies at k (v) + p * page_stride + o * token_stride + h *
 * head_stride + i, strides in elements, the same for k and v: [page][offset][head][i] and
 * [page][head][offset][i] are both possible.  dtype LORA_BF16, LORA_F32 or LORA_FP8E4M3;
 * an e4m3 cache stands for its values times k_scale (keys) and v_scale (values), which are
 * positive and finite (ignored for the other types).  Rules, checked by the calls:
 * head_dim a multiple of 16 up to LORA_MAX_HEAD_DIM (SHAPE above it, else ALIGN), strides
 * multiples of 16, below 2^25 for token_stride, large enough that no two elements share
 * an address (SHAPE), k and v 16-byte aligned (ALIGN).
 */
typedef struct lora_kv_cache {
  void* k;
  void* v;
  int64_t page_stride, token_stride, head_stride;
  int32_t num_pages, page_size, num_heads, head_dim;
  int32_t dtype;
  float k_scale, v_scale;
} lora_kv_cache;

/*
 * Block table, slot map and positions of one step, from the request lengths, with the
 * pages themselves taken from and given back to a ring of free pages, all on the GPU.
 * Request r has past_lens[r] tokens in the cache and gets new_lens[r] >= 0 more in this
 * step, or has ended (new_lens[r] = -1).  Its tokens follow those of request r - 1 in the
 * batch.  free_pages[num_pages] is a ring of page ids: cursor[0] is the place of the
 * first free one, cursor[1] their number.
 *   - A request needs ceil((past + new) / page_size) - ceil(past / page_size) pages.
 *     Requests draw from the ring in order; the first request whose need (with those
 *     before it) passes the number of free pages is refused, and so is every later one
 *     that needs any.  A granted request's new page ids go into its block table row.
 *   - An ended request's pages (those of its past tokens) go to the ring's end, in order
 *     of request and page; the step itself does not draw them.  Its row stays as it is.
 * Written: seq_lens[num_seqs] = past + new, or 0 for ended and refused requests (lora_paged_attention
 * then gives zeros; a refused request keeps its pages and asks again with the same past, so the next
 * step's past is seq_lens only where that is above 0, else 0 after an end and the past before it
 * otherwise); query_start[num_seqs + 1] = first token of each request; for t <
 * num_tokens positions[t] = past + index in the request and slots[t] (-1 for refused
 * requests); tokens past the batch's last get position 0 and slot -1, so a step of fixed size can be
 * padded.  cursor_out[0..1] = the ring after the step; cursor_out may be cursor (a step
 * replayed from a graph then advances).  cursor[2] and cursor[3] are scratch words of the
 * call, zero between calls.  meta[LORA_PLAN_META] = tokens, pages taken, pages given back,
 * requests refused, invalid entries, free pages after, 0, 0.  No output may overlap
 * another vector, past_lens and seq_lens among them (cursor_out and cursor apart).
 * Invalid entries: a negative past, new_lens below -1 (the request counts as having no
 * tokens) or past + new above max_pages * page_size (its tokens get slot -1, its length
 * 0); a page id outside [0, num_pages) in the ring or in an existing part of a row (the
 * tokens there get slot -1; it is given back as -1); each token beyond num_tokens (not
 * written, and query_start stops at num_tokens).
 * block_table: [num_seqs] rows of max_pages ids, row stride ld_table.  One launch on
 * `stream` of `device`.  Two calls that share a cursor must not overlap in time.
 * Errors: INVALID_ARG (a NULL pointer: past_lens, new_lens, seq_lens, block_table may be
 * NULL with num_seqs = 0, positions and slots with num_tokens = 0, meta always), SHAPE
 * (num_seqs outside [0, LORA_MAX_SEQS], num_tokens < 0, page_size, num_pages < 1 or too
 * many, max_pages < 1, ld_table < max_pages, max_pages * page_size above 2^31 - 1).
 */
lora_status lora_page_plan(int device, const int32_t* past_lens, const int32_t* new_lens, int num_seqs, int num_tokens,
                           int page_size, int num_pages, int32_t* free_pages, int32_t* cursor, int32_t* cursor_out,
                           int32_t* block_table, int ld_table, int max_pages, int32_t* seq_lens, int32_t* query_start,
                           int32_t* positions, int32_t* slots, int32_t* meta, hipStream_t stream);

/*
 * Rotary frequencies, radians a position, of rot_dim / 2 pairs: f_i = base^(-2 i /
 * rot_dim), then scaled for contexts longer than the original_len that the weights were
 * trained on:
 *   LORA_ROPE_PLAIN       f_i
 *   LORA_ROPE_LINEAR      f_i / factor (positions interpolated)
 *   LORA_ROPE_WAVELENGTH  turns n = original_len f_i / (2 pi): f_i where n >= high, f_i /
 *                         factor where n <= low, in between w f_i + (1 - w) f_i / factor,
 *                         w = (n - low) / (high - low)
 *   LORA_ROPE_DIM         the same blend, linear in the pair's index between the pairs
 *                         that make `high` and `low` turns over original_len: i_n = rot_dim
 *                         ln(original_len / (2 pi n)) / (2 ln base), lo = floor(i_high), hi
 *                         = ceil(i_low), both kept in [0, rot_dim - 1], w = 1 - clamp((i - lo) /
 *                         max(hi - lo, 0.001), 0, 1)
 * Pure host function, in double.  Errors: freqs NULL, base <= 1, or (scaled) factor < 1, not finite
 * -> INVALID_ARG; for the last two original_len <= 0 or not 0 < low < high ->
 * INVALID_ARG; rot_dim not an even number in [2, LORA_MAX_HEAD_DIM], unknown scaling -> SHAPE.
 */
typedef enum { LORA_ROPE_PLAIN = 0, LORA_ROPE_LINEAR = 1, LORA_ROPE_WAVELENGTH = 2, LORA_ROPE_DIM = 3 } lora_rope_scaling;
lora_status lora_rotary_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double low,
                                    double high, double* freqs);

/*
 * A rotary embedding of the first rot_dim values of a head: pair i turns by position *
 * freqs[i] and is multiplied by amplitude.  Pairs are (2i, 2i + 1) when `interleaved`, else (i, i
 * + rot_dim / 2); values past rot_dim pass unchanged.  freqs: host array of rot_dim / 2
 * values, read during the call (lora_rotary_frequencies, or any others).  Errors: out or
 * freqs NULL, a frequency or the amplitude not finite -> INVALID_ARG; rot_dim as above -> SHAPE;
 * NO_DEVICE / OOM.
 */
typedef struct lora_rotary lora_rotary;
lora_status lora_rotary_create(lora_rotary** out, int device, int rot_dim, int interleaved, const double* freqs,
                               double amplitude);
lora_status lora_rotary_destroy(lora_rotary* rotary);

/*
 * Rotary positions on a step's packed q/k/v rows, and the keys and values into the cache:
 * row t of qkv is [num_q_heads + 2 num_heads][head_dim] (q heads, k heads, v heads; row
 * stride ldqkv).  q_out[t] (row stride ldq) = the turned q heads, k[slot] = the turned k
 * heads, v[slot] = the v heads.  Angles are formed in 64 bits (good to 2^-50 of a turn while
 * position * freqs[i] is below 2^50 turns; 16-bit rows then take 2^-26), the turn in fp32, one rounding
 * to the stored type; an e4m3 cache stores x / scale, clamped to [-448, 448], NaN kept.
 * q_out may be qkv itself (the turn in place; else they must not overlap).  A slot outside
 * the cache stores nothing; which of two tokens with one slot is kept is not defined.
 * dtype (of qkv and q_out): LORA_BF16 with a bf16 or e4m3 cache, LORA_F32 with an fp32
 * one (else DTYPE).  Errors: INVALID_ARG (NULL, or a scale that is not positive and finite), SHAPE (num_tokens < 0,
 * num_q_heads not a positive multiple of num_heads, rot_dim > head_dim, strides below the rows' width, the cache's
 * rules), ALIGN (ldqkv, ldq multiples of 8, pointers 16-byte aligned).
 */
lora_status lora_rotary_append(const lora_rotary* rotary, const void* qkv, int ldqkv, lora_dtype dtype, int num_q_heads,
                               const int32_t* positions, const int32_t* slots, int num_tokens, void* q_out, int ldq,
                               const lora_kv_cache* cache, hipStream_t stream);

/*
 * Attention of a step's tokens over the paged cache.  The object owns the workspace for
 * max_seqs sequences and max_tokens new tokens of num_q_heads query and num_kv_heads key/value
 * heads: partial results of long sequences, which several workgroups share (256 KiB a head_dim
 * value on 256 compute units, 32 MiB at 128, whatever the other sizes), and the counters
 * that tell the last of them to join.
 * Errors of create: out NULL -> INVALID_ARG; max_seqs outside [1, LORA_MAX_SEQS],
 * max_tokens outside [1, 2^24] or, times num_q_heads / num_kv_heads, above 2^30, num_kv_heads outside
 * [1, 1024], num_q_heads not a multiple of it or above 1024, head_dim above
 * LORA_MAX_HEAD_DIM -> SHAPE; head_dim not a positive multiple of 16 -> ALIGN;
 * NO_DEVICE / OOM.
 */
typedef struct lora_attention lora_attention;
lora_status lora_attention_create(lora_attention** out, int device, int max_seqs, int max_tokens, int num_q_heads,
                                  int num_kv_heads, int head_dim);
lora_status lora_attention_destroy(lora_attention* attention);

/*
 * out[t][h] = sum_j softmax_j(scale q[t][h] . k_j) v_j over the cached tokens j that token
 * t sees: token t is the i-th of the n = query_start[r+1] - query_start[r] new tokens of
 * its sequence r and stands at position P = seq_lens[r] - n + i; it sees j <= P, and with
 * window > 0 only j > P - window.  (The new tokens' own keys and values are in the cache:
 * lora_rotary_append.)  Query head h reads kv head h / (num_q_heads / num_heads).  lse[t][h]
 * (fp32, may be NULL) = ln sum_j exp(scale q . k_j).  A token that sees nothing (length
 * 0, absent pages) gets zeros and lse = -inf, as does one whose every score is -inf; a NaN score
 * makes its token's head NaN in out and lse.  What lies in the cache at unseen places,
 * infinities and NaN included, has no effect.
 * q, out: [num_tokens][num_q_heads * head_dim], row strides ldq and ldo, dtype as for
 * lora_rotary_append (out has q's dtype).  Sums, maxima and products accumulate in fp32,
 * with one rounding to out.  The result is bitwise the same on every call.  Rows of no sequence are left as
 * they were; seq_lens outside [0, max_pages * page_size] are taken as the nearer bound,
 * query_start outside [0, num_tokens] likewise; a sequence that ends before it starts has
 * no tokens (starts that overlap so much that the work passes 2^30 steps: nothing is
 * written).  One launch on `stream`.  Two calls on one object must not overlap in time.
 * Errors: INVALID_ARG (NULL pointer, scale not finite, window < 0), SHAPE (heads or
 * head_dim not the object's, ld_table < max_pages, strides below the rows' width,
 * max_pages < 1, the cache's rules, num_tokens * num_q_heads of 2^30 and more that need 2^30
 * steps), CAPACITY (num_seqs or num_tokens above the object's), DTYPE, ALIGN.
 */
lora_status lora_paged_attention(const lora_attention* attention, const void* q, int ldq, lora_dtype dtype,
                                 const lora_kv_cache* cache, const int32_t* block_table, int ld_table, int max_pages,
                                 const int32_t* seq_lens, const int32_t* query_start, int num_seqs, int num_tokens,
                                 float scale, int window, void* out, int ldo, float* lse, hipStream_t stream);

/*
 * Index checks (diagnostics): a library built with -DRAXLORA_DEBUG (build.py
 * --debug: libraxlora_debug.so) checks, in its kernels, every index it takes from
 * memory (token ids, slots, sorted positions, workspace rows) against its range; a
 * failed check is counted and the access goes to index 0 instead, so a wrong index
 * shows as a count rather than a fault.  (The page plan, rotary append and paged attention
 * take wrong words as their contracts say, in every build, and count nothing here.)  *enabled = 1 in such a build, 0 otherwise
 * (where *faults is always 0); *faults = the checks failed on the current device since
 * the last reset (all kernels of the library, after the work enqueued so far has
 * finished: the call synchronises the device); reset != 0 clears the count.
 * Errors: NULL -> INVALID_ARG; a HIP error reading the counts -> HIP.
 */
lora_status lora_index_checks(int* enabled, unsigned long long* faults, int reset);

/*
 * Bandwidth probe (diagnostics): the rate this GPU's memory gives a plain streaming
 * kernel, the ceiling against which the LoRA kernels' traffic is read.  ratio <= 0:
 * read read_bytes from src (device, 16-byte aligned), 16 bytes per lane, and write
 * one 4-byte word per thread into dst (needs dst_bytes >= 4 MiB).  ratio > 0: read
 * read_bytes and write read_bytes / ratio bytes to dst (each 16-byte chunk of dst is
 * the xor of `ratio` chunks of src).  One launch, enqueued on `stream`.
 * Errors: NULL -> INVALID_ARG; alignment -> ALIGN; sizes -> SHAPE.
 */
lora_status lora_bandwidth_probe(const void* src, uint64_t read_bytes, void* dst, uint64_t dst_bytes, int ratio,
                                 hipStream_t stream);

/*
 * Kernel timing (diagnostics).  While enabled (process-wide), every kernel that
 * the routing, shrink, expand, linear, embedding, page plan, rotary append and paged
 * attention calls launch is started
 * with hipExtLaunchKernel and a pair of events stamped at that kernel's own start
 * and end, on the stream it runs on.  lora_timing_report waits for the recorded
 * events, writes per kernel id (0 routing, 1 shrink, 2 expand, 3 finish_u: the
 * pass of lora_shrink that adds the k-split partial sums into the caller's u,
 * 4 gather: the embedding rows of lora_embedding, 5 page_plan, 6 rotary_append, 7
 * attention; the shrink and expand launches cover both short and long segments) the summed milliseconds and the
 * number of launches into total_ms[0..max_kernels) and launches[0..max_kernels), and
 * clears the record.  lora_timing_kernel_name gives the name of an id ("" if none).
 * Errors: INVALID_ARG for NULL arrays with max_kernels > 0; HIP if an event fails.
 */
lora_status lora_timing_enable(int on);
lora_status lora_timing_report(double* total_ms, int* launches, int max_kernels);
const char* lora_timing_kernel_name(int kernel);

#ifdef __cplusplus
}
#endif

#endif /* RAXLORA_H */
