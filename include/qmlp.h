/*
 * qmlp.h -- C ABI of libqmlp.so, the weight-quantized SwiGLU MLP for GB300
 * (sm_103a). Plain pointers and sizes only.
 *
 * The operation (vllm.cpp issue "tp>1 fp8w tail-MLP shard host-dequantizes
 * every layer", "Proposed fix"):
 *   act[m, i] = bf16( SiLU(sigma_g[i] * sum_k x[m,k] Wg[i,k]) *
 *                          (sigma_u[i] * sum_k x[m,k] Wu[i,k]) )
 *   out[m, o] = bf16( sigma_d[o] * sum_i act[m,i] Wd[o,i] )
 * with the weights dequantized on the fly from resident packed bytes:
 *   NVFP4 (Qwen3.8-27B-NVFP4, "NVFP4 numerics as implemented"):
 *     W[n,k] = E2M1(nibble) * E4M3(scale[n, k/16]); byte k/2 of row n holds k
 *     in its low nibble when k is even; sigma = fp32(1 / global_scale).
 *   FP8 per-channel W8A16 (vllm.cpp issue, "Mechanism on the tp>1 path"):
 *     W[n,k] = e4m3fn(w[n,k]); sigma[n] = scale[n] (fp32).
 * SiLU(t) = t / (1 + exp(-t)). Accumulation is fp32 on the GPU; act is
 * rounded to bf16 before the down projection; out is bf16.
 *
 * Conventions for every entry point:
 *  - A status is returned; no entry point falls back to a CPU computation and
 *    none aborts the process. QMLP_OK is 0.
 *  - "device" pointers are CUDA device addresses on the current device;
 *    "host" pointers are host addresses (pinned or pageable).
 *  - All device pointers passed to forward calls must be 16-byte aligned.
 *  - Streams: a CUstream/cudaStream_t value; NULL means the legacy default
 *    stream. Forward calls only enqueue work (except *_host, which waits).
 *  - One handle serves one stream at a time: its workspace is shared by all
 *    calls on it.
 *  - One GPU per process: the kernels' shared-memory attributes are set on
 *    the first launch of each kernel in the process, for the device current
 *    then; handles on a second device of the same process get QMLP_ERR_CUDA
 *    from the launches that need a large shared-memory window. Run one
 *    process per GPU.
 *  - Validation happens before any launch; a rejected call launches nothing.
 *  - Launch failures return QMLP_ERR_CUDA. Errors raised asynchronously by a
 *    kernel surface on a later call or on the caller's synchronization; a
 *    kernel that gives up a bounded wait records it in the handle, and
 *    qmlp_check / qmlp_moe_check return QMLP_ERR_DEVICE_TIMEOUT.
 */
#ifndef QMLP_H
#define QMLP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* qmlp_stream_t; /* identical to cudaStream_t */

typedef enum {
    QMLP_OK = 0,
    QMLP_ERR_INVALID_ARG = 1,     /* null pointer, bad enum, bad count     */
    QMLP_ERR_ALIGNMENT = 2,       /* a device pointer not 16-byte aligned  */
    QMLP_ERR_ALIAS = 3,           /* output overlaps an input or workspace */
    QMLP_ERR_SHAPE = 4,           /* K, I, M, E or topk outside the limits */
    QMLP_ERR_UNSUPPORTED_ARCH = 5,/* device is not compute capability 10.3 */
    QMLP_ERR_OOM = 6,             /* device allocation failed at create    */
    QMLP_ERR_CUDA = 7,            /* a CUDA runtime call or launch failed  */
    QMLP_ERR_DEVICE_TIMEOUT = 8,  /* a kernel gave up a bounded wait       */
    QMLP_ERR_DEVICE_BOUNDS = 9    /* an index check failed (checking build) */
} qmlp_status;

typedef enum { QMLP_FMT_NVFP4 = 1, QMLP_FMT_FP8_PC = 2 } qmlp_format;
typedef enum { QMLP_DT_BF16 = 1, QMLP_DT_FP16 = 2, QMLP_DT_FP32 = 3 } qmlp_dtype;
typedef enum { QMLP_META_3B = 3, QMLP_META_4B = 4 } qmlp_meta;
/* Kernel family used by a forward call: AUTO picks the decode (GEMV) family
 * for small token counts and the tensor-core GEMM above. GEMM_PAIR is the
 * tensor-core GEMM on CTA pairs (tcgen05.mma.cta_group::2: two SMs share a
 * 256-token x 256-row tile, each decoding half of its weight rows) for
 * M >= 256; AUTO does not choose it (the single-CTA GEMM measured faster on
 * the 27B-class prefill shape). GEMM_DQ is the dequantise-once GEMM: each
 * projection is first decoded, once per call, into bf16 tiles in buffers
 * the handle holds (6 I K bytes, allocated by qmlp_create when max_M >=
 * 768, with a CUDA stream and two events of the handle's own: in a whole
 * forward the down projection is decoded on that stream while the gate/up
 * GEMM runs, forked from and joined back to the caller's stream with
 * events, so the call stays stream-ordered and can be captured in a CUDA
 * graph), and the tensor-core GEMM then multiplies those tiles with the bf16
 * activations as given (no per-token prescale), with no decoding in its main
 * loop (on CTA pairs from M = 256, as GEMM_PAIR, each CTA loading
 * half of every decoded tile); AUTO takes it from M = 768 on. The products
 * are of the same exact weight values either way. */
typedef enum {
    QMLP_PATH_AUTO = 0,
    QMLP_PATH_GEMV = 1,
    QMLP_PATH_GEMM = 2,
    QMLP_PATH_GEMM_PAIR = 3,
    QMLP_PATH_GEMM_DQ = 4
} qmlp_path;

/* One projection [N, K] as the checkpoint stores it. Pointers may be host or
 * device memory; they are only read during qmlp_create.
 *  NVFP4: w     = u8 [N, K/2], two E2M1 codes per byte, low nibble = even k
 *         scale = u8 [N, K/16], E4M3 group scales
 *         global_scale = fp32; the dequantization factor is 1/global_scale
 *  FP8:   w     = u8 [N, K], e4m3fn codes
 *         scale = fp32 [N], per output channel; global_scale is ignored */
typedef struct {
    const uint8_t* w;
    const void* scale;
    float global_scale;
} qmlp_proj;

/* Dense MLP description: hidden size K, intermediate size I, largest token
 * count max_M any forward call will use. gate/up are [I, K], down is [K, I].
 * Limits: K % 16 == 0, I % 16 == 0, 16 <= K, I <= 65536, 1 <= max_M <= 65536. */
typedef struct {
    qmlp_format fmt;
    int K;
    int I;
    int max_M;
    qmlp_proj gate;
    qmlp_proj up;
    qmlp_proj down;
} qmlp_desc;

typedef struct qmlp_s qmlp_t;

/* Create a dense MLP handle. Copies the weights into memory the handle owns,
 * reordered for the kernels (create-time repack; the weight bytes are kept
 * packed, never expanded), computes sigma = fp32(1/global) for NVFP4, and
 * allocates the forward workspace for max_M tokens. Synchronizes `stream`
 * before returning, so the caller may free its buffers afterwards.
 * Errors: INVALID_ARG (null/unknown fmt), SHAPE, UNSUPPORTED_ARCH, OOM, CUDA.
 * On error *out is NULL and nothing is leaked. */
qmlp_status qmlp_create(qmlp_t** out, const qmlp_desc* desc, qmlp_stream_t stream);

/* Free every buffer owned by the handle (waits for its pending work). NULL is
 * a no-op. */
void qmlp_destroy(qmlp_t* h);

/* The MLP block (see the top of this file) on M tokens.
 *  x   = device bf16 [M, K] (row-major), read only
 *  out = device bf16 [M, K] (row-major), written
 * Allocates nothing; enqueues its kernels on `stream`.
 * Errors: INVALID_ARG (null), ALIGNMENT (x/out not 16-B aligned), ALIAS (out
 * overlaps x), SHAPE (M < 1 or M > max_M), CUDA. */
qmlp_status qmlp_forward(qmlp_t* h, const void* x, int M, void* out, qmlp_stream_t stream);

/* As qmlp_forward, forcing a kernel family. GEMM, GEMM_PAIR and GEMM_DQ
 * require a handle whose max_M reaches the GEMM threshold (and K % 256,
 * I % 128 == 0); GEMM_PAIR also M >= 256; GEMM_DQ a handle created with
 * max_M >= 768 (any M up to max_M; the handle's buffers and side stream,
 * see qmlp_path). Otherwise SHAPE. */
qmlp_status qmlp_forward_path(qmlp_t* h, qmlp_path path, const void* x, int M, void* out,
                              qmlp_stream_t stream);

/* One half of the forward, for callers that overlap or time the two
 * projections separately (stage 0 followed by stage 1 equals qmlp_forward):
 *  stage 0: act = SwiGLU(x) into the handle's workspace; x = device bf16
 *           [M, K]; out must be NULL.
 *  stage 1: out = the down projection of the workspace act written by the
 *           previous stage-0 call with the same M; x must be NULL; out =
 *           device bf16 [M, K].
 * Errors: as qmlp_forward_path (INVALID_ARG for a wrong NULL pattern). */
qmlp_status qmlp_forward_stage(qmlp_t* h, int stage, qmlp_path path, const void* x, int M, void* out,
                               qmlp_stream_t stream);

/* End-to-end call from host buffers (x: host bf16 [M, K], out: host bf16
 * [M, K]); returns after `stream` has finished. Pinned (device-mapped) host
 * buffers, 16-byte aligned and not overlapping: one small kernel copies x
 * over the coherent CPU-GPU link into the handle's device stage, and the
 * kernels write the output in place into the host buffer. Otherwise x is
 * copied to the staging buffer and the result copied back by the copy engine
 * (pageable memory works but serializes the copies).
 * Errors: as qmlp_forward. */
qmlp_status qmlp_forward_host(qmlp_t* h, const void* x_host, int M, void* out_host,
                              qmlp_stream_t stream);

/* Forward that also returns the intermediate: act = device bf16 [M, I]
 * (the values the down projection consumed). Errors: as qmlp_forward_path,
 * plus ALIAS if act overlaps x or out. */
qmlp_status qmlp_forward_debug(qmlp_t* h, qmlp_path path, const void* x, int M, void* act,
                               void* out, qmlp_stream_t stream);

/* One projection in isolation, through the same kernels, with no scale
 * factor applied (no 1/global, no per-channel scale) and fp32 output:
 *   y[m, n] = sum_k x[m,k] * W[n,k],  W = E2M1*E4M3 (NVFP4) or e4m3fn (FP8)
 *  which = 0 gate, 1 up (x is [M, K]); 2 down (x is [M, I]).
 *  x = device bf16 [M, Kp], y = device fp32 [M, N].
 * With a one-hot x this returns single decoded weights exactly.
 * Errors: as qmlp_forward_path. */
qmlp_status qmlp_debug_project(qmlp_t* h, int which, qmlp_path path, const void* x, int M,
                               float* y, qmlp_stream_t stream);

/* CTAs of the decode kernel that partitions the intermediate dimension (each
 * CTA computes gate/up for its slice of I and the down projection over that
 * slice; the partial outputs are added in a fixed order -- after a grid
 * barrier inside the kernel for one NVFP4 token, else by a small reduce
 * kernel launched after it). 0 when the shape has no such partition on this
 * device (the stream-K kernel is used instead). Used for M <= 8; the tensor-
 * core GEMM takes M >= 9 when this partition exists.
 * The one-token NVFP4 schedule waits (bounded, 2 s) at that grid barrier for
 * all its CTAs, one per SM: if kernels of other streams hold SMs for longer,
 * the call gives up, its output is not valid and qmlp_check returns
 * QMLP_ERR_DEVICE_TIMEOUT. */
int qmlp_decode_ctas(qmlp_t* h);

/* The I-partitioned decode kernel (see qmlp_decode_ctas) with its raw
 * epilogues, for tests that check its own weight layouts bit for bit:
 *  x      = device bf16 [M, K]; act_in = device bf16 [M, I] (the down
 *           projection consumes act_in instead of the SwiGLU of x)
 *  g, u   = device fp32 [M, I]: sum_k x[m,k] W[i,k] of gate / up, no factor
 *  out_f32= device fp32 [M, K]: sum_i act_in[m,i] Wd[o,i], no factor
 * With one-hot x (act_in) every value is a single decoded weight exactly.
 * 1 <= M <= 8. Errors: INVALID_ARG, ALIGNMENT, ALIAS, SHAPE (no partition for
 * this shape, or M out of range), CUDA. */
qmlp_status qmlp_debug_split(qmlp_t* h, const void* x, const void* act_in, int M, float* g, float* u,
                             float* out_f32, qmlp_stream_t stream);

/* Error-path tests only: every later launch of this handle's decode
 * (I-partitioned) and tensor-core GEMM kernels gives up a wait on another
 * role or CTA after limit_ns (0: the default of 2 s), and, when
 * withhold_last_step is non-zero, their producers never issue their last
 * weight step, so those waits run out: the kernels record it, leave without
 * a fault, and qmlp_check returns QMLP_ERR_DEVICE_TIMEOUT. Errors: INVALID_ARG. */
qmlp_status qmlp_debug_set_wait(qmlp_t* h, uint64_t limit_ns, int withhold_last_step);

/*
 * Index checks. A library built with -DQMLP_DEBUG_BOUNDS (libqmlp_bounds.so;
 * the default build compiles the checks away) checks, in every kernel, the
 * index of each global access whose address comes from layout arithmetic or
 * runtime data (weight-bank blocks and records, partial buffers, outputs,
 * route lists, the adapters' slots, tiles and rows) against the size of its
 * buffer, as far as the library knows it. A failed check never traps:
 * the kernel records the first one and skips the access (a load reads zero,
 * a store is dropped, a bulk copy is taken from the start of its buffer), so
 * the call's outputs are then invalid but the device stays usable. This
 * build stands in for a memory checker where none can run.
 */
/* 1 for a checking build, else 0. */
int qmlp_debug_bounds_enabled(void);

/* Synchronize the device, then report and clear the first failed index
 * check of any kernel since the last call: *site = the check's number
 * (per source file: 1-9 decode kernel, 11-19 tensor-core GEMM, 21-29 stream-K
 * and split-K decode kernels, 31-39 one-token routed experts, 41-49 grouped
 * routed experts, 51-59 tensor-parallel combine, 61-69 low-rank products,
 * 71-79 AdamW, 81-89 norms, 91-99 linear,
 * 101-109 mixture-of-experts layer) and *index = the checked
 * index (low 48 bits), or 0 and 0. Returns OK, DEVICE_BOUNDS (a check
 * failed), INVALID_ARG (a NULL pointer) or CUDA. A default build always
 * reports OK. */
qmlp_status qmlp_debug_bounds(int* site, unsigned long long* index);

/* Checking builds, tests only: from now on the decode kernel's checks allow
 * only the first gate_up_bank_bytes bytes of each of its gate and up record
 * banks (0: the whole bank), so its later weight steps fail their check --
 * the copies are then taken from the bank's start, which exists -- and
 * qmlp_debug_bounds reports site 1. Errors: INVALID_ARG (NULL handle, or a
 * default build). */
qmlp_status qmlp_debug_bounds_limit(qmlp_t* h, size_t gate_up_bank_bytes);

/*
 * Tensor-parallel shard over the intermediate dimension (vllm.cpp issue "tp>1
 * fp8w tail-MLP shard host-dequantizes every layer", "Proposed fix"): rank r
 * of n keeps gate/up rows [r I/n, (r+1) I/n) and the same columns of down, and
 * one sum over the ranks' [M, K] partials gives the layer's output.
 */
/* Create rank `rank`'s shard from the description of the WHOLE layer (the
 * same pointers and sizes qmlp_create takes; only the shard's rows and columns
 * are read). The handle's intermediate size is I / nranks; forward on it
 * returns bf16(sigma_d x its own partial). Limits: as qmlp_create, plus
 * 0 <= rank < nranks, I % nranks == 0, (I / nranks) % 16 == 0.
 * Errors: as qmlp_create (INVALID_ARG for a bad rank). */
qmlp_status qmlp_create_shard(qmlp_t** out, const qmlp_desc* desc, int rank, int nranks, qmlp_stream_t stream);

/* This shard's partial: partial[m, o] = sum over the shard's i of act[m,i]
 * Wd[o,i] in fp32 with no down factor (act = bf16 SwiGLU, as qmlp_forward).
 *  x = device bf16 [M, K]; partial = device fp32 [M, K].
 * Errors: as qmlp_forward. */
qmlp_status qmlp_forward_partial(qmlp_t* h, const void* x, int M, float* partial, qmlp_stream_t stream);

/* The exchange step after the partials are gathered (an all-gather of the
 * [M, K] fp32 partials, rank-major): out[m, o] = bf16( sigma_d[o] * sum over
 * r = 0..nranks-1 in rank order of partials[r][m][o] ). The order is fixed,
 * so every rank computes the same bytes.
 *  partials = device fp32 [nranks][M][K]; out = device bf16 [M, K]
 * nranks must equal the handle's. Errors: INVALID_ARG, SHAPE, ALIGNMENT,
 * ALIAS, CUDA. */
qmlp_status qmlp_shard_combine(qmlp_t* h, const float* partials, int nranks, int M, void* out,
                               qmlp_stream_t stream);

/* Rank, rank count and intermediate size of a handle (0, 1 and I for a
 * whole-layer handle). Returns 0 for a NULL handle, else 1. */
int qmlp_shard_info(qmlp_t* h, int* rank, int* nranks, int* I_shard);

/* Synchronize `stream` and report (then clear) a bounded-wait give-up
 * recorded by this handle's kernels: OK or DEVICE_TIMEOUT (CUDA on a sticky
 * device error). */
qmlp_status qmlp_check(qmlp_t* h, qmlp_stream_t stream);

/*
 * Routed-expert AWQ int4 group-32 MLP, one token (1Cat-vLLM PR "[Kernel][SM70]
 * Add native-g32 AWQ QPN M1 operator", "What it does"):
 *   for each route r in router order with 0 <= ids[r] < E:
 *     h      = x . W13[ids[r]]^T             (fp32 accumulation, N = 2I)
 *     g, u   = fp16(h[:I]), fp16(h[I:])
 *     act[r] = fp16(SiLU(g) * u)
 *     y[r]   = fp16(act[r] . W2[ids[r]]^T)   (fp32 accumulation, N = K)
 *   out = fp16( sum over valid r, in router order, of router_w[r] * y[r] )
 *         (fp32 accumulation, no atomics)
 * Weights: W[e, n, k] = half_fma(q, scale, bias): q is the u4 code (low nibble
 * = even k), one metadata record per (e, n, k/32): 4-byte {fp16 scale, fp16
 * bias} or 3-byte {fp16 scale, u8 zero} with bias = half(-zero*scale); records
 * are little-endian, scale first. Invalid ids (< 0 or >= E) contribute zero;
 * duplicate valid ids are separate routes with their own router weights.
 */
typedef struct {
    int E;            /* experts                     */
    int K;            /* hidden size (W13 in, W2 out) */
    int I;            /* intermediate per expert     */
    qmlp_meta meta;   /* 3- or 4-byte records        */
    const uint8_t* w13;       /* [E, 2I, K/2]              host or device */
    const uint8_t* w13_meta;  /* [E, 2I, K/32] x meta bytes              */
    const uint8_t* w2;        /* [E, K, I/2]                             */
    const uint8_t* w2_meta;   /* [E, K, I/32] x meta bytes               */
} qmlp_moe_desc;

typedef struct qmlp_moe_s qmlp_moe_t;

/* Create a routed-expert handle: copies the banks into handle-owned device
 * memory (reordered for the kernels, same bytes). Limits: K % 64 == 0,
 * I % 32 == 0, 32 <= I <= 1024, 64 <= K <= 16384, 1 <= E. Synchronizes.
 * Errors: INVALID_ARG, SHAPE, UNSUPPORTED_ARCH, OOM, CUDA. */
qmlp_status qmlp_moe_create(qmlp_moe_t** out, const qmlp_moe_desc* desc, qmlp_stream_t stream);
void qmlp_moe_destroy(qmlp_moe_t* h);

/* The routed-expert step above for one token.
 *  x          = device [K], bf16 or fp16 per xdt
 *  expert_ids = device int32 [topk]  (read on the device: may change between
 *               CUDA-graph replays)
 *  router_w   = device fp32 [topk]
 *  out        = device fp16 [K]
 * 1 <= topk <= 16. Allocates nothing; graph-capturable.
 * Errors: INVALID_ARG, ALIGNMENT, ALIAS (out overlaps x, ids or router_w),
 * SHAPE, CUDA. */
qmlp_status qmlp_moe_m1_forward(qmlp_moe_t* h, const void* x, qmlp_dtype xdt,
                                const int32_t* expert_ids, const float* router_w, int topk,
                                void* out, qmlp_stream_t stream);

/* As qmlp_moe_m1_forward, also writing the per-stage fp16 tensors (device):
 *  gu [topk, 2I], act [topk, I], y [topk, K]; rows of invalid routes are not
 *  written. Any of gu/act/y may be NULL. */
qmlp_status qmlp_moe_debug_stages(qmlp_moe_t* h, const void* x, qmlp_dtype xdt,
                                  const int32_t* expert_ids, const float* router_w, int topk,
                                  void* out, void* gu, void* act, void* y, qmlp_stream_t stream);

/* Reserve the workspace of multi-token calls: after this, qmlp_moe_forward
 * accepts 1 <= M <= max_tokens (routes = M * topk <= max_tokens * 16). Sizes
 * the handle-owned fp16 intermediates for max_tokens * 16 routes (act [.., I],
 * y [.., K]) plus the route and group lists; a larger later reservation adds
 * a larger workspace (the old one is freed by destroy). Allocates and
 * synchronizes the stream: call it before capturing graphs. A handle starts
 * with max_tokens = 1. Limits: K <= 8192 and E <= 8192 for M > 1.
 * Errors: INVALID_ARG, SHAPE, OOM, CUDA. */
qmlp_status qmlp_moe_reserve(qmlp_moe_t* h, int max_tokens, qmlp_stream_t stream);

/* The routed-expert step for M tokens, every token independently exactly as
 * qmlp_moe_m1_forward computes it (the source PR defines the one-token
 * operator; tokens do not interact):
 *  x          = device [M, K], bf16 or fp16 per xdt (row-major)
 *  expert_ids = device int32 [M, topk] (token t's routes in router order)
 *  router_w   = device fp32 [M, topk]
 *  out        = device fp16 [M, K]
 * M == 1 runs the one-token kernels. For M > 1 the valid routes of all tokens
 * are sorted by expert on the device and tokens that share an expert share
 * its weight reads (groups of up to 16 routes); results do not depend on the
 * grouping and are the same bytes every call. 1 <= topk <= 16,
 * 1 <= M <= the reserved max_tokens. Allocates nothing; graph-capturable.
 * Errors: INVALID_ARG, ALIGNMENT, ALIAS (out overlaps x, ids or router_w),
 * SHAPE, CUDA. */
qmlp_status qmlp_moe_forward(qmlp_moe_t* h, const void* x, qmlp_dtype xdt, const int32_t* expert_ids,
                             const float* router_w, int topk, int M, void* out, qmlp_stream_t stream);

qmlp_status qmlp_moe_check(qmlp_moe_t* h, qmlp_stream_t stream);

/* The routed-expert step of qmlp_moe_m1_forward without a handle, for callers
 * that cannot allocate device memory when they run it (an allocator-owning
 * runtime that forbids foreign allocations, or code whose device memory is
 * fixed after warm-up). It allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library call. The source pages have no counterpart; this is a
 * library convenience over the same kernels.
 *  banks = the expert banks as DEVICE pointers in the checkpoint layout of
 *          qmlp_moe_desc (read directly, never copied), w13/w2 16-byte aligned
 *  x, expert_ids, router_w, out: as qmlp_moe_m1_forward.
 * Scratch: the fp16 SwiGLU intermediate lives in one file-scope device array
 * of 16 x 1024 fp16 (32 KiB) that every GPU loading the library keeps until
 * exit; hence topk <= 16 and I <= 1024, larger sizes return QMLP_ERR_SHAPE.
 * The first call on a device looks up the array's device address (once per
 * device, on the current device); make that first call before any stream
 * capture. All calls share the array, which keeps the last call's contents
 * (no call needs it cleared: each route's row is written before it is read);
 * calls whose kernels overlap on the GPU (other streams, or other threads)
 * race on it and must be serialized by the caller. The looked-up address is
 * kept for the life of the process: resetting the device (cudaDeviceReset,
 * or tearing down and recreating its primary context) while the library
 * stays loaded is not supported for this entry point.
 * Errors: INVALID_ARG, ALIGNMENT, ALIAS (out overlaps x, ids, router_w or any
 * of the four banks), SHAPE, UNSUPPORTED_ARCH, CUDA. */
qmlp_status qmlp_moe_m1_forward_noalloc(const qmlp_moe_desc* banks, const void* x, qmlp_dtype xdt,
                                        const int32_t* expert_ids, const float* router_w, int topk,
                                        void* out, qmlp_stream_t stream);

/*
 * Low-rank adapters (LoRA) of many requests at once beside the dense MLP. An
 * adapter of a projection W [N, D] is A [r, D], B [N, r] and a factor c; the
 * projection of z becomes  W z + c B (A z). Every token names the slot of its
 * adapter, so requests with different adapters share one call and one read of
 * the quantized weights:
 *   g = sigma_g x Wg^T + c B_g A_g x   (u alike),  act = bf16(SiLU(g) u)
 *   out = bf16( sigma_d act Wd^T + c B_d A_d act )
 * with each token's own A, B and c. Sums are fp32, and c A z is held as fp32.
 * Values of an adapter that are not finite reach the tokens that name it (as Inf
 * or NaN) and no others.
 */
/* One adapter: bf16 device arrays, any alignment of 2 bytes, any rank from 1.
 * A projection that is not adapted has both its pointers NULL. */
typedef struct {
    int rank;
    float scale; /* c: alpha / r */
    const void* gate_a; /* [r, K] */
    const void* gate_b; /* [I, r] */
    const void* up_a;   /* [r, K] */
    const void* up_b;   /* [I, r] */
    const void* down_a; /* [r, I] */
    const void* down_b; /* [K, r] */
} qmlp_adapter;

typedef struct qmlp_lora_s qmlp_lora_t;

/* Make `slots` empty adapter slots of ranks up to max_rank for the handle h,
 * which must outlive them. Holds slots * 3 (K + I) * R bf16 values, R = 16, 32
 * or 64 (max_rank rounded up), 4 max(2 I, K) bytes a token of h's max_M for the
 * adapters' terms, and where h has the dequantise-once GEMM (and all its factors
 * are at least 2^-60) the adapters once more as images for it (two to seven times
 * the padded copies, up to 4 GiB; past that calls do without) and 2 K bytes a
 * token. The slots share h's workspace: calls on them and on h go on one stream
 * at a time.
 * On a shard's handle (qmlp_create_shard) an adapter has the shard's rows of the
 * gate and up B and its columns of the down A, and out is the rank's own term in
 * bf16, as qmlp_forward's.
 * Limits: 1 <= slots <= 1024, 1 <= max_rank <= 64. Synchronizes `stream`.
 * Errors: INVALID_ARG, SHAPE, OOM, CUDA. */
qmlp_status qmlp_lora_create(qmlp_lora_t** out, qmlp_t* h, int slots, int max_rank, qmlp_stream_t stream);
void qmlp_lora_destroy(qmlp_lora_t* l);

/* Copy an adapter into a slot (in stream order: its arrays may be changed by
 * later work on `stream`). NULL empties the slot.
 * Errors: INVALID_ARG (null handle, slot out of range, one of A and B NULL),
 * SHAPE (rank < 1 or over max_rank), ALIGNMENT (2 bytes), CUDA. */
qmlp_status qmlp_lora_set(qmlp_lora_t* l, int slot, const qmlp_adapter* adapter, qmlp_stream_t stream);

/* The MLP block with each token's adapter.
 *  x   = device bf16 [M, K];  out = device bf16 [M, K]
 *  ids = device int32 [M]: the token's slot; a value outside [0, slots) or an
 *        empty slot: the block without an adapter (read on the device)
 * Allocates nothing; can be captured in a CUDA graph (x and ids may change
 * between replays). 1 <= M <= h's max_M. The same call gives the same bytes.
 * Errors: as qmlp_forward (ALIGNMENT: ids 4 bytes; ALIAS: out overlaps ids). */
qmlp_status qmlp_lora_forward(qmlp_lora_t* l, const void* x, const int32_t* ids, int M, void* out,
                              qmlp_stream_t stream);

/*
 * Training through the dense MLP: its forward, keeping what the backward pass
 * needs, and the backward pass through the frozen quantized weights, with one
 * low-rank adapter or none. With d = the gradient of a loss by ...:
 *   dact = (dout sigma_d) Wd + c (dout B_d) A_d
 *   dg = dact u SiLU'(g),  du = dact SiLU(g)
 *   dx = (dg sigma_g) Wg + (du sigma_u) Wu + c (dg B_g) A_g + c (du B_u) A_u
 *   dB_p = c dy^T (z A_p^T),  dA_p = c (dy B_p)^T z    (z the projection's input, dy its output's gradient)
 * Sums are fp32; g and u are kept in fp32, act in bf16; dg sigma_g and du
 * sigma_u are rounded once to bf16 between the two products. dx and the
 * adapter's gradients are bf16. The sums' order depends on the sizes alone:
 * the same call gives the same bytes.
 */
typedef struct qmlp_train_s qmlp_train_t;

/* Make the training workspace of h (made with max_M >= 768, K % 256 == 0 and
 * I % 128 == 0: the dequantise-once GEMM), which must outlive it, for adapters
 * of ranks up to max_rank (1..64). It shares h's workspace: calls on it and on
 * h go on one stream at a time. Synchronizes `stream`.
 * Errors: INVALID_ARG (null; an NVFP4 factor 1/global under 2^-60), SHAPE,
 * OOM, CUDA. */
qmlp_status qmlp_train_create(qmlp_train_t** out, qmlp_t* h, int max_rank, qmlp_stream_t stream);
void qmlp_train_destroy(qmlp_train_t* t);

/* Bytes of the buffer that a forward of M tokens fills for its backward pass:
 * about 10 I a token (8 I of them for whole groups of 32 tokens) and 2 I more for
 * each of the first 255; 0 where M is out of range. It grows with M: a buffer for
 * M tokens serves any smaller number. */
size_t qmlp_train_saved_bytes(qmlp_train_t* t, int M);

/* The block as qmlp_lora_forward with one adapter for every token (NULL:
 * none), for any 1 <= M <= max_M.
 *  x = device bf16 [M, K];  out = device bf16 [M, K]
 *  saved = device, qmlp_train_saved_bytes(t, M) bytes, 16-byte aligned
 * Allocates nothing; can be captured in a CUDA graph.
 * Errors: as qmlp_forward and qmlp_lora_set. */
qmlp_status qmlp_train_forward(qmlp_train_t* t, const qmlp_adapter* adapter, const void* x, int M, void* out,
                               void* saved, qmlp_stream_t stream);

/* The backward pass of the forward that filled `saved` with the same x, M and
 * adapter (only read).
 *  dout = device bf16 [M, K];  dx = device bf16 [M, K]
 *  grads = where the gradients of the adapter's parts go: bf16, shaped and
 *          packed as the parts, so of the adapter's rank; a NULL part (or grads
 *          NULL) is not wanted. The rank and scale in it are not read. Without an
 *          adapter: NULL.
 * Errors: as qmlp_train_forward (INVALID_ARG: gradients without an adapter or
 * of a part that it lacks). */
qmlp_status qmlp_train_backward(qmlp_train_t* t, const qmlp_adapter* adapter, const void* x, int M, const void* saved,
                                const void* dout, void* dx, const qmlp_adapter* grads, qmlp_stream_t stream);

/*
 * AdamW over many tensors at once (one launch a step), for the adapters and
 * other small tensors trained beside the frozen weights. For every element,
 * in fp32, with step number t:
 *   g = grad_scale * grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * 8-bit states: each 256 consecutive elements of a tensor have one fp32 scale
 * (the last block may be short): m = e4m3fn(code) * scale, and sqrt(v) =
 * e4m3fn(code) * scale, where the scale is the block's largest magnitude / 448
 * and a root above zero keeps at least the smallest code. A new state is
 * zeros (codes and scales). A gradient that is not finite makes its element's
 * states NaN (and, where it is infinite, its block's), as in any AdamW: check
 * for it before the step.
 */
typedef enum { QMLP_STATE_FP32 = 1, QMLP_STATE_8BIT = 2 } qmlp_state;

typedef struct {
    int64_t n;        /* elements, >= 1                                            */
    void* param;      /* device [n], fp32 or bf16                                  */
    float* master;    /* device fp32 [n] beside a bf16 param, or NULL: the step is
                         taken on it and param = bf16(master) is written           */
    const void* grad; /* device [n], fp32 or bf16                                  */
    void* m;          /* device [n]: fp32, or e4m3fn codes                         */
    void* v;          /* device [n]: fp32, or the e4m3fn codes of its square root  */
    float* m_scale;   /* 8-bit states: device fp32 [ceil(n / 256)]; else NULL      */
    float* v_scale;
} qmlp_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    double grad_scale; /* multiplies every gradient (1: none)  */
    int64_t step;      /* t, from 1                            */
} qmlp_adamw_hyper;

typedef struct qmlp_adamw_s qmlp_adamw_t;

/* Make a handle over `count` tensors (host array, copied; the tensors stay the
 * caller's and must live as long as the handle). All parameters have one type
 * (pdt: FP32 or BF16), all gradients one (gdt: FP32 or BF16), all states one
 * (state); with a master, every tensor has one. Any alignment of the elements'
 * own size is served; tensors whose pointers are 16-byte aligned (8 for
 * codes) are read and written 8 elements at a time. Synchronizes `stream`.
 * Errors: INVALID_ARG (null, bad enum, mixed masters, a master beside fp32,
 * missing scales), SHAPE (count < 1, n < 1, over 2^31 chunks of 2048),
 * ALIGNMENT, ALIAS (a written buffer overlaps another one), UNSUPPORTED_ARCH,
 * OOM, CUDA. */
qmlp_status qmlp_adamw_create(qmlp_adamw_t** out, const qmlp_adamw_tensor* tensors, int count, qmlp_dtype pdt,
                              qmlp_dtype gdt, qmlp_state state, qmlp_stream_t stream);
void qmlp_adamw_destroy(qmlp_adamw_t* h);

/* One step on every tensor. Allocates nothing; can be captured in a CUDA graph
 * (the hyperparameters are then the captured ones).
 * Errors: INVALID_ARG (null; step < 1; beta outside [0, 1); a value that is
 * not finite), CUDA. */
qmlp_status qmlp_adamw_step(qmlp_adamw_t* h, const qmlp_adamw_hyper* hyper, qmlp_stream_t stream);

/*
 * The norms before and after a block, fused with the block's gate, residual and
 * residual scale: what stands between two blocks of a decoder layer in one pass.
 * For every token, with z the block's output and r the residual stream:
 *   n = z / rms(z) * (post_w + offset)     (post_w NULL: n = z)
 *   h = r + scale * gate * n               (z NULL: h = r; residual NULL: r = 0)
 *   y = h / rms(h) * (pre_w + offset)      rms(v) = sqrt(mean(v^2) + eps)
 * The norm reads h before its rounding to the stream's type: h and y are rounded
 * once each. Sums, with the squares, are fp32. The backward pass gives the
 * gradients of z, r, both weights and the gate; sums over tokens are fp32 in an
 * order that depends on the sizes alone: the same call gives the same bytes.
 */
/* What the gate has: nothing, a value a channel [K], a token [M] or an element [M, K]. */
typedef enum { QMLP_GATE_NONE = 0, QMLP_GATE_CHANNEL = 1, QMLP_GATE_TOKEN = 2, QMLP_GATE_FULL = 3 } qmlp_gate;

typedef struct {
    int K;               /* 1 .. 16384                                              */
    float eps;
    float weight_offset; /* added to both weights (1 for weights kept about zero)   */
    float scale;         /* of the block's output                                   */
    qmlp_dtype dt;       /* z, out, gate a token / element, their gradients: BF16, FP16 */
    qmlp_dtype rdt;      /* the residual stream and its gradients: dt or FP32        */
    qmlp_dtype wdt;      /* weights, gate a channel, their gradients: dt or FP32     */
    qmlp_gate gate;
} qmlp_norm_desc;

/* Device arrays, row-major and contiguous, of any alignment of their elements
 * (stats: 8 bytes). Where K is a multiple of 8 and all are 16-byte aligned, rows
 * are read 16 bytes at a time. */
typedef struct {
    const void* z;        /* [M, K], or NULL: no block, only the norm before         */
    const void* residual; /* [M, K], or NULL                                         */
    const void* post_w;   /* [K], or NULL: no norm after the block                   */
    const void* pre_w;    /* [K], or NULL: no norm before the next one (no out)      */
    const void* gate;     /* as the handle's gate; NULL without one or without z     */
    void* residual_out;   /* h [M, K], or NULL; may be residual itself (no backward then) */
    void* out;            /* y [M, K], exactly where pre_w is                        */
    float* stats;         /* [M][2]: 1/rms of z and h, for the backward pass, or NULL */
} qmlp_norm_io;

/* Gradients: of y (exactly where pre_w is) and of h behind (NULL: zero), read; the
 * others written, NULL where not wanted. dresidual may be dresidual_out itself. */
typedef struct {
    const void* dout;
    const void* dresidual_out;
    void* dz;
    void* dresidual;
    void* dpost_w;
    void* dpre_w;
    void* dgate;
} qmlp_norm_grads;

typedef struct qmlp_norm_s qmlp_norm_t;

/* Make a handle (it holds 24 K bytes an SM for the backward pass's column sums).
 * Errors: INVALID_ARG (null, types, a value that is not finite), SHAPE,
 * UNSUPPORTED_ARCH, OOM, CUDA. */
qmlp_status qmlp_norm_create(qmlp_norm_t** out, const qmlp_norm_desc* desc, qmlp_stream_t stream);
void qmlp_norm_destroy(qmlp_norm_t* h);

/* Forward on M tokens. Allocates nothing; can be captured in a CUDA graph.
 * Errors: INVALID_ARG (nothing to norm, post_w without z, a gate where the handle
 * has none or none where it has one, out without pre_w or the reverse), SHAPE
 * (M < 1), ALIGNMENT, ALIAS (an output overlaps another array), CUDA. */
qmlp_status qmlp_norm_forward(qmlp_norm_t* h, const qmlp_norm_io* io, int M, qmlp_stream_t stream);

/* Backward: io as the forward's, with the stats that it wrote (residual_out and
 * out are not read). residual is the one that the forward read: one that it wrote
 * residual_out over is gone, and the caller keeps a copy. Errors: as the forward;
 * INVALID_ARG also for no stats, no gradient to start from, or a gradient of what io
 * lacks; ALIAS also where residual_out overlaps residual. */
qmlp_status qmlp_norm_backward(qmlp_norm_t* h, const qmlp_norm_io* io, const qmlp_norm_grads* grads, int M,
                               qmlp_stream_t stream);

/*
 * One projection with 4-bit weights and group scales, for the projections beside
 * the MLP (attention's, an output head's):
 *   y[m, n] = c sum_k x[m, k] W[n, k] + bias[n]
 *   NVFP4: W[n, k] = E2M1(code) E4M3(scale[n, k / 16]), c = fp32(1 / global_scale)
 *   INT4:  W[n, k] = (code - zero[n, k / group]) scale[n, k / group], c = 1
 * Sums are fp32 and y is rounded once, to the type of the output.
 */
typedef enum { QMLP_LINEAR_NVFP4 = 1, QMLP_LINEAR_INT4 = 2 } qmlp_linear_format;

/* Arrays in host or device memory, read only by qmlp_linear_create, in the
 * checkpoint's order: two codes a byte, the low nibble the even k. */
typedef struct {
    qmlp_linear_format fmt;
    int N;                /* outputs, 1 .. 2^20                                    */
    int K;                /* inputs, a multiple of 16 and of group, 16 .. 65536    */
    int max_M;            /* most tokens of a call, 1 .. 65536                     */
    int group;            /* INT4: 32, 64 or 128; NVFP4: 16                        */
    const uint8_t* w;     /* u8 [N, K/2]                                           */
    const void* scale;    /* NVFP4: E4M3 [N, K/16]; INT4: fp16 [N, K/group]        */
    const uint8_t* zero;  /* INT4: u8 [N, K/group]; NVFP4: NULL                    */
    float global_scale;   /* NVFP4                                                 */
    const float* bias;    /* fp32 [N], or NULL                                     */
} qmlp_linear_desc;

typedef struct qmlp_linear_s qmlp_linear_t;

/* Make a handle: copies the weights into memory of its own, reordered for the
 * kernels (packed as they are), and makes the workspace of calls of up to max_M
 * tokens. Synchronizes `stream`.
 * Errors: INVALID_ARG, SHAPE, UNSUPPORTED_ARCH, OOM, CUDA. */
qmlp_status qmlp_linear_create(qmlp_linear_t** out, const qmlp_linear_desc* desc, qmlp_stream_t stream);
void qmlp_linear_destroy(qmlp_linear_t* h);

/* y = x W^T + bias on M tokens.
 *  x   = device [M, K], bf16 or fp16 per xdt
 *  out = device [M, N], bf16, fp16 or fp32 per odt
 * Allocates nothing; can be captured in a CUDA graph. The same call gives the same
 * bytes. One handle serves one stream at a time.
 * x is exact: fp16 as it is, bf16 times a power of two a token, exact for every value
 * within 2^29 of the token's largest. Up to 64 tokens every product is exact too. From 65
 * on the weights are decoded once a call into images of the tensor-core GEMM (at most
 * 1 GiB held by a handle made for 65 tokens or more, in turn for larger projections), in
 * which an INT4 weight is rounded once to fp16; NVFP4's are exact in it. Into an fp32 out
 * what that rounding leaves is added by a second product, and sums leave the tensor cores'
 * accumulators every few steps whatever M is, so that it keeps fp32's precision.
 * Errors: INVALID_ARG, ALIGNMENT (16 bytes), ALIAS, SHAPE (M < 1 or over max_M),
 * CUDA. */
qmlp_status qmlp_linear_forward(qmlp_linear_t* h, const void* x, qmlp_dtype xdt, int M, void* out, qmlp_dtype odt,
                                qmlp_stream_t stream);
/* As qmlp_check. */
qmlp_status qmlp_linear_check(qmlp_linear_t* h, qmlp_stream_t stream);

/*
 * A whole mixture-of-experts layer over the banks of a routed-expert handle: router,
 * selection, routed and shared experts, weighted sum. For every token x, with E
 * routed experts and the last `shared` of the handle's experts shared ones:
 *   l[e] = router[e] . x;   p = softmax(l) or sigmoid(l)
 *   the topk experts with the largest p[e] (+ bias[e]) are selected, ties to the
 *   lowest e (a NaN ranks below every number);
 *   w[e] = route_scale p[e], over the sum of the selected p where renorm is set
 *   a shared expert's w is 1, or sigmoid(shared_gate . x)
 *   out = sum of w[e] W2[e] (SiLU(g) u),  g, u = the halves of W13[e] x
 * (a shared expert of n times the width is n shared experts of the handle's I).
 * Sums are fp32, the intermediate is rounded once, to fp16 times a power of two of the
 * token and expert (to two fp16 for an fp32 out), and out once: values have fp32's range
 * up to out's type. A token's result does not depend on the others of the call. Up to 16
 * tokens whose x fits in shared memory (2 K bytes a token) run as one kernel; more run
 * the router, the selection and the kernels of qmlp_moe_forward, without that entry
 * point's roundings of the stages to fp16.
 */
typedef enum { QMLP_SCORE_SOFTMAX = 1, QMLP_SCORE_SIGMOID = 2 } qmlp_score;

typedef struct {
    const void* router;      /* [E, K], host or device, copied; E = the handle's E - shared */
    qmlp_dtype rdt;          /* type of router and shared_gate: BF16, FP16 or FP32          */
    const float* bias;       /* fp32 [E] that selection (not w) adds to p, or NULL          */
    const void* shared_gate; /* [shared, K], or NULL: w = 1                                 */
    int shared;              /* >= 0                                                        */
    int topk;                /* 1 .. E; topk + shared <= 16                                 */
    qmlp_score score;
    int renorm;
    float route_scale;
    int max_tokens;          /* of a call                                                   */
} qmlp_moe_layer_desc;

typedef struct qmlp_moe_layer_s qmlp_moe_layer_t;

/* Make a layer over the handle's banks (which must outlive it and whose workspace
 * for more than 16 tokens it shares: calls on both go on one stream at a time).
 * Reserves max_tokens on the handle (qmlp_moe_reserve; its limits, K <= 8192 among them,
 * hold where not every call of up to max_tokens is the one kernel's, and with more than
 * eight selected and shared experts a token the workspace is then larger: 4 bytes for each
 * of them and each of K + I values). Copies the router. E <= 1024. Synchronizes `stream`.
 * Errors: INVALID_ARG, SHAPE, OOM, CUDA. */
qmlp_status qmlp_moe_layer_create(qmlp_moe_layer_t** out, qmlp_moe_t* moe, const qmlp_moe_layer_desc* desc,
                                  qmlp_stream_t stream);
void qmlp_moe_layer_destroy(qmlp_moe_layer_t* h);

/* The layer on M tokens.
 *  x   = device [M, K], bf16 or fp16 per xdt;  out = device [M, K] of type odt
 *  ids, weights = device int32 / fp32 [M, topk]: the selected experts, largest
 *        first, and their w; either may be NULL
 * Allocates nothing; can be captured in a CUDA graph. The same call gives the same
 * bytes. The one-kernel form is a cooperative launch with a CTA an SM: it starts
 * when the whole GPU has room, and its grid barriers wait 2 s at most (then out is
 * not valid and qmlp_moe_layer_check returns QMLP_ERR_DEVICE_TIMEOUT).
 * Errors: INVALID_ARG, ALIGNMENT (16 bytes; ids and weights 4), ALIAS, SHAPE, CUDA. */
qmlp_status qmlp_moe_layer_forward(qmlp_moe_layer_t* h, const void* x, qmlp_dtype xdt, int M, void* out, qmlp_dtype odt,
                                   int32_t* ids, float* weights, qmlp_stream_t stream);
qmlp_status qmlp_moe_layer_check(qmlp_moe_layer_t* h, qmlp_stream_t stream);

/* Human-readable name of a status ("QMLP_OK", ...). Never NULL. */
const char* qmlp_status_str(qmlp_status s);

/* ABI version of this header (major * 100 + minor): 104 (dequantise-once GEMM path). */
int qmlp_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* QMLP_H */
