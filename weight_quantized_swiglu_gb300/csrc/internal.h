// internal.h -- host-side structures shared by the qmlp translation units.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qmlp.h"

namespace qmlp {

enum Fmt { kNVFP4 = 1, kFP8 = 2 };

// Rows per tensor-core tile of the GEMV kernels and k per "chunk" (four
// NVFP4 scale groups of 16).
constexpr int kTileRows = 16;
constexpr int kChunkK = 64;

// Epilogue of a GEMV launch.
enum GemvEpi {
    kEpiSwiGLU = 0,  // two projections (gate, up) -> act = bf16(SiLU(g)*u)
    kEpiPlain = 1,   // one projection -> bf16(sigma * acc)
    kEpiRaw = 2,     // one projection -> fp32 acc (no scale), debug
    kEpiSwiGLUGrad = 3, // d act -> [d gate | d up] (GEMM, training)
    kEpiOut = 4         // one projection, factor a row -> bf16, fp16 or fp32, + bias, any number of columns (GEMM)
};

// One projection [N, K] in the GEMV ("fragment-native") layout: one record
// per 16-row x 64-k chunk, row-tile-major (see gemv_frag.cuh):
//  NVFP4: 576 B = 512 B of E2M1 bytes in mma A-fragment order + 64 B of E4M3
//         scales; FP8: 1024 B of e4m3fn bytes, with chs = fp32 [N] scales.
// Nt = N/16 row tiles, Kc = ceil(K/64) chunks (zero padded).
// Records are stored interleaved for the stream kernel: warp w of TWr
// streaming warps owns the logical records [w*Lr, (w+1)*Lr) (row-tile-major
// order), taken Rr at a time; logical record u = w*Lr + k is stored at
// ((k / Rr) * TWr + w) * Rr + k % Rr, so at step j the 16 warps of a CTA
// find their Rr records each in one contiguous block and the GPU sweeps one
// contiguous window at a time. Lr is a multiple of Rr.
struct GemvProj {
    const uint8_t* wc = nullptr;
    const float* chs = nullptr;
    float inv_g = 1.0f;
    int N = 0, K = 0, Nt = 0, Kc = 0;
    int Lr = 1, TWr = 1, Rr = 1;
};
__host__ __device__ inline size_t gemv_rec_pos(size_t u, int Lr, int TWr, int Rr) {
    const size_t w = u / (size_t)Lr, k = u % (size_t)Lr;
    return ((k / (size_t)Rr) * (size_t)TWr + w) * (size_t)Rr + k % (size_t)Rr;
}
// Streaming warps of the layout on a device with num_sms SMs.
int gemv_layout_warps(int num_sms);

struct GemvLaunch {
    int fmt;
    int epi;
    GemvProj p0, p1;         // p1 used by kEpiSwiGLU only
    const void* x;           // bf16 [M, K]
    int M;
    void* out;               // bf16 [M, N] (act or out) or fp32 [M, N] (raw)
    float* part;             // fp32 split-K partials
    size_t part_cap;         // elements available in part
    int* counters;           // >= Nt zeroed ints
};

cudaError_t launch_gemv(const GemvLaunch& L, int num_sms, cudaStream_t s);

// Persistent stream-K GEMV (gemv_stream.cu). One phase = one projection, or
// gate+up with the SwiGLU epilogue; with a second phase the launch is
// cooperative and runs gate/up -> grid barrier -> down.
struct GemvStreamPhase {
    int epi;
    GemvProj p0, p1;
    const void* x;   // bf16 [M, p0.K]
    void* out;       // bf16 or fp32 [M, p0.N]
    int* counters;   // >= p0.Nt zeroed ints
};
bool gemv_stream_fits(int fmt, int M, int K, int np, int R);
size_t gemv_stream_part_elems(int K, int I, int num_sms);
cudaError_t launch_gemv_stream(int fmt, int M, const GemvStreamPhase& A, const GemvStreamPhase* B, float* part,
                               size_t part_cap, unsigned* bar, int* err, int num_sms, cudaStream_t s);

// Create-time repack into the GEMV layout. src pointers are device copies of
// the checkpoint layout.
cudaError_t repack_nvfp4_gemv(const uint8_t* w, const uint8_t* scale, int N, int K, int Lr, int TWr, int Rr,
                              uint8_t* wc, cudaStream_t s);
cudaError_t repack_fp8_gemv(const uint8_t* w, int N, int K, int Lr, int TWr, int Rr, uint8_t* wc, cudaStream_t s);
size_t gemv_codes_bytes(int fmt, int N, int K, int Lr, int TWr);
// Records per warp per step of the layout: gate/up (streamed in pairs) take
// half as many as a projection streamed alone, so one step fills the same
// number of bytes in both cases; FP8 records (1024 B) take half as many as
// NVFP4 ones (576 B), so a step is 32-37 KB for both formats.
__host__ __device__ constexpr int gemv_recs_pair(int fmt) { return fmt == kFP8 ? 1 : 2; }
__host__ __device__ constexpr int gemv_recs_single(int fmt) { return fmt == kFP8 ? 2 : 4; }
// Largest split-K partial buffer (fp32 elements) any GEMV launch of a handle
// with these sizes can need for M <= 16.
size_t gemv_part_elems(int K, int I, int num_sms);

// ---------------------------------------------------------------------------
// I-partitioned fused decode MLP (gemv_split.cu): CTA b of G owns gate/up
// row tiles [T*b, T*(b+1)) and the matching Cb = T/4 down k-chunks.
// ---------------------------------------------------------------------------
struct SplitPlan {
    int G = 0;        // CTAs (0: no plan for this shape / device)
    int T = 0;        // gate/up row tiles per CTA
    int Cb = 0;       // down 64-k chunks per CTA
    int LA = 0;       // gate/up records per warp (= T*Kc/16; the gate/up layout uses Lr = LA, TWr = 16G)
    int LB = 0;       // down records per warp in the CTA-sliced layout (multiple of RB)
    int RA = 0, RB = 0;  // records per warp per step: gate/up pairs, down
    int SA = 0;       // most warps sharing one gate/up tile
};
SplitPlan plan_split(int fmt, int K, int I, int num_sms);
bool split_fits(int fmt, int M, int K, const SplitPlan& P);
// Whether the decode kernel reduces its partials itself (schedule (a)).
inline bool split_in_kernel(int fmt, int M) { return fmt == kNVFP4 && M == 1; }
bool split_lora_fits(int fmt, int M, int K, int lora_r, const SplitPlan& P);
size_t split_part_elems(int K, const SplitPlan& P);       // fp32 partials for M <= 16
size_t split_codes_bytes(int fmt, const SplitPlan& P);     // down records, CTA-sliced
// Down projection [K, I] into the CTA-sliced layout: local record u = w*LB + k
// of CTA b (u < Nt*Cb) is (row tile u / Cb, chunk Cb*b + u % Cb), stored at
// ((k / RB) * 16G + 16b + w) * RB + k % RB; records past Nt*Cb are zero.
cudaError_t repack_nvfp4_split(const uint8_t* w, const uint8_t* scale, int N, int K, const SplitPlan& P,
                               uint8_t* wc, cudaStream_t s);
cudaError_t repack_fp8_split(const uint8_t* w, int N, int K, const SplitPlan& P, uint8_t* wc, cudaStream_t s);
// Low-rank adapters inside the decode kernel (see gemv_split.cu).
struct SplitLora {
    const int* ids = nullptr;   // [M] slots (null: no adapters)
    const int* rank = nullptr;  // [slots]
    const float* scale = nullptr;
    int slots = 0, Rp = 0;
    const float* v = nullptr;   // fp32 [M][2 Rp]: c A x of gate and up, written by the launch before
    const __nv_bfloat16* b_gu = nullptr;  // [slots][2][I][Rp]
    const __nv_bfloat16* a_d = nullptr;   // [slots][Rp][I]
    const __nv_bfloat16* b_d = nullptr;   // [slots][K][Rp]
    float* vd = nullptr;        // [G][M][Rp]: the CTAs' shares of A_d act
};
struct SplitLaunch {
    int fmt = 0, M = 0, K = 0, I = 0;
    GemvProj gate, up;               // GEMV layout with TWr = 16G, Lr = LA
    const uint8_t* wdown = nullptr;  // CTA-sliced down records
    const float* chsd = nullptr;     // FP8 down per-channel scales
    float invd = 1.0f;               // NVFP4 down 1/global
    const void* x = nullptr;         // bf16 [M, K]
    bool x_in_host = false;          // x is device-mapped host memory: staged with plain loads
    void* act_out = nullptr;         // optional bf16 [M, I]
    void* out = nullptr;             // bf16 [M, K]
    float* out_f32 = nullptr;        // optional fp32 [M, K]: sums without the down factor, written instead of out
    const void* act_in = nullptr;    // optional bf16 [M, I]: the down projection consumes these (debug)
    float* dbg_g = nullptr;          // optional fp32 [M, I]: raw gate dot products (debug; with dbg_u)
    float* dbg_u = nullptr;          // optional fp32 [M, I]: raw up dot products (debug)
    SplitLora lora;
    float* part = nullptr;           // >= split_part_elems
    unsigned long long* ticket = nullptr;  // grid-barrier ticket counter (zeroed at create)
    int* err = nullptr;
    uint64_t wait_ns = 0;            // bounded-wait limit (0: the kernel's default of 2 s)
    bool withhold = false;           // error-path tests: the last weight step is never issued
    size_t lim_a = 0;                // index-check tests: bytes of the gate/up banks the checks allow (0: all)
};
cudaError_t launch_split(const SplitLaunch& L, const SplitPlan& P, cudaStream_t s);

// Tensor-parallel combine (tp_shard.cu): out[m, o] = bf16( sigma_d[o] * sum
// over r = 0..nranks-1, in rank order, of partials[r][m][o] ), sigma_d = invd
// (NVFP4) or chsd[o] (FP8).
cudaError_t launch_shard_combine(int fmt, const float* partials, int nranks, int M, int K, float invd,
                                 const float* chsd, void* out, cudaStream_t s);

// ---------------------------------------------------------------------------
// Tensor-core prefill GEMM (NVFP4, tcgen05)
// ---------------------------------------------------------------------------
struct GemmProj {
    int fmt = kNVFP4;                    // kNVFP4 or kFP8
    const uint8_t* tiles = nullptr;      // weight blocks [N/256][K/64][9216 B NVFP4 | 16384 B FP8], see gemm_tc.cu
    float inv_g0 = 1.0f, inv_g1 = 1.0f;  // NVFP4 global factors: (gate, up) when interleaved, else both = down
    const float* cs0 = nullptr;          // FP8 per-channel scales: gate when interleaved, else the projection's
    const float* cs1 = nullptr;          // FP8 up scales when interleaved
    int N = 0, K = 0;                    // N weight rows (2I when interleaved), K contraction length
    bool interleaved = false;            // tile rows = 128 gate rows then the same 128 up rows
};
size_t gemm_tiles_bytes(int fmt, int N, int K);
cudaError_t repack_fp8_gemm(const uint8_t* w0, const uint8_t* w1, int N, int K, bool interleave, uint8_t* tiles,
                            cudaStream_t s);
cudaError_t repack_nvfp4_gemm(const uint8_t* w0, const uint8_t* s0, const uint8_t* w1,
                              const uint8_t* s1, int N, int K, bool interleave, uint8_t* tiles,
                              cudaStream_t s);
struct GemmLaunch {
    int epi = kEpiPlain;  // kEpiSwiGLU / kEpiPlain / kEpiRaw
    int raw_sel = 0;      // kEpiRaw on an interleaved GEMM: 0 = gate rows, 1 = up rows
    GemmProj w;
    const void* a = nullptr;  // bf16 [M, K]
    int M = 0;
    void* out = nullptr;      // bf16 [M, N_out] or fp32 [M, N_out] (raw)
    void* a16 = nullptr;      // workspace fp16 [M, K]: prescaled activations
    int* sig = nullptr;       // workspace [M]: per-token prescale exponents
    int* err = nullptr;       // device error word
    float* ws = nullptr;      // split-K partials, >= gemm_splitk_ws_elems (null: no split-K)
    uint64_t wait_ns = 0;     // bounded-wait limit (0: the kernel's default of 2 s)
    bool withhold = false;    // error-path tests: the last k-step of each CTA is never loaded
    bool pair = false;        // the CTA-pair kernel (M >= kPairMinM; never split-K)
    uint8_t* wdec = nullptr;  // dequantise-once: decoded stage images of w (null: the decoder warps decode)
    size_t wdec_bytes = 0;    // bytes of wdec, >= gemm_decoded_bytes(w.N, w.K)
    // fp32 [M][ldadd], added after the factor: gate's I columns then up's (SwiGLU),
    // or the output's columns (plain, grad); the terms of low-rank adapters
    const float* add = nullptr;
    size_t ldadd = 0, add_elems = 0;  // add_elems: index checks
    // early: the kernels that write add are launched just before, each with
    // programmatic dependent launch; nothing else that the GEMM reads (prescaled
    // activations, images) comes from them. It reads those without a wait, so the
    // first of these kernels lets the next one start only after its own wait, when
    // all that came before has completed and is visible
    bool early = false;
    bool prescaled = false;      // a16 and sig are written (launch_gemm_prescale)
    void* gu_g = nullptr;        // training: fp32 gate and up values, kept by SwiGLU and read by SwiGLUGrad,
    void* gu_u = nullptr;        // gemm_gu_bytes(M, I) each
    int ncols = 0;               // SwiGLUGrad: I; out = [M][2I]
    float gf0 = 1.0f, gf1 = 1.0f;  // SwiGLUGrad: factors of d gate, d up, or per column:
    const float* gc0 = nullptr;
    const float* gc1 = nullptr;
    bool f16 = false;            // dequantise-once: images in fp16, activations prescaled to fp16 (into a16)
    bool split_tail = false;     // CTA pairs, plain: the last tiles may be split over the contraction (into ws)
    int ext = 0;                 // CTA pairs: further contraction steps of 64, bf16: activations [M][64 ext]
    const void* ext_a = nullptr; // and stage images [N / 256][ext] (low-rank adapters)
    const void* ext_b = nullptr;
    // several adapters: the entries of each 256-token tile {first, count}, their
    // slots; ext_a then holds 256 rows an entry, ext_b the images slot by slot
    const int2* ents = nullptr;
    const int* ent_slot = nullptr;
    int entries = 0, slots = 0;
    const int* rows = nullptr;   // plain: the output row of each token
    const int* add_rows = nullptr;  // CTA pairs: only tokens whose value is not 0 get `add` (null: all)
    void* out_lo = nullptr;      // with gu_g: optional, bf16 of what the rounding of out leaves
    bool images_ready = false;  // dequantise-once: wdec already holds w's images (no predecode launch)
    // kEpiOut (CTA pairs, f16 images, w.fmt FP8: a factor a row): out = [M][ldo] of odt
    // (0 fp32, 1 bf16, 2 fp16), the first ncols of w.N columns written, + bias
    int ldo = 0, odt = 1;
    const float* bias = nullptr;
    int ka = 0;                 // row length of a (0: w.K): k past it is zero
    bool unscaled = false;      // a16 is fp16 as it came: no exponents
    bool onto = false;          // kEpiOut, fp32: added to what out holds
};
constexpr int kPairMinM = 256;  // one 256-token tile of a CTA pair
// Fewest tokens of one projection that the GEMM takes, a 256-token tile of them in part:
// its time hardly depends on their number (17408 x 5120 81 us from 65 to 255 tokens; launches
// of 64 tokens each 80 us at 128, 120 at 192; 5120 x 5120 36 to 73 us, 1024 x 5120 22 to 58
// at 130), one launch of up to 64 takes half of it. (The MLP's GEMM with decoder warps, which
// has neither these records nor INT4, is ahead of images up to some 700 tokens: three
// projections of the 27B-class block 178 us at 256 tokens and 322 at 512, images 103 to 132 a
// projection at 300.)
constexpr int kLinearGemmM = 65;
cudaError_t launch_gemm_prescale(const void* a, int M, int K, void* a16, int* sig, int num_sms, cudaStream_t s);
cudaError_t launch_gemm(const GemmLaunch& L, int num_sms, cudaStream_t s);
size_t gemm_splitk_ws_elems(int num_sms);
size_t gemm_decoded_bytes(int N, int K);  // bf16 stage images of an [N, K] projection (2 N K bytes)
// The dequantise-once predecode of projection P into wdec, on its own.
cudaError_t launch_gemm_predecode(const GemmProj& P, uint8_t* wdec, size_t wdec_bytes, int num_sms, cudaStream_t s);
// Images of the transposed projection (contraction over its N rows, its K
// columns as output rows, padded to 256).
size_t gemm_decoded_t_bytes(int N, int K);
cudaError_t launch_gemm_predecode_t(const GemmProj& P, const float* mul0, const float* mul1, bool f16, uint8_t* img,
                                    size_t img_bytes, cudaStream_t s);
inline size_t gemm_gu_bytes(int M, int I) { return (size_t)((M + 31) / 32) * 32 * I * 4; }
bool gemm_supported(int K, int N);

// ---------------------------------------------------------------------------
// Routed-expert AWQ M=1
// ---------------------------------------------------------------------------
struct MoeLaunch {
    int E, K, I, meta_bytes;
    int sliced = 0;           // 1: the banks are lane-sliced (the handle's copy), 0: checkpoint layout
    const uint8_t* w13;       // see moe_awq.cu
    const uint8_t* w13_meta;
    const uint8_t* w2;
    const uint8_t* w2_meta;
    const void* x;
    int x_is_bf16;
    const int32_t* ids;
    const float* rw;
    int topk;
    __half* out;
    __half* act_ws;           // [16][I] workspace
    __half* gu_dbg;           // optional [topk][2I]
    __half* act_dbg;          // optional [topk][I]
    __half* y_dbg;            // optional [topk][K]
};
cudaError_t launch_moe(const MoeLaunch& L, int num_sms, cudaStream_t s);

// M tokens, routes grouped by expert (see moe_grouped.cu).
constexpr int kMoeMaxI = 1024;         // of a routed-expert handle
constexpr int kMoeGroupedMaxK = 8192;  // x of a group's 8 tokens is staged in shared memory
constexpr int kMoeGroupedMaxE = 8192;  // the routing CTA keeps 4 ints per expert in shared memory
struct MoeGroupedLaunch {
    int E, K, I, meta_bytes, M, topk;
    int num_sms = 0;
    const uint8_t* w13;
    const uint8_t* w13_meta;
    const uint8_t* w2;
    const uint8_t* w2_meta;
    const void* x;                 // [M, K]
    int x_is_bf16;
    const int32_t* ids;            // [M, topk]
    const float* rw;               // [M, topk]
    void* out;                     // [M, K]
    int odt = 2;                   // type of out: 0 fp32, 1 bf16, 2 fp16 (without act32: 2)
    __half* act_ws = nullptr;      // [>= M*topk, I]
    __half* y_ws = nullptr;        // [>= M*topk, K]
    // instead, stages that are not limited to fp16's range (the mixture-of-experts
    // layer): the same in fp32, and [>= M*topk] zeros
    float* act32 = nullptr;
    float* y32 = nullptr;
    int* amax = nullptr;
    int* route_list;               // [>= M*topk]
    int4* groups;                  // [>= moe_grouped_max_groups(M*topk, E)]
    int* n_groups;                 // one int
};
size_t moe_grouped_max_groups(int routes, int E);
cudaError_t launch_moe_grouped(const MoeGroupedLaunch& L, cudaStream_t s);
// W13 bank of a handle in warp blocks: the one-token and grouped W13 kernels
// split K over kMoeKSplit warps, and warp ks of row octet o (gate rows
// 8o..8o+7 and the matching up rows) reads one contiguous block per expert.
// Block (e, o, ks) = [q (gate 0 / up 1)][pair p][lane l = 4g + t][16 B]: the
// 16 bytes are chunks c = ks*cpw + 2p and +1 (64 k each, zero past the warp's
// range), 8 bytes per chunk = the 32-bit words lane t picks from the chunk's
// two 16-byte units of row g (byte t of each word of the unit). Metadata:
// block (e, o, ks) = [q][g][the 2*cpw records of those chunks, padded to a
// multiple of 16 bytes, sized for whole batches of 4 chunks: the one-token
// kernel loads a batch's records at once]. Byte counts per block below.
constexpr int kMoeKSplit = 10;
__host__ __device__ inline int moe_w13_cpw(int K) { return (K / 64 + kMoeKSplit - 1) / kMoeKSplit; }
__host__ __device__ inline int moe_w13_pairs(int K) { return (moe_w13_cpw(K) + 1) / 2; }
__host__ __device__ inline size_t moe_w13_block_bytes(int K) { return (size_t)2 * moe_w13_pairs(K) * 512; }
__host__ __device__ inline int moe_w13_meta_stride(int K, int MB) {
    return (2 * ((moe_w13_cpw(K) + 3) / 4 * 4) * MB + 15) / 16 * 16;
}
__host__ __device__ inline size_t moe_w13_meta_block_bytes(int K, int MB) { return (size_t)2 * 8 * moe_w13_meta_stride(K, MB); }
inline size_t moe_w13_bank_bytes(int E, int I, int K) { return (size_t)E * (I / 8) * kMoeKSplit * moe_w13_block_bytes(K); }
inline size_t moe_w13_meta_bank_bytes(int E, int I, int K, int MB) {
    return (size_t)E * (I / 8) * kMoeKSplit * moe_w13_meta_block_bytes(K, MB);
}
// checkpoint W13 codes [E, 2I, K/2] and records [E, 2I, K/32] x MB -> the
// warp-block bank above
cudaError_t repack_moe_w13_blocks(const uint8_t* w, const uint8_t* meta, int meta_bytes, int E, int I, int K,
                                  uint8_t* w_out, uint8_t* meta_out, cudaStream_t s);
cudaError_t repack_moe(const uint8_t* w, const uint8_t* meta, int meta_bytes, int E, int N,
                       int Kr, uint8_t* w_out, uint8_t* meta_out, cudaStream_t s);

// ---------------------------------------------------------------------------
// AdamW over many tensors (adamw.cu)
// ---------------------------------------------------------------------------
constexpr int kAdamWBlock = 256;   // elements that share a scale in an 8-bit state
constexpr int kAdamWChunk = 2048;  // elements a CTA takes: 8 blocks of one tensor
struct alignas(16) AdamWChunk {    // one CTA's part of a tensor; pointers at its first element
    void* param;
    float* master;   // fp32 master of a bf16 parameter, or null
    const void* grad;
    void* m;
    void* v;
    float* m_scale;  // 8-bit states: the scale of the chunk's first block
    float* v_scale;
    int n;           // elements, 1 .. kAdamWChunk
    int vec;         // every pointer is aligned for 8 elements at a time
};
struct AdamWStep {  // the constants of a step, fp32 of fp64 values
    float gscale, b1, omb1, b2, omb2, rbc2, eps, decay, step;
};
cudaError_t launch_adamw(const AdamWChunk* chunks, long count, bool param_bf16, bool master, bool grad_bf16, bool s8,
                         const AdamWStep& k, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// Norms before and after a block (norm.cuh)
// ---------------------------------------------------------------------------
enum NormGate { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };
constexpr int kNormMaxK = 16384;
struct NormArgs {
    long M = 0;
    int K = 0;
    float eps = 0, rK = 0, offset = 0, scale = 1;  // rK: 1 / K
    int gate_kind = kGateNone;
    bool w_f32 = false;        // weights (and a channel gate) are fp32, else of z's type
    bool vec = false;          // every pointer is 16-byte aligned
    const void *z = nullptr, *r = nullptr, *post_w = nullptr, *pre_w = nullptr, *gate = nullptr;
    void *h = nullptr, *y = nullptr;
    float2* stats = nullptr;   // [M] 1/rms of z and h
    // backward
    const void *dy = nullptr, *dh = nullptr;
    void *dz = nullptr, *dr = nullptr, *dpost = nullptr, *dpre = nullptr, *dgate = nullptr;
    float* part = nullptr;     // [shares][3][K]: the CTAs' column sums (null: none is wanted)
    int shares = 0, num_sms = 0;
    size_t elems = 0, part_elems = 0;  // index checks: M K; floats of part
};
// A kernel's limit of dynamic shared memory, raised once a device (`done`: a bit each).
template <typename F>
cudaError_t smem_once(F* kernel, int bytes, unsigned long& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done |= 1ul << dev;
    return e;
}
cudaError_t launch_norm_f16(const NormArgs& a, bool r_f32, bool backward, cudaStream_t s);
cudaError_t launch_norm(const NormArgs& a, bool t_f16, bool r_f32, bool backward, cudaStream_t s);

// ---------------------------------------------------------------------------
// One projection with 4-bit weights and group scales (linear.cu)
// ---------------------------------------------------------------------------
constexpr int kLinearChunk = 128;  // k of a record of 16 rows
// Bytes of a record: codes, then scales and zeros of its groups (group 16: NVFP4)
constexpr int linear_rec_bytes(int group) {
    return 16 * kLinearChunk / 2 + 16 * (kLinearChunk / group) * (group == 16 ? 1 : 3);
}
size_t linear_bytes(int group, int N, int K);
cudaError_t repack_linear(int group, const uint8_t* w, const void* scale, const uint8_t* zero, int N, int K, uint8_t* out,
                          cudaStream_t s);
struct LinearArgs {
    int M = 0, N = 0, K = 0;
    const uint8_t* w = nullptr;   // records [N / 16][K / 128], rounded up
    size_t w_bytes = 0;
    float factor = 1.0f;          // NVFP4: 1 / global
    const float* bias = nullptr;  // fp32 [N], or null
    const void* x = nullptr;      // [M, K], bf16 or fp16
    bool x_bf16 = true;
    void* out = nullptr;          // [M, N]
    int odt = 0;                  // 0 fp32, 1 bf16, 2 fp16
    int* err = nullptr;           // device error word
    void* xf = nullptr;           // workspace of more than kLinearFew tokens: linear_x_bytes
    size_t xf_elems = 0;          // its 16-byte pieces
    int* sig = nullptr;           // [max_M] exponents of the tokens
};
constexpr int kLinearFew = 8;   // tokens whose x stays in shared memory
constexpr int kLinearMid = 64;  // tokens of linear_mid_kernel; more are the GEMM's
size_t linear_x_bytes(int K, int M);
cudaError_t launch_linear(int group, const LinearArgs& a, int num_sms, cudaStream_t s);
// Stage images of the tensor-core GEMM (fp16, rows times 2^-exponent of their factor)
// of rows n0.. (a multiple of 256) of the records: N rows padded to 256, K to 64. The
// factors of all rows: c, for INT4 times a power of two that keeps a row's images in
// fp16's range. rest: of INT4 what the images' rounding to fp16 leaves.
cudaError_t launch_linear_images(int group, const uint8_t* w, size_t w_bytes, const float* factors, int N, int K, int n0,
                                 int rows, bool rest, uint8_t* img, size_t img_bytes, cudaStream_t s);
cudaError_t launch_linear_factors(int group, const void* scale, int N, int K, float c, float* factors, int padded,
                                  cudaStream_t s);

// ---------------------------------------------------------------------------
// A whole mixture-of-experts layer (moe_layer.cu)
// ---------------------------------------------------------------------------
constexpr int kMoeLayerFew = 16;     // tokens that the one-kernel form takes at most
constexpr int kMoeLayerMaxE = 1024;  // routed experts
struct MoeLayerArgs {
    int M = 0, E = 0, S = 0, K = 0, I = 0, topk = 0;  // E routed experts, S shared ones behind them in the banks
    bool softmax = true, renorm = true;
    float rscale = 1.0f;
    // router and shared gates as fragments (router_frag_kernel): planes of fp16 words,
    // tiles of 16 rows; the rows' exponents [16 rtiles]
    const uint4* rfrag = nullptr;
    const int* rexp = nullptr;
    size_t rfrag_elems = 0;
    int planes = 1, rtiles = 0;
    bool sgate = false;             // the shared experts have gates: rows E..E + S - 1
    const float* bias = nullptr;    // [E], or null
    const uint8_t *w13 = nullptr, *w13_meta = nullptr, *w2 = nullptr, *w2_meta = nullptr;  // the handle's banks
    const void* x = nullptr;        // [M, K]
    bool x_bf16 = true;
    void* out = nullptr;            // [M, K]
    int odt = 1;                    // 0 fp32, 1 bf16, 2 fp16
    int32_t* ids_out = nullptr;     // [M, topk], or null
    float* w_out = nullptr;
    float* logits = nullptr;        // [max_tokens][E + S], few tokens: one such array a split of k
    int32_t* ids = nullptr;         // more tokens: [M][topk + S]
    float* weights = nullptr;
    float* act = nullptr;           // few tokens: [M (topk + S)][I]
    int* amax = nullptr;            // [max_tokens (topk + S)]: bits of the largest |act|
    uint4* act16 = nullptr;         // act in fp16, in the order of the products
    size_t act16_elems = 0;
    unsigned long long* ticket = nullptr;
    int* err = nullptr;
    uint64_t limit = 0;
    int slots = 0;                  // experts that M tokens can name, at most
    size_t w13_bytes = 0, w13_meta_bytes = 0, w2_bytes = 0, w2_meta_bytes = 0, logit_elems = 0, act_elems = 0;
};
constexpr int kMoeRouterSplits = 4;  // splits of the router's k over CTAs, at most
bool moe_layer_few(int M, int K, int I, int E, int S, int topk, int meta_bytes);
cudaError_t launch_router_layout(const MoeLayerArgs& a, const void* w, const void* sg, int type, uint4* frag, int* rexp,
                                 cudaStream_t s);
cudaError_t launch_moe_layer_few(MoeLayerArgs a, int meta_bytes, int num_sms, cudaStream_t s);
cudaError_t launch_moe_router(const MoeLayerArgs& a, cudaStream_t s);

// Index checks of a QMLP_DEBUG_BOUNDS build (common.cuh): each translation
// unit's first failed check, (site << 48) | index, or 0; reading clears it.
// The default build returns 0.
cudaError_t bounds_take_gemv_split(unsigned long long* v);
cudaError_t bounds_take_gemm_tc(unsigned long long* v);
cudaError_t bounds_take_gemv_stream(unsigned long long* v);
cudaError_t bounds_take_gemv_dec(unsigned long long* v);
cudaError_t bounds_take_moe_awq(unsigned long long* v);
cudaError_t bounds_take_moe_grouped(unsigned long long* v);
cudaError_t bounds_take_tp_shard(unsigned long long* v);
cudaError_t bounds_take_lowrank(unsigned long long* v);
cudaError_t bounds_take_adamw(unsigned long long* v);
cudaError_t bounds_take_norm(unsigned long long* v);
cudaError_t bounds_take_norm_f16(unsigned long long* v);
cudaError_t bounds_take_linear(unsigned long long* v);
cudaError_t bounds_take_moe_layer(unsigned long long* v);

}  // namespace qmlp
