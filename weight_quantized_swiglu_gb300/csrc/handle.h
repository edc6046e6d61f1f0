// handle.h -- the dense and routed-expert handles and the host-side helpers shared by
// the files that implement the C ABI (api.cu, api_adapt.cu, api_layer.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <functional>
#include <vector>

#include "internal.h"
#include "qmlp.h"

namespace qmlp {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

inline qmlp_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return QMLP_OK;
    if (e == cudaErrorMemoryAllocation) return QMLP_ERR_OOM;
    return QMLP_ERR_CUDA;
}

// Fault injection for host-side tests of the error paths: QMLP_FAULT_INJECT=
// "alloc" makes every device allocation fail, "alloc:N" the N-th one a handle
// makes (N >= 1; the earlier ones succeed and must be released), "launch"
// makes forward calls return QMLP_ERR_CUDA before launching anything.
inline bool fault(const char* what) {
    const char* v = getenv("QMLP_FAULT_INJECT");
    return v && strcmp(v, what) == 0;
}
inline long fault_alloc_index() {
    const char* v = getenv("QMLP_FAULT_INJECT");
    if (!v || strncmp(v, "alloc:", 6) != 0) return 0;
    return strtol(v + 6, nullptr, 10);
}

struct Owner {
    std::vector<void*> ptrs;
    long count = 0;  // allocations attempted by this owner
    cudaError_t alloc(void** p, size_t bytes) {
        *p = nullptr;
        ++count;
        if (fault("alloc") || fault_alloc_index() == count) return cudaErrorMemoryAllocation;
        if (bytes == 0) bytes = 16;
        cudaError_t e = cudaMalloc(p, bytes);
        if (e == cudaSuccess) ptrs.push_back(*p);
        return e;
    }
    void release() {
        for (void* p : ptrs) cudaFree(p);
        ptrs.clear();
    }
};

// No C++ exception leaves a C entry: what the host cannot allocate is OOM.
template <typename F>
qmlp_status guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return QMLP_ERR_OOM;
    }
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether a written range overlaps any other one (ranges sorted in place).
struct Range {
    uintptr_t at, end;
    bool written;
};
inline bool any_alias(std::vector<Range>& r) {
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
    uintptr_t end = 0, wend = 0;  // the farthest end of any earlier range, and of any written one
    for (const Range& x : r) {
        if (x.at < wend || (x.written && x.at < end)) return true;
        end = std::max(end, x.end);
        if (x.written) wend = std::max(wend, x.end);
    }
    return false;
}

inline qmlp_status check_device(int* dev, int* num_sms) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return QMLP_ERR_CUDA;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
        return QMLP_ERR_CUDA;
    if (major != 10 || minor != 3) return QMLP_ERR_UNSUPPORTED_ARCH;
    return QMLP_OK;
}

}  // namespace qmlp

struct qmlp_moe_s {
    int E = 0, K = 0, I = 0, meta = 0, device = 0, num_sms = 0;
    uint8_t *w13 = nullptr, *w13_meta = nullptr, *w2 = nullptr, *w2_meta = nullptr;
    __half* act_ws = nullptr;
    int* err = nullptr;
    // multi-token workspace (moe_reserve): routes = max_tokens * 16
    int max_tokens = 1;
    size_t g_bytes = 16 * sizeof(__half);  // of a token and column in the two below
    void* g_act = nullptr;     // fp16 [routes, I], or fewer routes in fp32
    void* g_y = nullptr;       // fp16 [routes, K], or fewer routes in fp32
    int* g_route = nullptr;    // [routes]
    int4* g_groups = nullptr;  // [moe_grouped_max_groups(routes, E)]
    int* g_ngroups = nullptr;
    qmlp::Owner mem;
};

// Makes the workspace of calls of max_tokens tokens, with `bytes` (of all its routes)
// for a token and column, where the handle does not have it.
qmlp_status moe_reserve(qmlp_moe_s* h, int max_tokens, size_t bytes, cudaStream_t s);
// The grouped routed experts on M tokens (reserved for). amax null: the stages in fp16,
// out too. Else [M, topk] zeros: the stages in fp32 and scaled (reserved with 4 topk
// bytes or more), out of type odt (0 fp32, 1 bf16, 2 fp16).
cudaError_t moe_grouped(qmlp_moe_s* h, const void* x, bool x_bf16, const int32_t* ids, const float* rw, int topk, int M,
                        void* out, int odt, int* amax, cudaStream_t s);

struct qmlp_s {
    int fmt = 0, K = 0, I = 0, max_M = 0, device = 0, num_sms = 0;
    qmlp::GemvProj gv[3];  // gate, up, down
    int layout_warps = 0;       // streaming warps of the GEMV record layout
    qmlp::SplitPlan sp;               // I-partitioned decode plan (sp.G == 0: none)
    uint8_t* wsplit = nullptr;  // down records in the CTA-sliced layout
    float* spart = nullptr;     // [G][16][K] fp32 partial outputs
    unsigned long long* ticket = nullptr;  // grid-barrier ticket counter
    size_t lim_a = 0;  // index-check tests: bytes of the decode kernel's gate/up banks the checks allow (0: all)
    bool has_gemm = false;
    qmlp::GemmProj gm_gu, gm_d;
    void* a16 = nullptr;       // fp16 [max_M, max(K, I)] (GEMM prescaled activations)
    uint8_t* wdec = nullptr;   // dequantise-once GEMM: one projection's decoded bf16 stage images
    size_t wdec_bytes = 0;
    uint8_t* wdec2 = nullptr;  // the down projection's images, decoded on `side` beside the gate/up GEMM
    size_t wdec2_bytes = 0;
    cudaStream_t side = nullptr;  // the handle's own stream for that predecode
    cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
    float* gemm_ws = nullptr;  // split-K partials of the GEMM (small M)
    int* sig = nullptr;        // [max_M] per-token prescale exponents
    void* act = nullptr;       // bf16 [max_M, I]
    float* part = nullptr;     // split-K partials
    size_t part_cap = 0;
    int* counters = nullptr;   // [Nt(gate/up) + Nt(down)]
    int* err = nullptr;        // device error word
    unsigned* bar = nullptr;   // grid barrier {count, generation}
    void* x_stage = nullptr;   // bf16 [max_M, K] (forward_host)
    void* out_stage = nullptr; // bf16 [max_M, K]
    int rank = 0, nranks = 1;  // tensor-parallel shard of the intermediate dimension
    uint64_t wait_ns = 0;      // error-path tests: bounded-wait limit of the kernels (0: default)
    bool withhold = false;     // error-path tests: the kernels' producers skip their last step
    qmlp::Owner mem;
};

constexpr int kMaxGemvM = 16;

// Largest token block one launch of the I-partitioned decode kernel takes: 16
// for FP8 (two 8-token column tiles, x staged in two halves) where the
// partition allows it, else 8. Measured on the 27B-class shape at 16 tokens:
// FP8 85 us against 96 us on the split-K GEMM; NVFP4 144 us against 87 us
// (its group scales cost two fp32 FMAs per accumulator element, and every CTA
// writes and the reduce kernel reads a [16, K] fp32 partial: 2 x 44.6 MB).
inline int split_max_m(const qmlp_s* h) {
    if (!h->sp.G) return 0;
    return h->fmt == qmlp::kFP8 && qmlp::split_fits(h->fmt, kMaxGemvM, h->K, h->sp) ? kMaxGemvM : 8;
}

// Fewest tokens the automatic path sends to the tensor-core GEMM: past what
// one launch of the I-partitioned decode kernel takes (a second launch, which
// streams the weights again, loses to the split-K GEMM: measured on the
// 27B-class shape, 106-142 us for 9..16 tokens as two 8-token launches
// against 87-117 us). Shapes without the I partition decode 16 tokens per
// stream-K pass.
inline int gemm_min_m(const qmlp_s* h) { return h->sp.G ? split_max_m(h) + 1 : kMaxGemvM + 1; }

// Fewest tokens the automatic path sends to the dequantise-once GEMM (each
// projection decoded once per call into fp16 stage images, then a GEMM
// without decoder warps), and the handle's max_M from which it holds the
// decode buffer (4 I K bytes: the larger projection). Measured on the
// 27B-class shape (NVFP4 / FP8, ms, decoder warps against decoded once):
// M = 512 0.322 / 0.345 against 0.357 / 0.386; M = 1024 0.607 / 0.644
// against 0.552 / 0.578; M = 8192 3.49 / 3.70 against 2.79 / 2.80. With the
// CTA-pair form: M = 640 0.360 / 0.386 against 0.378 / 0.409, M = 768
// 0.402 / 0.428 against 0.383 / 0.414 (below, the down projection's few
// 256-token tiles leave most pairs idle).
constexpr int kDqMinM = 768;
// The dequantise-once GEMM runs on CTA pairs from kPairMinM tokens (measured
// at M = 8192, NVFP4 / FP8: 2.67 / 2.72 ms against 2.79 / 2.81 on single
// CTAs; at M = 1024 0.520 / 0.550 against 0.553 / 0.578).
constexpr bool kDqPair = true;

// The I-partitioned decode kernel on M tokens, without its output: act goes to
// the workspace.
inline qmlp::SplitLaunch split_launch(const qmlp_s* h, const void* x, int M) {
    qmlp::SplitLaunch S;
    S.fmt = h->fmt;
    S.M = M;
    S.K = h->K;
    S.I = h->I;
    S.gate = h->gv[0];
    S.up = h->gv[1];
    S.wdown = h->wsplit;
    S.chsd = h->gv[2].chs;
    S.invd = h->gv[2].inv_g;
    S.x = x;
    S.act_out = h->act;
    S.part = h->spart;
    S.ticket = h->ticket;
    S.err = h->err;
    S.wait_ns = h->wait_ns;
    S.withhold = h->withhold;
    S.lim_a = h->lim_a;
    return S;
}

// Terms of low-rank adapters that the GEMMs add: gate and up [M][2I], which
// `before` computes, then, once `between` has run on the workspace act, down's
// [M][K]. ev: an event for the images decoded beside `before`.
struct GemmTerms {
    const float* add = nullptr;
    const float* add_down = nullptr;
    cudaEvent_t ev = nullptr;
    std::function<cudaError_t(cudaStream_t)> before, between;
    // or (tokens in the order of `rows`, x = their rows): further steps of the GEMMs
    int ext = 0, ext_down = 0;
    const void *v = nullptr, *img = nullptr, *img_down = nullptr;
    const int2* ents = nullptr;
    const int* ent_slot = nullptr;
    int entries = 0, slots = 0;
    const int* rows = nullptr;
    const int* add_rows = nullptr;  // add and add_down: only to these tokens
    size_t add_elems = 0;           // index checks: values that add and add_down hold
};
qmlp_status run_gemm(qmlp_s* h, qmlp_path path, int stages, const void* x, int M, void* out, cudaStream_t s,
                     float* out_f32, const GemmTerms* ex);
