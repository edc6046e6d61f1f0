// handle.h -- the dense handle and the host-side helpers shared by the files
// that implement the C ABI (api.cu, api_adapt.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
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
