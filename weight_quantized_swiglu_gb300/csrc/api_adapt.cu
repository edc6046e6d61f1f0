// api_adapt.cu -- the C ABI of training and serving adapters beside the
// frozen quantized weights (declared in include/qmlp.h): AdamW over many
// tensors. Argument checks, ownership and dispatch only, as api.cu.
#include <math.h>

#include "handle.h"

using namespace qmlp;

struct qmlp_adamw_s {
    AdamWChunk* chunks = nullptr;
    long count = 0;
    bool param_bf16 = false, master = false, grad_bf16 = false, s8 = false;
    Owner mem;
};

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether a written range overlaps any other one (ranges sorted in place).
struct Range {
    uintptr_t at, end;
    bool written;
};
bool any_alias(std::vector<Range>& r) {
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
    uintptr_t end = 0, wend = 0;  // the farthest end of any earlier range, and of any written one
    for (const Range& x : r) {
        if (x.at < wend || (x.written && x.at < end)) return true;
        end = std::max(end, x.end);
        if (x.written) wend = std::max(wend, x.end);
    }
    return false;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
qmlp_status qmlp_adamw_create(qmlp_adamw_t** out, const qmlp_adamw_tensor* ts, int count, qmlp_dtype pdt,
                              qmlp_dtype gdt, qmlp_state state, qmlp_stream_t stream) {
    if (!out) return QMLP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!ts) return QMLP_ERR_INVALID_ARG;
    if ((pdt != QMLP_DT_FP32 && pdt != QMLP_DT_BF16) || (gdt != QMLP_DT_FP32 && gdt != QMLP_DT_BF16) ||
        (state != QMLP_STATE_FP32 && state != QMLP_STATE_8BIT))
        return QMLP_ERR_INVALID_ARG;
    if (count < 1) return QMLP_ERR_SHAPE;
    const bool s8 = state == QMLP_STATE_8BIT, pb = pdt == QMLP_DT_BF16, gb = gdt == QMLP_DT_BF16;
    const bool master = ts[0].master != nullptr;
    if (master && !pb) return QMLP_ERR_INVALID_ARG;
    const size_t pe = pb ? 2 : 4, ge = gb ? 2 : 4, se = s8 ? 1 : 4;
    std::vector<Range> ranges;
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        const qmlp_adamw_tensor& t = ts[i];
        if (!t.param || !t.grad || !t.m || !t.v || (t.master != nullptr) != master ||
            (s8 && (!t.m_scale || !t.v_scale)) || (!s8 && (t.m_scale || t.v_scale)))
            return QMLP_ERR_INVALID_ARG;
        if (t.n < 1 || t.n > ((int64_t)1 << 40)) return QMLP_ERR_SHAPE;
        if (!aligned(t.param, pe) || !aligned(t.grad, ge) || !aligned(t.m, se) || !aligned(t.v, se) ||
            !aligned(t.master, 4) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
            return QMLP_ERR_ALIGNMENT;
        total += (t.n + kAdamWChunk - 1) / kAdamWChunk;
        if (total > 0x7fffffff) return QMLP_ERR_SHAPE;
        auto add = [&](const void* p, size_t bytes, bool w) {
            if (p) ranges.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, w});
        };
        const size_t n = (size_t)t.n, nb = (n + kAdamWBlock - 1) / kAdamWBlock;
        add(t.param, n * pe, true);
        add(t.master, n * 4, true);
        add(t.grad, n * ge, false);
        add(t.m, n * se, true);
        add(t.v, n * se, true);
        add(t.m_scale, nb * 4, true);
        add(t.v_scale, nb * 4, true);
    }
    if (any_alias(ranges)) return QMLP_ERR_ALIAS;
    int dev = 0, sms = 0;
    qmlp_status st = check_device(&dev, &sms);
    if (st != QMLP_OK) return st;
    std::vector<AdamWChunk> table;
    table.reserve((size_t)total);
    for (int i = 0; i < count; ++i) {
        const qmlp_adamw_tensor& t = ts[i];
        const bool vec = aligned16(t.param) && aligned16(t.grad) && aligned16(t.master) &&
                         aligned(t.m, s8 ? 8 : 16) && aligned(t.v, s8 ? 8 : 16);
        for (int64_t at = 0; at < t.n; at += kAdamWChunk) {
            AdamWChunk c;
            c.param = static_cast<uint8_t*>(t.param) + at * pe;
            c.master = master ? t.master + at : nullptr;
            c.grad = static_cast<const uint8_t*>(t.grad) + at * ge;
            c.m = static_cast<uint8_t*>(t.m) + at * se;
            c.v = static_cast<uint8_t*>(t.v) + at * se;
            c.m_scale = s8 ? t.m_scale + at / kAdamWBlock : nullptr;
            c.v_scale = s8 ? t.v_scale + at / kAdamWBlock : nullptr;
            c.n = (int)std::min<int64_t>(kAdamWChunk, t.n - at);
            c.vec = vec ? 1 : 0;
            table.push_back(c);
        }
    }
    qmlp_adamw_t* h = new qmlp_adamw_t();
    h->count = (long)table.size();
    h->param_bf16 = pb;
    h->master = master;
    h->grad_bf16 = gb;
    h->s8 = s8;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = h->mem.alloc(reinterpret_cast<void**>(&h->chunks), table.size() * sizeof(AdamWChunk));
    if (e != cudaSuccess) st = from_cuda(e);
    else if (cudaMemcpyAsync(h->chunks, table.data(), table.size() * sizeof(AdamWChunk), cudaMemcpyHostToDevice, s) !=
                 cudaSuccess ||
             cudaStreamSynchronize(s) != cudaSuccess)
        st = QMLP_ERR_CUDA;
    if (st != QMLP_OK) {
        cudaStreamSynchronize(s);
        h->mem.release();
        delete h;
        return st;
    }
    *out = h;
    return QMLP_OK;
}

void qmlp_adamw_destroy(qmlp_adamw_t* h) {
    if (!h) return;
    cudaDeviceSynchronize();
    h->mem.release();
    delete h;
}

qmlp_status qmlp_adamw_step(qmlp_adamw_t* h, const qmlp_adamw_hyper* y, qmlp_stream_t stream) {
    if (!h || !y) return QMLP_ERR_INVALID_ARG;
    if (y->step < 1 || !(y->beta1 >= 0 && y->beta1 < 1) || !(y->beta2 >= 0 && y->beta2 < 1) || !isfinite(y->lr) ||
        !isfinite(y->eps) || !isfinite(y->weight_decay) || !isfinite(y->grad_scale))
        return QMLP_ERR_INVALID_ARG;
    if (fault("launch")) return QMLP_ERR_CUDA;
    AdamWStep k;
    k.gscale = (float)y->grad_scale;
    k.b1 = (float)y->beta1;
    k.omb1 = (float)(1.0 - y->beta1);
    k.b2 = (float)y->beta2;
    k.omb2 = (float)(1.0 - y->beta2);
    k.rbc2 = (float)(1.0 / sqrt(1.0 - pow(y->beta2, (double)y->step)));
    k.eps = (float)y->eps;
    k.decay = (float)(1.0 - y->lr * y->weight_decay);
    k.step = (float)(y->lr / (1.0 - pow(y->beta1, (double)y->step)));
    return launch_adamw(h->chunks, h->count, h->param_bf16, h->master, h->grad_bf16, h->s8, k,
                        reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QMLP_OK
               : QMLP_ERR_CUDA;
}

}  // extern "C"
