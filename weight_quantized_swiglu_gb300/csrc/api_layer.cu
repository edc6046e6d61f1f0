// api_layer.cu -- the C ABI of the operators around the quantized blocks of a
// decoder layer (declared in include/qmlp.h): the norms before and after a block.
// Argument checks, ownership and dispatch only, as api.cu.
#include <math.h>

#include "handle.h"

using namespace qmlp;

struct qmlp_norm_s {
    qmlp_norm_desc d;
    int num_sms = 0;
    float* part = nullptr;  // [shares][3][K]: column sums of the backward pass's CTAs
    int shares = 0;
    Owner mem;
};

namespace {

size_t dt_bytes(qmlp_dtype t) { return t == QMLP_DT_FP32 ? 4 : 2; }
bool half_type(qmlp_dtype t) { return t == QMLP_DT_BF16 || t == QMLP_DT_FP16; }
// fp32 or the other 16-bit type
bool same_or_fp32(qmlp_dtype t, qmlp_dtype of) { return t == of || t == QMLP_DT_FP32; }

Range range(const void* p, size_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes, written};
}

// The checks and arguments that forward and backward share.
struct NormCall {
    NormArgs a;
    std::vector<Range> ranges;
    bool aligned_all = true;  // every pointer for 8 elements at a time

    qmlp_status add(const void* p, qmlp_dtype t, size_t n, bool written) {
        if (!p) return QMLP_OK;
        if (!aligned(p, dt_bytes(t))) return QMLP_ERR_ALIGNMENT;
        aligned_all = aligned_all && aligned16(p);
        ranges.push_back(range(p, n * dt_bytes(t), written));
        return QMLP_OK;
    }
};

qmlp_status norm_call(const qmlp_norm_t* h, const qmlp_norm_io* io, int M, bool backward, NormCall& c) {
    if (!h || !io) return QMLP_ERR_INVALID_ARG;
    const qmlp_norm_desc& d = h->d;
    if (M < 1) return QMLP_ERR_SHAPE;
    // something to norm, and a gate exactly where the handle has one
    if ((!io->z && !io->residual) || (!io->post_w && !io->pre_w && !io->z) || (io->post_w && !io->z) ||
        (io->gate != nullptr) != (d.gate != QMLP_GATE_NONE && io->z != nullptr))
        return QMLP_ERR_INVALID_ARG;
    const size_t n = (size_t)M * d.K;
    NormArgs& a = c.a;
    a.M = M;
    a.K = d.K;
    a.eps = d.eps;
    a.rK = 1.0f / (float)d.K;
    a.offset = d.weight_offset;
    a.scale = d.scale;
    a.gate_kind = io->z ? (int)d.gate : kGateNone;
    a.w_f32 = d.wdt == QMLP_DT_FP32;
    a.z = io->z;
    a.r = io->residual;
    a.post_w = io->post_w;
    a.pre_w = io->pre_w;
    a.gate = io->gate;
    a.stats = reinterpret_cast<float2*>(io->stats);
    a.elems = n;
    const size_t gn = d.gate == QMLP_GATE_CHANNEL ? (size_t)d.K : d.gate == QMLP_GATE_TOKEN ? (size_t)M : n;
    qmlp_status st = QMLP_OK;
    auto add = [&](const void* p, qmlp_dtype t, size_t k, bool w) {
        if (st == QMLP_OK) st = c.add(p, t, k, w);
    };
    add(io->z, d.dt, n, false);
    if (backward || io->residual != io->residual_out) add(io->residual, d.rdt, n, false);
    add(io->post_w, d.wdt, d.K, false);
    add(io->pre_w, d.wdt, d.K, false);
    if (d.gate == QMLP_GATE_TOKEN) {  // one value a row: any alignment of its type
        if (io->gate && !aligned(io->gate, 2)) return QMLP_ERR_ALIGNMENT;
        if (io->gate) c.ranges.push_back(range(io->gate, gn * 2, false));
    } else {
        add(io->gate, d.gate == QMLP_GATE_CHANNEL ? d.wdt : d.dt, gn, false);
    }
    if (io->stats) {
        if (!aligned(io->stats, 8)) return QMLP_ERR_ALIGNMENT;
        c.ranges.push_back(range(io->stats, (size_t)M * 8, !backward));
    }
    return st;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Norms before and after a block
// ---------------------------------------------------------------------------
qmlp_status qmlp_norm_create(qmlp_norm_t** out, const qmlp_norm_desc* d, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        if (!out) return QMLP_ERR_INVALID_ARG;
        *out = nullptr;
        if (!d || !half_type(d->dt) || !same_or_fp32(d->rdt, d->dt) || !same_or_fp32(d->wdt, d->dt) ||
            d->gate < QMLP_GATE_NONE || d->gate > QMLP_GATE_FULL || !(d->eps >= 0) || !isfinite(d->eps) ||
            !isfinite(d->weight_offset) || !isfinite(d->scale))
            return QMLP_ERR_INVALID_ARG;
        if (d->K < 1 || d->K > kNormMaxK) return QMLP_ERR_SHAPE;
        int dev = 0, sms = 0;
        qmlp_status st = check_device(&dev, &sms);
        if (st != QMLP_OK) return st;
        qmlp_norm_t* h = new qmlp_norm_t();
        h->d = *d;
        h->num_sms = sms;
        h->shares = 2 * sms;
        const cudaError_t e =
            h->mem.alloc(reinterpret_cast<void**>(&h->part), (size_t)h->shares * 3 * d->K * sizeof(float));
        if (e != cudaSuccess) {
            h->mem.release();
            delete h;
            return from_cuda(e);
        }
        *out = h;
        (void)stream;
        return QMLP_OK;
    });
}

void qmlp_norm_destroy(qmlp_norm_t* h) {
    if (!h) return;
    cudaDeviceSynchronize();
    h->mem.release();
    delete h;
}

qmlp_status qmlp_norm_forward(qmlp_norm_t* h, const qmlp_norm_io* io, int M, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        NormCall c;
        qmlp_status st = norm_call(h, io, M, false, c);
        if (st != QMLP_OK) return st;
        if ((io->pre_w != nullptr) != (io->out != nullptr) || (!io->residual_out && !io->out))
            return QMLP_ERR_INVALID_ARG;
        const size_t n = (size_t)M * h->d.K;
        if ((st = c.add(io->residual_out, h->d.rdt, n, true)) != QMLP_OK ||
            (st = c.add(io->out, h->d.dt, n, true)) != QMLP_OK)
            return st;
        if (any_alias(c.ranges)) return QMLP_ERR_ALIAS;
        if (fault("launch")) return QMLP_ERR_CUDA;
        c.a.h = io->residual_out;
        c.a.y = io->out;
        c.a.vec = c.aligned_all && h->d.K % 8 == 0;
        return from_cuda(launch_norm(c.a, h->d.dt == QMLP_DT_FP16, h->d.rdt == QMLP_DT_FP32, false,
                                     reinterpret_cast<cudaStream_t>(stream)));
    });
}

qmlp_status qmlp_norm_backward(qmlp_norm_t* h, const qmlp_norm_io* io, const qmlp_norm_grads* g, int M,
                               qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        NormCall c;
        qmlp_status st = norm_call(h, io, M, true, c);
        if (st != QMLP_OK) return st;
        const qmlp_norm_desc& d = h->d;
        // an output's gradient for the norm before; gradients only of what is there
        if (!g || !io->stats || (io->pre_w != nullptr) != (g->dout != nullptr) || (!g->dout && !g->dresidual_out) ||
            (g->dz && !io->z) || (g->dresidual && !io->residual) || (g->dpost_w && !io->post_w) ||
            (g->dpre_w && !io->pre_w) || (g->dgate && !io->gate))
            return QMLP_ERR_INVALID_ARG;
        const size_t n = (size_t)M * d.K;
        auto add = [&](const void* p, qmlp_dtype t, size_t k, bool w) {
            if (st == QMLP_OK) st = c.add(p, t, k, w);
        };
        add(g->dout, d.dt, n, false);
        if (g->dresidual_out != g->dresidual) add(g->dresidual_out, d.rdt, n, false);
        add(g->dz, d.dt, n, true);
        add(g->dresidual, d.rdt, n, true);
        add(g->dpost_w, d.wdt, d.K, true);
        add(g->dpre_w, d.wdt, d.K, true);
        if (d.gate == QMLP_GATE_TOKEN && g->dgate) {
            if (!aligned(g->dgate, 2)) return QMLP_ERR_ALIGNMENT;
            c.ranges.push_back(range(g->dgate, (size_t)M * 2, true));
        } else if (d.gate == QMLP_GATE_CHANNEL) {
            add(g->dgate, d.wdt, d.K, true);
        } else {
            add(g->dgate, d.dt, n, true);
        }
        if (st != QMLP_OK) return st;
        if (any_alias(c.ranges)) return QMLP_ERR_ALIAS;
        if (fault("launch")) return QMLP_ERR_CUDA;
        NormArgs& a = c.a;
        a.dy = g->dout;
        a.dh = g->dresidual_out;
        a.dz = g->dz;
        a.dr = g->dresidual;
        a.dpost = g->dpost_w;
        a.dpre = g->dpre_w;
        a.dgate = g->dgate;
        a.shares = h->shares;
        a.part = g->dpost_w || g->dpre_w || (g->dgate && d.gate == QMLP_GATE_CHANNEL) ? h->part : nullptr;
        a.part_elems = (size_t)h->shares * 3 * d.K;
        a.vec = c.aligned_all && d.K % 8 == 0;
        return from_cuda(launch_norm(a, d.dt == QMLP_DT_FP16, d.rdt == QMLP_DT_FP32, true,
                                     reinterpret_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
