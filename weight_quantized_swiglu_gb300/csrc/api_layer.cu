// api_layer.cu -- the C ABI of the operators around the quantized blocks of a
// decoder layer (declared in include/qmlp.h): the norms before and after a block,
// one projection with 4-bit weights, a whole mixture-of-experts layer.
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

struct qmlp_linear_s {
    int group = 16, N = 0, K = 0, max_M = 0, num_sms = 0;
    uint8_t* w = nullptr;
    size_t w_bytes = 0;
    float factor = 1.0f;
    float* bias = nullptr;
    // max_M >= kLinearGemmM: the tensor-core GEMM, `slab` rows of W at a time
    int slab = 0;
    float* factors = nullptr;  // [N rounded up to 256]
    uint8_t* img = nullptr;
    size_t img_bytes = 0;
    void* a16 = nullptr;       // fp16 [max_M, K]: bf16 tokens times a power of two each
    int* sig = nullptr;        // [max_M]
    float* ws = nullptr;       // shares of split tiles
    int* err = nullptr;        // device error word
    void* xf = nullptr;        // few tokens: x in the order of the products
    size_t xf_bytes = 0;
    Owner mem;
};

constexpr size_t kLinearImages = (size_t)1 << 30;  // bytes of images that a handle holds at most

struct qmlp_moe_layer_s {
    qmlp_moe_t* moe = nullptr;
    int max_tokens = 0;
    MoeLayerArgs a;  // everything but the call's own
    Owner mem;
};

namespace {

size_t dt_bytes(qmlp_dtype t) { return t == QMLP_DT_FP32 ? 4 : 2; }
int dt_code(qmlp_dtype t) { return t == QMLP_DT_FP32 ? 0 : t == QMLP_DT_BF16 ? 1 : 2; }
bool half_type(qmlp_dtype t) { return t == QMLP_DT_BF16 || t == QMLP_DT_FP16; }
// fp32 or the other 16-bit type
bool same_or_fp32(qmlp_dtype t, qmlp_dtype of) { return t == of || t == QMLP_DT_FP32; }

// Waits for the stream, reports and clears a recorded give-up of a bounded wait.
qmlp_status check_word(int* err, qmlp_stream_t stream) {
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return QMLP_ERR_CUDA;
    int v = 0;
    if (!err) return QMLP_OK;
    if (cudaMemcpy(&v, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return QMLP_ERR_CUDA;
    if (v == 0) return QMLP_OK;
    cudaMemset(err, 0, sizeof(int));
    return QMLP_ERR_DEVICE_TIMEOUT;
}

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
    a.num_sms = h->num_sms;
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
        c.a.vec = c.aligned_all;
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
        // the arrays of a forward in place: its residual is gone
        if (io->residual && io->residual_out &&
            overlaps(io->residual, n * dt_bytes(d.rdt), io->residual_out, n * dt_bytes(d.rdt)))
            return QMLP_ERR_ALIAS;
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
        a.vec = c.aligned_all;
        return from_cuda(launch_norm(a, d.dt == QMLP_DT_FP16, d.rdt == QMLP_DT_FP32, true,
                                     reinterpret_cast<cudaStream_t>(stream)));
    });
}

// ---------------------------------------------------------------------------
// One projection with 4-bit weights and group scales
// ---------------------------------------------------------------------------
qmlp_status qmlp_linear_create(qmlp_linear_t** out, const qmlp_linear_desc* d, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        if (!out) return QMLP_ERR_INVALID_ARG;
        *out = nullptr;
        if (!d || !d->w || !d->scale || (d->fmt != QMLP_LINEAR_NVFP4 && d->fmt != QMLP_LINEAR_INT4))
            return QMLP_ERR_INVALID_ARG;
        const bool nv = d->fmt == QMLP_LINEAR_NVFP4;
        if ((d->zero != nullptr) == nv || (nv ? d->group != 16 : d->group != 32 && d->group != 64 && d->group != 128) ||
            (nv && (d->global_scale == 0.0f || !isfinite(d->global_scale))))
            return QMLP_ERR_INVALID_ARG;
        if (d->N < 1 || d->N > (1 << 20) || d->K < 16 || d->K > 65536 || d->K % d->group || d->max_M < 1 ||
            d->max_M > 65536)
            return QMLP_ERR_SHAPE;
        int dev = 0, sms = 0;
        qmlp_status st = check_device(&dev, &sms);
        if (st != QMLP_OK) return st;
        qmlp_linear_t* h = new qmlp_linear_t();
        Owner tmp;  // the checkpoint's arrays on the device, while they are reordered
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        h->group = d->group;
        h->N = d->N;
        h->K = d->K;
        h->max_M = d->max_M;
        h->num_sms = sms;
        h->factor = nv ? (float)(1.0 / (double)d->global_scale) : 1.0f;
        h->w_bytes = linear_bytes(d->group, d->N, d->K);
        const size_t rows = (size_t)d->N, groups = rows * (d->K / d->group);
        cudaError_t e = cudaSuccess;
        auto stage = [&](const void* src, size_t bytes) -> void* {
            void* p = nullptr;
            if (src && e == cudaSuccess && (e = tmp.alloc(&p, bytes)) == cudaSuccess)
                e = cudaMemcpyAsync(p, src, bytes, cudaMemcpyDefault, s);
            return p;
        };
        const void* w = stage(d->w, rows * (d->K / 2));
        const void* sc = stage(d->scale, groups * (nv ? 1 : 2));
        const void* z = stage(d->zero, groups);
        if (e == cudaSuccess) e = h->mem.alloc(reinterpret_cast<void**>(&h->w), h->w_bytes);
        if (e == cudaSuccess) e = h->mem.alloc(reinterpret_cast<void**>(&h->err), 16);
        if (e == cudaSuccess) e = cudaMemsetAsync(h->err, 0, 16, s);
        if (d->max_M > kLinearFew) {
            h->xf_bytes = linear_x_bytes(d->K, d->max_M);
            if (e == cudaSuccess) e = h->mem.alloc(&h->xf, h->xf_bytes);
            if (e == cudaSuccess) e = h->mem.alloc(reinterpret_cast<void**>(&h->sig), (size_t)d->max_M * 4);
        }
        if (e == cudaSuccess && d->bias) {
            e = h->mem.alloc(reinterpret_cast<void**>(&h->bias), rows * 4);
            if (e == cudaSuccess) e = cudaMemcpyAsync(h->bias, d->bias, rows * 4, cudaMemcpyDefault, s);
        }
        if (e == cudaSuccess)
            e = repack_linear(d->group, static_cast<const uint8_t*>(w), sc, static_cast<const uint8_t*>(z), d->N, d->K,
                              h->w, s);
        if (d->max_M >= kLinearGemmM) {
            const int padded = (d->N + 255) / 256 * 256, Kp = (d->K + 63) / 64 * 64;
            h->slab = (int)std::max<size_t>(256, std::min<size_t>(padded, kLinearImages / (2 * (size_t)Kp) / 256 * 256));
            h->img_bytes = gemm_decoded_bytes(h->slab, Kp);
            const size_t need[4] = {(size_t)padded * 4, h->img_bytes, (size_t)d->max_M * d->K * 2,
                                    gemm_splitk_ws_elems(sms) * 4};
            void** dst[4] = {reinterpret_cast<void**>(&h->factors), reinterpret_cast<void**>(&h->img), &h->a16,
                             reinterpret_cast<void**>(&h->ws)};
            for (int i = 0; i < 4 && e == cudaSuccess; ++i) e = h->mem.alloc(dst[i], need[i]);
            if (e == cudaSuccess) e = launch_linear_factors(d->group, sc, d->N, d->K, h->factor, h->factors, padded, s);
        }
        const cudaError_t e2 = cudaStreamSynchronize(s);
        tmp.release();
        if (e == cudaSuccess) e = e2;
        if (e != cudaSuccess) {
            h->mem.release();
            delete h;
            return from_cuda(e);
        }
        *out = h;
        return QMLP_OK;
    });
}

void qmlp_linear_destroy(qmlp_linear_t* h) {
    if (!h) return;
    cudaDeviceSynchronize();
    h->mem.release();
    delete h;
}

qmlp_status qmlp_linear_forward(qmlp_linear_t* h, const void* x, qmlp_dtype xdt, int M, void* out, qmlp_dtype odt,
                                qmlp_stream_t stream) {
    if (!h || !x || !out || !half_type(xdt) || (!half_type(odt) && odt != QMLP_DT_FP32)) return QMLP_ERR_INVALID_ARG;
    if (M < 1 || M > h->max_M) return QMLP_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(out)) return QMLP_ERR_ALIGNMENT;
    if (overlaps(out, (size_t)M * h->N * dt_bytes(odt), x, (size_t)M * h->K * 2)) return QMLP_ERR_ALIAS;
    if (fault("launch")) return QMLP_ERR_CUDA;
    LinearArgs a;
    a.M = M;
    a.N = h->N;
    a.K = h->K;
    a.w = h->w;
    a.w_bytes = h->w_bytes;
    a.factor = h->factor;
    a.bias = h->bias;
    a.x = x;
    a.x_bf16 = xdt == QMLP_DT_BF16;
    a.out = out;
    a.odt = dt_code(odt);
    a.err = h->err;
    a.xf = h->xf;
    a.xf_elems = h->xf_bytes / 16;
    a.sig = h->sig;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M < kLinearGemmM) return from_cuda(launch_linear(h->group, a, h->num_sms, s));
    // many tokens: the weights decoded once into stage images, rows of W in slabs
    const int Kp = (h->K + 63) / 64 * 64;
    for (int n0 = 0; n0 < h->N; n0 += h->slab) {
        const int rows = std::min(h->slab, (h->N - n0 + 255) / 256 * 256), cols = std::min(h->slab, h->N - n0);
        cudaError_t e = launch_linear_images(h->group, h->w, h->w_bytes, h->factors, h->N, h->K, n0, rows, false, h->img,
                                             h->img_bytes, s);
        if (e != cudaSuccess) return from_cuda(e);
        GemmLaunch g;
        g.epi = kEpiOut;
        g.w.fmt = kFP8;
        g.w.N = rows;
        g.w.K = Kp;
        g.w.cs0 = h->factors + n0;
        g.a = x;
        g.M = M;
        g.out = static_cast<uint8_t*>(out) + (size_t)n0 * dt_bytes(odt);
        g.ldo = h->N;
        g.ncols = cols;
        g.odt = a.odt;
        g.bias = h->bias ? h->bias + n0 : nullptr;
        g.ka = h->K;
        // (the activations are scaled once, before the first slab)
        g.unscaled = !a.x_bf16;
        g.prescaled = !a.x_bf16 || n0 > 0;
        g.a16 = a.x_bf16 ? h->a16 : const_cast<void*>(x);
        g.sig = h->sig;
        g.err = h->err;
        g.ws = h->ws;
        g.pair = true;
        g.wdec = h->img;
        g.wdec_bytes = h->img_bytes;
        g.f16 = true;
        g.split_tail = true;
        g.images_ready = true;
        if ((e = launch_gemm(g, h->num_sms, s)) != cudaSuccess) return from_cuda(e);
        if (h->group == 16 || a.odt != 0) continue;
        // INT4 into fp32: what the images' rounding to fp16 left, a second product on top
        e = launch_linear_images(h->group, h->w, h->w_bytes, h->factors, h->N, h->K, n0, rows, true, h->img, h->img_bytes, s);
        if (e != cudaSuccess) return from_cuda(e);
        g.bias = nullptr;
        g.prescaled = true;
        g.onto = true;
        if ((e = launch_gemm(g, h->num_sms, s)) != cudaSuccess) return from_cuda(e);
    }
    return QMLP_OK;
}

qmlp_status qmlp_linear_check(qmlp_linear_t* h, qmlp_stream_t stream) {
    if (!h) return QMLP_ERR_INVALID_ARG;
    return check_word(h->err, stream);
}

// ---------------------------------------------------------------------------
// A whole mixture-of-experts layer
// ---------------------------------------------------------------------------
qmlp_status qmlp_moe_layer_create(qmlp_moe_layer_t** out, qmlp_moe_t* moe, const qmlp_moe_layer_desc* d,
                                  qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        if (!out) return QMLP_ERR_INVALID_ARG;
        *out = nullptr;
        if (!moe || !d || !d->router || (!half_type(d->rdt) && d->rdt != QMLP_DT_FP32) ||
            (d->score != QMLP_SCORE_SOFTMAX && d->score != QMLP_SCORE_SIGMOID) || !isfinite(d->route_scale) ||
            (d->shared_gate && d->shared < 1))
            return QMLP_ERR_INVALID_ARG;
        const int E = moe->E - d->shared, nsel = d->topk + d->shared;
        if (d->shared < 0 || E < 1 || E > kMoeLayerMaxE || d->topk < 1 || d->topk > E || nsel > 16 ||
            d->max_tokens < 1 || d->max_tokens > (1 << 20))
            return QMLP_ERR_SHAPE;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        // the grouped kernels' workspace; what it does not take is no fault where every
        // number of tokens is the one kernel's
        bool one = d->max_tokens <= kMoeLayerFew;
        for (int m = 1; one && m <= d->max_tokens; ++m) one = moe_layer_few(m, moe->K, moe->I, E, d->shared, d->topk, moe->meta);
        if (d->max_tokens > 1) {
            const size_t bytes = one ? moe->g_bytes : std::max<size_t>(moe->g_bytes, 4 * (size_t)nsel);
            const qmlp_status st = moe_reserve(moe, d->max_tokens, bytes, s);
            if (st != QMLP_OK && !(one && st == QMLP_ERR_SHAPE)) return st;
        }
        qmlp_moe_layer_t* h = new qmlp_moe_layer_t();
        h->moe = moe;
        h->max_tokens = d->max_tokens;
        MoeLayerArgs& a = h->a;
        a.E = E;
        a.S = d->shared;
        a.K = moe->K;
        a.I = moe->I;
        a.topk = d->topk;
        a.softmax = d->score == QMLP_SCORE_SOFTMAX;
        a.renorm = d->renorm != 0;
        a.rscale = d->route_scale;
        a.sgate = d->shared_gate != nullptr;
        a.planes = d->rdt == QMLP_DT_FP32 ? 2 : 1;
        a.rtiles = (E + (a.sgate ? a.S : 0) + 15) / 16;
        a.rfrag_elems = (size_t)a.planes * a.rtiles * (a.K / 32) * 64;
        a.w13 = moe->w13;
        a.w13_meta = moe->w13_meta;
        a.w2 = moe->w2;
        a.w2_meta = moe->w2_meta;
        const size_t few = (size_t)std::min(d->max_tokens, kMoeLayerFew) * nsel, rows = (size_t)d->max_tokens;
        a.logit_elems = std::max(rows, (size_t)kMoeRouterSplits * std::min(d->max_tokens, kMoeLayerFew)) * (E + a.S);
        a.act_elems = few * a.I;
        a.w13_bytes = moe_w13_bank_bytes(moe->E, a.I, a.K);
        a.w13_meta_bytes = moe_w13_meta_bank_bytes(moe->E, a.I, a.K, moe->meta);
        a.w2_bytes = (size_t)moe->E * a.K * (a.I / 2);
        a.w2_meta_bytes = (size_t)moe->E * a.K * (a.I / 32) * moe->meta;
        cudaError_t e = cudaSuccess;
        auto make = [&](size_t bytes, const void* src) -> void* {
            void* p = nullptr;
            if (e == cudaSuccess && (e = h->mem.alloc(&p, bytes)) == cudaSuccess && src)
                e = cudaMemcpyAsync(p, src, bytes, cudaMemcpyDefault, s);
            return p;
        };
        const size_t re = dt_bytes(d->rdt) * a.K;
        Owner tmp;  // the router as given, while it is laid out
        auto stage = [&](size_t bytes, const void* src) -> void* {
            void* p = nullptr;
            if (src && e == cudaSuccess && (e = tmp.alloc(&p, bytes)) == cudaSuccess)
                e = cudaMemcpyAsync(p, src, bytes, cudaMemcpyDefault, s);
            return p;
        };
        const void* w = stage(re * E, d->router);
        const void* sg = stage(re * a.S, d->shared_gate);
        uint4* frag = static_cast<uint4*>(make(a.rfrag_elems * 16, nullptr));
        int* rexp = static_cast<int*>(make((size_t)a.rtiles * 16 * 4, nullptr));
        if (e == cudaSuccess) e = launch_router_layout(a, w, sg, dt_code(d->rdt), frag, rexp, s);
        a.rfrag = frag;
        a.rexp = rexp;
        if (d->bias) a.bias = static_cast<float*>(make((size_t)E * 4, d->bias));
        a.logits = static_cast<float*>(make(a.logit_elems * 4, nullptr));
        a.ids = static_cast<int32_t*>(make(rows * nsel * 4, nullptr));
        a.weights = static_cast<float*>(make(rows * nsel * 4, nullptr));
        a.act = static_cast<float*>(make(a.act_elems * 4, nullptr));
        a.amax = static_cast<int*>(make(rows * nsel * 4, nullptr));
        a.act16_elems = a.act_elems / 8 * 2;  // (twice: what rounding to fp16 leaves)
        a.act16 = static_cast<uint4*>(make(a.act16_elems * 16, nullptr));
        uint8_t* words = static_cast<uint8_t*>(make(16, nullptr));
        if (e == cudaSuccess) e = cudaMemsetAsync(words, 0, 16, s);
        a.ticket = reinterpret_cast<unsigned long long*>(words);
        a.err = reinterpret_cast<int*>(words + 8);
        const cudaError_t e2 = cudaStreamSynchronize(s);
        tmp.release();
        if (e == cudaSuccess) e = e2;
        if (e != cudaSuccess) {
            h->mem.release();
            delete h;
            return from_cuda(e);
        }
        *out = h;
        return QMLP_OK;
    });
}

void qmlp_moe_layer_destroy(qmlp_moe_layer_t* h) {
    if (!h) return;
    cudaDeviceSynchronize();
    h->mem.release();
    delete h;
}

qmlp_status qmlp_moe_layer_forward(qmlp_moe_layer_t* h, const void* x, qmlp_dtype xdt, int M, void* out, qmlp_dtype odt,
                                   int32_t* ids, float* weights, qmlp_stream_t stream) {
    if (!h || !x || !out || !half_type(xdt) || (!half_type(odt) && odt != QMLP_DT_FP32)) return QMLP_ERR_INVALID_ARG;
    if (M < 1 || M > h->max_tokens) return QMLP_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(out) || !aligned(ids, 4) || !aligned(weights, 4)) return QMLP_ERR_ALIGNMENT;
    MoeLayerArgs a = h->a;
    const size_t n = (size_t)M * a.K, c = (size_t)M * a.topk * 4;
    const void* p[4] = {out, x, ids, weights};
    const size_t bytes[4] = {n * dt_bytes(odt), n * 2, c, c};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (p[i] && p[j] && overlaps(p[i], bytes[i], p[j], bytes[j])) return QMLP_ERR_ALIAS;
    if (fault("launch")) return QMLP_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.M = M;
    a.x = x;
    a.x_bf16 = xdt == QMLP_DT_BF16;
    a.out = out;
    a.odt = dt_code(odt);
    a.ids_out = ids;
    a.w_out = weights;
    if (moe_layer_few(M, a.K, a.I, a.E, a.S, a.topk, h->moe->meta))
        return from_cuda(launch_moe_layer_few(a, h->moe->meta, h->moe->num_sms, s));
    cudaError_t e = launch_moe_router(a, s);
    if (e == cudaSuccess)
        e = moe_grouped(h->moe, x, a.x_bf16, a.ids, a.weights, a.topk + a.S, M, out, a.odt, a.amax, s);
    return from_cuda(e);
}

qmlp_status qmlp_moe_layer_check(qmlp_moe_layer_t* h, qmlp_stream_t stream) {
    if (!h) return QMLP_ERR_INVALID_ARG;
    return check_word(h->a.err, stream);
}

}  // extern "C"
