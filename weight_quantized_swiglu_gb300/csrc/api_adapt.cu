// api_adapt.cu -- the C ABI of training and serving adapters beside the
// frozen quantized weights (declared in include/qmlp.h): AdamW over many
// tensors. Argument checks, ownership and dispatch only, as api.cu.
#include <math.h>

#include "handle.h"
#include "lowrank.cuh"

using namespace qmlp;

// The padded copies of adapters and the workspace of their products.
struct qmlp_lora_s {
    qmlp_t* h = nullptr;
    int slots = 0, max_rank = 0, Rp = 0;  // Rp: 16, 32 or 64
    __nv_bfloat16* a_gu = nullptr;  // [slots][2][Rp][K]
    __nv_bfloat16* a_d = nullptr;   // [slots][Rp][I]
    __nv_bfloat16* b_gu = nullptr;  // [slots][2][I][Rp]
    __nv_bfloat16* b_d = nullptr;   // [slots][K][Rp]
    float* scale = nullptr;         // [slots]
    int* rank = nullptr;            // [slots], 0: empty
    float* v = nullptr;             // few tokens: [kLrFew][2 Rp]
    __nv_bfloat16* vw = nullptr;    // [kLrWords][max_M][2 Rp], by position
    float* y = nullptr;             // [max_M][max(2I, K)]: the adapters' terms
    float* raw = nullptr;           // [kLrFew][2I + K]: projections without their factors
    int* perm = nullptr;
    int4* tiles = nullptr;
    int* n_tiles = nullptr;
    float* part = nullptr;
    int* cnt = nullptr;
    Owner mem;
};

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

qmlp_status check_adapter(const qmlp_adapter* a, int max_rank) {
    const void* p[6] = {a->gate_a, a->gate_b, a->up_a, a->up_b, a->down_a, a->down_b};
    for (int i = 0; i < 6; i += 2)
        if ((p[i] != nullptr) != (p[i + 1] != nullptr)) return QMLP_ERR_INVALID_ARG;
    if (a->rank < 1 || a->rank > max_rank) return QMLP_ERR_SHAPE;
    for (const void* q : p)
        if (!aligned(q, 2)) return QMLP_ERR_ALIGNMENT;
    return QMLP_OK;
}

// The adapter's arrays as the pack kernel's parts (A of gate, up, down, then
// B), into a slot of l.
LrPack pack_of(const qmlp_lora_s* l, int slot, const qmlp_adapter* a) {
    const size_t K = l->h->K, I = l->h->I, R = l->Rp;
    LrPack p;
    using B = __nv_bfloat16;
    auto src = [](const void* q) { return static_cast<const B*>(q); };
    const B* s[6] = {src(a->gate_a), src(a->up_a), src(a->down_a), src(a->gate_b), src(a->up_b), src(a->down_b)};
    B* d[6] = {l->a_gu + slot * 2 * R * K, l->a_gu + (slot * 2 + 1) * R * K, l->a_d + slot * R * I,
               l->b_gu + slot * 2 * I * R, l->b_gu + (slot * 2 + 1) * I * R, l->b_d + slot * K * R};
    const int rows[6] = {(int)R, (int)R, (int)R, (int)I, (int)I, (int)K};
    const int cols[6] = {(int)K, (int)K, (int)I, (int)R, (int)R, (int)R};
    for (int i = 0; i < 6; ++i) {
        p.part[i].src = s[i];
        p.part[i].dst = d[i];
        p.part[i].rows = rows[i];
        p.part[i].cols = cols[i];
    }
    p.r = a->rank;
    p.scale = a->scale;
    p.rank_out = l->rank + slot;
    p.scale_out = l->scale + slot;
    return p;
}

// The products of a call's adapters. down: of act, else gate and up of x.
LrTokens tokens_of(const qmlp_lora_s* l, int M) {
    LrTokens t;
    t.tiles = l->tiles;
    t.n_tiles = l->n_tiles;
    t.perm = l->perm;
    t.M = M;
    return t;
}
cudaError_t lora_shrink(const qmlp_lora_s* l, bool down, const void* z, int M, cudaStream_t s) {
    LrShrink a;
    a.tok = tokens_of(l, M);
    a.x = static_cast<const __nv_bfloat16*>(z);
    a.D = down ? l->h->I : l->h->K;
    a.ldx = a.D;
    a.w = down ? l->a_d : l->a_gu;
    a.w_slot = (size_t)(down ? 1 : 2) * l->Rp * a.D;
    a.scale = l->scale;
    a.v = l->vw;
    a.v_word = (size_t)l->h->max_M * 2 * l->Rp;
    a.ldv = (down ? 1 : 2) * l->Rp;
    a.part = l->part;
    a.cnt = l->cnt;
    return launch_lr_shrink(a, a.ldv, false, lr_max_tiles(M, l->slots), 1, l->h->num_sms, s);
}
cudaError_t lora_expand(const qmlp_lora_s* l, bool down, int M, cudaStream_t s) {
    LrExpand a;
    a.tok = tokens_of(l, M);
    a.v = l->vw;
    a.v_word = (size_t)l->h->max_M * 2 * l->Rp;
    a.ldv = (down ? 1 : 2) * l->Rp;
    a.N = down ? l->h->K : l->h->I;
    a.w = down ? l->b_d : l->b_gu;
    a.w_z = (size_t)a.N * l->Rp;
    a.w_slot = (down ? 1 : 2) * a.w_z;
    a.y = l->y;
    a.ldy = (size_t)(down ? 1 : 2) * a.N;
    return launch_lr_expand(a, l->Rp, false, lr_max_tiles(M, l->slots), down ? 1 : 2, s);
}
LrFew few_of(const qmlp_lora_s* l, bool down, const int32_t* ids) {
    LrFew a;
    a.ids = ids;
    a.rank = l->rank;
    a.scale = l->scale;
    a.slots = l->slots;
    a.Rp = l->Rp;
    a.ncol = (down ? 1 : 2) * l->Rp;
    a.v = l->v;
    return a;
}
cudaError_t lora_shrink_few(const qmlp_lora_s* l, bool down, const void* z, const int32_t* ids, int M, cudaStream_t s) {
    LrFew a = few_of(l, down, ids);
    a.x = static_cast<const __nv_bfloat16*>(z);
    a.D = down ? l->h->I : l->h->K;
    a.w = down ? l->a_d : l->a_gu;
    a.w_slot = (size_t)a.ncol * a.D;
    return launch_lr_shrink_few(a, M, s);
}
// out: the block's output from down's raw projection; else the terms into y.
cudaError_t lora_expand_few(const qmlp_lora_s* l, bool down, const int32_t* ids, int M, const float* raw, void* out,
                            cudaStream_t s) {
    LrFew a = few_of(l, down, ids);
    a.D = down ? l->h->K : l->h->I;
    a.w = down ? l->b_d : l->b_gu;
    a.w_slot = (size_t)a.ncol * a.D;
    a.y = l->y;
    a.ldy = (size_t)(down ? 1 : 2) * a.D;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.raw = raw;
    a.factor = l->h->gv[2].chs;
    a.factor_all = l->h->gv[2].inv_g;
    return launch_lr_expand_few(a, M, down ? 1 : 2, s);
}

// One block of at most kLrFew tokens on the GEMV kernels.
qmlp_status lora_block(qmlp_lora_s* l, const void* x, const int32_t* ids, int M, void* out, cudaStream_t s) {
    qmlp_t* h = l->h;
    if (lora_shrink_few(l, false, x, ids, M, s) != cudaSuccess ||
        lora_expand_few(l, false, ids, M, nullptr, nullptr, s) != cudaSuccess)
        return QMLP_ERR_CUDA;
    float* raw_d = l->raw;
    if (h->sp.G && M <= split_max_m(h) && split_fits(h->fmt, M, h->K, h->sp)) {
        SplitLaunch S = split_launch(h, x, M);
        S.add = l->y;
        S.out_f32 = raw_d;
        if (launch_split(S, h->sp, s) != cudaSuccess) return QMLP_ERR_CUDA;
    } else {
        // the two projections on their own, then the activation
        float* rg = l->raw + (size_t)kLrFew * h->K;
        float* ru = rg + (size_t)kLrFew * h->I;
        qmlp_status st = qmlp_debug_project(h, 0, QMLP_PATH_GEMV, x, M, rg, s);
        if (st == QMLP_OK) st = qmlp_debug_project(h, 1, QMLP_PATH_GEMV, x, M, ru, s);
        if (st != QMLP_OK) return st;
        LrSwiGLU a;
        a.raw_g = rg;
        a.raw_u = ru;
        a.y = l->y;
        a.fg = h->gv[0].chs;
        a.fu = h->gv[1].chs;
        a.fg_all = h->gv[0].inv_g;
        a.fu_all = h->gv[1].inv_g;
        a.act = static_cast<__nv_bfloat16*>(h->act);
        a.M = M;
        a.I = h->I;
        if (launch_lr_swiglu_raw(a, s) != cudaSuccess) return QMLP_ERR_CUDA;
        st = qmlp_debug_project(h, 2, QMLP_PATH_GEMV, h->act, M, raw_d, s);
        if (st != QMLP_OK) return st;
    }
    if (lora_shrink_few(l, true, h->act, ids, M, s) != cudaSuccess ||
        lora_expand_few(l, true, ids, M, raw_d, out, s) != cudaSuccess)
        return QMLP_ERR_CUDA;
    return QMLP_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// low-rank adapters
// ---------------------------------------------------------------------------
qmlp_status qmlp_lora_create(qmlp_lora_t** out, qmlp_t* h, int slots, int max_rank, qmlp_stream_t stream) {
    if (!out) return QMLP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!h) return QMLP_ERR_INVALID_ARG;
    if (slots < 1 || slots > kLrMaxSlots || max_rank < 1 || max_rank > kLrMaxRank) return QMLP_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    qmlp_lora_t* l = new qmlp_lora_t();
    l->h = h;
    l->slots = slots;
    l->max_rank = max_rank;
    l->Rp = max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : 64;
    const size_t K = h->K, I = h->I, R = l->Rp, S = slots, M = h->max_M;
    const size_t tiles = (size_t)lr_max_tiles(h->max_M, slots);
    cudaError_t e = cudaSuccess;
    auto get = [&](auto** p, size_t count, bool zero) {
        if (e != cudaSuccess) return;
        const size_t bytes = count * sizeof(**p);
        if ((e = l->mem.alloc(reinterpret_cast<void**>(p), bytes)) == cudaSuccess && zero) e = cudaMemsetAsync(*p, 0, bytes, s);
    };
    get(&l->a_gu, S * 2 * R * K, true);
    get(&l->a_d, S * R * I, true);
    get(&l->b_gu, S * 2 * I * R, true);
    get(&l->b_d, S * K * R, true);
    get(&l->scale, S, true);
    get(&l->rank, S, true);
    get(&l->v, (size_t)kLrFew * 2 * R, false);
    get(&l->vw, kLrWords * M * 2 * R, false);
    get(&l->y, M * std::max(2 * I, K), false);
    get(&l->raw, (size_t)kLrFew * (2 * I + K), false);
    get(&l->perm, M, false);
    get(&l->tiles, tiles, false);
    get(&l->n_tiles, 1, true);
    get(&l->part, lr_part_elems(h->num_sms), false);
    get(&l->cnt, tiles * 2, true);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) {
        cudaStreamSynchronize(s);
        l->mem.release();
        delete l;
        return from_cuda(e);
    }
    *out = l;
    return QMLP_OK;
}

void qmlp_lora_destroy(qmlp_lora_t* l) {
    if (!l) return;
    cudaDeviceSynchronize();
    l->mem.release();
    delete l;
}

qmlp_status qmlp_lora_set(qmlp_lora_t* l, int slot, const qmlp_adapter* a, qmlp_stream_t stream) {
    if (!l || slot < 0 || slot >= l->slots) return QMLP_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!a) return cudaMemsetAsync(l->rank + slot, 0, sizeof(int), s) == cudaSuccess ? QMLP_OK : QMLP_ERR_CUDA;
    const qmlp_status st = check_adapter(a, l->max_rank);
    if (st != QMLP_OK) return st;
    if (fault("launch")) return QMLP_ERR_CUDA;
    return launch_lr_pack(pack_of(l, slot, a), s) == cudaSuccess ? QMLP_OK : QMLP_ERR_CUDA;
}

qmlp_status qmlp_lora_forward(qmlp_lora_t* l, const void* x, const int32_t* ids, int M, void* out,
                              qmlp_stream_t stream) {
    if (!l || !x || !ids || !out) return QMLP_ERR_INVALID_ARG;
    qmlp_t* h = l->h;
    if (M < 1 || M > h->max_M) return QMLP_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(out) || !aligned(ids, 4)) return QMLP_ERR_ALIGNMENT;
    const size_t xb = (size_t)M * h->K * 2, ab = (size_t)h->max_M * h->I * 2;
    if (overlaps(out, xb, x, xb) || overlaps(out, xb, ids, (size_t)M * 4) || overlaps(out, xb, h->act, ab))
        return QMLP_ERR_ALIAS;
    if (fault("launch")) return QMLP_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!(h->has_gemm && M >= gemm_min_m(h))) {
        const int block = h->sp.G ? split_max_m(h) : kLrFew;
        for (int m0 = 0; m0 < M; m0 += block) {
            const qmlp_status st =
                lora_block(l, static_cast<const uint8_t*>(x) + (size_t)m0 * h->K * 2, ids + m0, std::min(block, M - m0),
                           static_cast<uint8_t*>(out) + (size_t)m0 * h->K * 2, s);
            if (st != QMLP_OK) return st;
        }
        return QMLP_OK;
    }
    const bool few = M <= kLrFew;
    auto terms = [&](bool down, const void* z, cudaStream_t st) {
        cudaError_t e = few ? lora_shrink_few(l, down, z, ids, M, st) : lora_shrink(l, down, z, M, st);
        if (e == cudaSuccess)
            e = few ? lora_expand_few(l, down, ids, M, nullptr, nullptr, st) : lora_expand(l, down, M, st);
        return e;
    };
    if (!few && launch_lr_plan(ids, M, l->slots, l->rank, l->perm, l->tiles, l->n_tiles, s) != cudaSuccess)
        return QMLP_ERR_CUDA;
    if (terms(false, x, s) != cudaSuccess) return QMLP_ERR_CUDA;
    GemmTerms t;
    t.add = l->y;
    t.add_down = l->y;
    t.between = [&](cudaStream_t st) { return terms(true, h->act, st); };
    return run_gemm(h, QMLP_PATH_AUTO, 3, x, M, out, s, nullptr, &t);
}

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
