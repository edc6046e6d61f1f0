// api_adapt.cu -- the C ABI of serving adapters beside the frozen quantized
// weights, of training through them, and of AdamW over many tensors (declared
// in include/qmlp.h). Argument checks, ownership and dispatch only, as api.cu.
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
    size_t y_elems = 0;
    float* raw = nullptr;           // [kMaxGemvM][2I + K]: projections without their factors
    float* vd = nullptr;            // [G][kMaxGemvM][Rp]: the decode CTAs' shares of A_d act
    int* perm = nullptr;
    int4* tiles = nullptr;
    int* n_tiles = nullptr;
    cudaEvent_t ev = nullptr;
    // From kDqMinM tokens on the terms may be further contraction steps of the
    // GEMMs (see training's Words: T words, the factors divided out): tokens in
    // slot order, the adapters' images made when they are set
    bool steps = false;
    int T = 2, e_gu = 0, e_d = 0;    // steps an entry
    uint8_t* img_gu = nullptr;       // [slots][I / 128][e_gu] and [slots][K / 256][e_d] images of 32 KB
    uint8_t* img_d = nullptr;
    __nv_bfloat16* ev_v = nullptr;   // 256 rows an entry of 64 max(e_gu, e_d)
    size_t ev_elems = 0;
    void* x_rows = nullptr;          // bf16 [max_M][K]
    int2* ents = nullptr;
    int* ent_slot = nullptr;
    int* odd = nullptr;              // [slots]: whether B has values that the images leave out
    int* odd_rows = nullptr;         // [max_M], by position: its slot's
    Owner mem;
};

// The workspace of forward and backward with frozen weights.
struct qmlp_train_s {
    qmlp_t* h = nullptr;
    qmlp_lora_t* l = nullptr;        // one slot: the call's adapter
    uint8_t* img_t = nullptr;        // images of the transposed down projection
    size_t img_t_bytes = 0;
    __nv_bfloat16* bq = nullptr;     // two words of [2][I][Rp]: B of gate and up over the factors
    __nv_bfloat16* dgu = nullptr;    // [max_M][2I]: d gate, d up times their factors
    __nv_bfloat16* dgu_lo = nullptr; // [kTwoWordM][2I]: what their rounding leaves
    __nv_bfloat16* dv = nullptr;     // kLrWords planes of [max_M][2 Rp]
    __nv_bfloat16* dvd = nullptr;    // likewise [max_M][Rp]
    // From kPairMinM tokens on the adapter's terms are further contraction
    // steps of the GEMMs: T words of v beside T of the adapter (see LrImage).
    // NVFP4's one factor a projection goes into v (T = 2); FP8's per-channel
    // ones into the adapter's images (T = 3), if all can be divided by.
    bool steps = true;
    int T = 2;
    cudaEvent_t ev_img = nullptr;    // the images are there (side stream)
    uint8_t* img_gu = nullptr;       // images of B gate/up, B down; of A down, A gate/up
    uint8_t* img_d = nullptr;
    // FP8: the factors that d gate and d up carry (1 where a channel's is too
    // small to divide by: it is then in the weights' image, `row`)
    float* eff = nullptr;            // [2][I]
    float* row = nullptr;            // [2][I]
    float* mul_d = nullptr;          // [K]: down's factors over fac_d, a power of two, for its fp16 images
    float fac_d = 1.0f;
    Owner mem;
};

// Fewer tokens than this: act, d gate and d up are kept in two bf16 words for
// the products with the adapter, whose r sums a token are few enough for a
// rounding of their terms to show in a gradient; over more tokens it averages
// out. (One token, rank 4: the gradient of A 5.4e-3 off with one word.)
constexpr int kTwoWordM = 256;
// Weights a projection from which a forward of fewer than kPairMinM tokens does
// not decode them first (a step of 100 tokens, decoding against not: 5120 x 17408
// 618 / 496 us, 2048 x 5632 205 / 202, 1024 x 2816 149 / 148; 60 tokens, 2048 x
// 2048 146 / 158).
constexpr size_t kFewWeights = (size_t)8 << 20;

struct qmlp_adamw_s {
    AdamWChunk* chunks = nullptr;
    long count = 0;
    int num_sms = 0;
    bool param_bf16 = false, master = false, grad_bf16 = false, s8 = false;
    Owner mem;
};

namespace {

constexpr float kLeastFactor = 8.673617e-19f;  // 2^-60

__global__ void __launch_bounds__(256) factors_kernel(const float* g, const float* u, int I, float* eff, float* row) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * I) return;
    const float f = i < I ? g[i] : u[i - I];
    const bool big = !(fabsf(f) < kLeastFactor);
    eff[i] = big ? f : 1.0f;
    row[i] = big ? 1.0f : f;
}

// Where a call keeps c z A^T (or c dy B) of every token: bf16 words side by
// side in rows of ld, nc columns a word. As further steps of a GEMM: T words
// (the third again the first) and zeros up to a multiple of 64, with the parts'
// factors divided out; else kLrWords words for the expand kernel.
struct Words {
    __nv_bfloat16* p = nullptr;
    int nc = 0, ld = 0;
    bool ext = false;
    int T = 0;
    int steps() const { return ld / 64; }
};
constexpr size_t kImage = 32768;                // bytes of a stage image
constexpr size_t kMostImages = (size_t)4 << 30;  // bytes of images that the slots of a handle may hold
int word_ld(int nc, int T) { return (nc * T + 63) / 64 * 64; }
Words words_of(__nv_bfloat16* p, int nc, bool ext, int T) {
    Words w;
    w.p = p;
    w.nc = nc;
    w.ext = ext;
    w.T = ext ? T : kLrWords;
    w.ld = ext ? word_ld(nc, T) : nc * kLrWords;
    return w;
}
size_t words_room(size_t M, int nc) { return M * std::max(word_ld(nc, 3), nc * kLrWords); }

// Whether every factor of h's weights is large enough to divide by.
cudaError_t factors_divide(const qmlp_t* h, bool* ok, cudaStream_t s) {
    *ok = true;
    const int n[3] = {h->I, h->I, h->K};
    for (int i = 0; i < 3; ++i) {
        std::vector<float> f(1, h->gv[i].inv_g);
        if (h->fmt == kFP8) {
            f.resize(n[i]);
            cudaError_t e = cudaMemcpyAsync(f.data(), h->gv[i].chs, n[i] * sizeof(float), cudaMemcpyDeviceToHost, s);
            if (e == cudaSuccess) e = cudaStreamSynchronize(s);
            if (e != cudaSuccess) return e;
        }
        for (float v : f) *ok = *ok && fabsf(v) >= kLeastFactor;
    }
    return cudaSuccess;
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
    p.odd_out = l->odd ? l->odd + slot : nullptr;
    return p;
}

// The products of a call's adapters. down: of act, else gate and up of x.
LrTokens tokens_of(const qmlp_lora_s* l, int M) {
    LrTokens t;
    t.tiles = l->tiles;
    t.n_tiles = l->n_tiles;
    t.perm = l->perm;
    t.M = M;
    t.slots = l->slots;
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
    a.v_elems = a.v_word;  // of each word
    a.ldv = (down ? 1 : 2) * l->Rp;
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
    a.y_elems = l->y_elems;
    a.ldy = (size_t)(down ? 1 : 2) * a.N;
    return launch_lr_expand(a, l->Rp, false, lr_max_tiles(M, l->slots), down ? 1 : 2, s);
}
// The terms as steps of the GEMMs: z in slot order, v by entry.
cudaError_t lora_shrink_steps(const qmlp_lora_s* l, bool down, const void* z, int M, cudaStream_t s) {
    const qmlp_t* h = l->h;
    LrShrink a;
    a.tok = tokens_of(l, M);
    a.tok.perm = nullptr;
    a.x = static_cast<const __nv_bfloat16*>(z);
    a.D = down ? h->I : h->K;
    a.ldx = a.D;
    a.w = down ? l->a_d : l->a_gu;
    const int nc = (down ? 1 : 2) * l->Rp;
    a.w_slot = (size_t)nc * a.D;
    a.scale = l->scale;
    a.v = l->ev_v;
    a.v_elems = l->ev_elems;
    a.v_word = nc;
    a.ldv = word_ld(nc, l->T);
    a.entries = true;
    a.words = l->T;
    a.again = l->T == 3;
    a.pad = a.ldv - nc * l->T;
    if (h->fmt == kNVFP4) {
        a.mul0 = 1.0f / h->gv[down ? 2 : 0].inv_g;
        a.mul1 = 1.0f / h->gv[down ? 2 : 1].inv_g;
        a.half = l->Rp;
    }
    // the rows of an entry that are other slots'
    cudaError_t e =
        cudaMemsetAsync(l->ev_v, 0, (size_t)lr_max_entries(M, l->slots) * 256 * a.ldv * sizeof(*l->ev_v), s);
    if (e == cudaSuccess) e = launch_lr_shrink(a, nc, false, lr_max_tiles(M, l->slots), 1, h->num_sms, s);
    if (e != cudaSuccess) return e;
    LrOdd o;
    o.tok = a.tok;
    o.odd = l->odd;
    o.v = l->ev_v;
    o.v_elems = l->ev_elems;
    o.ldv = a.ldv;
    o.nc = nc;
    o.w = down ? l->b_d : l->b_gu;
    o.N = down ? h->K : h->I;
    o.R = l->Rp;
    o.w_slot = (size_t)(down ? 1 : 2) * o.N * o.R;
    o.T = l->T;
    o.div[0] = h->gv[down ? 2 : 0].chs;
    o.div[1] = h->gv[1].chs;
    if (h->fmt == kNVFP4) {
        o.mul[0] = h->gv[down ? 2 : 0].inv_g;
        o.mul[1] = h->gv[1].inv_g;
    }
    o.y = l->y;
    o.y_elems = l->y_elems;
    o.ldy = (size_t)(down ? 1 : 2) * o.N;
    return launch_lr_odd(o, lr_max_tiles(M, l->slots), down ? 1 : 2, s);
}
// Whether a call takes them so: M tokens on the pair GEMM, and the entries that
// the slots can make of them add at most 15% to gate/up's contraction (down's is
// longer). Measured on the 27B-class shape, steps against an fp32 array, us: 3001
// FP8 tokens of rank 64, 7 slots (12%) 1191 / 1302, 12 slots (15%) 1236 / 1300, 24
// (23%) 1290 / 1325, 48 (38%) 1417 / 1338; 3001 NVFP4 tokens of rank 16, 64 slots
// (8%) 1162 / 1241, 132 (15%) 1233 / 1271, 264 (29%) 1433 / 1404; 1024 FP8 tokens
// of rank 32, 12 slots (15%) 537 / 564. They meet at about 25%; up to there the
// slots' images cost memory that grows with them for the last 3%.
bool lora_steps(const qmlp_lora_s* l, int M) {
    if (!l->steps || M < kDqMinM) return false;
    const long most = (long)lr_max_entries(M, l->slots) * l->e_gu;
    return 100 * most <= 15L * (l->h->K / 64) * ((M + 255) / 256);
}
cudaError_t lora_images(const qmlp_lora_s* l, int slot, const qmlp_adapter* a, cudaStream_t s) {
    const qmlp_t* h = l->h;
    auto bf = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
    LrImage m;
    m.r = a->rank;
    m.R = l->Rp;
    m.T = l->T;
    m.sn = a->rank;
    m.sj = 1;
    m.parts = 2;
    m.src[0] = bf(a->gate_b);
    m.src[1] = bf(a->up_b);
    m.div[0] = h->gv[0].chs;
    m.div[1] = h->gv[1].chs;
    m.N = h->I;
    m.interleaved = 1;
    m.tiles = h->I / 128;
    m.ext = l->e_gu;
    m.img = l->img_gu + (size_t)slot * m.tiles * m.ext * kImage;
    m.img_bytes = (size_t)m.tiles * m.ext * kImage;
    m.odd = l->odd + slot;
    const cudaError_t e = launch_lr_image(m, s);
    if (e != cudaSuccess) return e;
    m.parts = 1;
    m.src[0] = bf(a->down_b);
    m.src[1] = nullptr;
    m.div[0] = h->gv[2].chs;
    m.N = h->K;
    m.interleaved = 0;
    m.tiles = h->K / 256;
    m.ext = l->e_d;
    m.img = l->img_d + (size_t)slot * m.tiles * m.ext * kImage;
    m.img_bytes = (size_t)m.tiles * m.ext * kImage;
    return launch_lr_image(m, s);
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
    a.v_elems = (size_t)kLrFew * 2 * l->Rp;
    a.y_elems = l->y_elems;
    return a;
}
cudaError_t lora_shrink_few(const qmlp_lora_s* l, bool down, const void* z, const int32_t* ids, int M, cudaStream_t s,
                            bool late = false) {
    LrFew a = few_of(l, down, ids);
    a.late = late;
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

// One block of at most kMaxGemvM tokens on the GEMV kernels.
qmlp_status lora_block(qmlp_lora_s* l, const void* x, const int32_t* ids, int M, void* out, cudaStream_t s) {
    qmlp_t* h = l->h;
    const bool split = h->sp.G && M <= split_max_m(h) && split_lora_fits(h->fmt, M, h->K, l->Rp, h->sp);
    if (lora_shrink_few(l, false, x, ids, M, s, split && split_in_kernel(h->fmt, M)) != cudaSuccess)
        return QMLP_ERR_CUDA;
    if (split) {
        SplitLaunch S = split_launch(h, x, M);
        S.out = out;
        S.lora.ids = ids;
        S.lora.rank = l->rank;
        S.lora.scale = l->scale;
        S.lora.slots = l->slots;
        S.lora.Rp = l->Rp;
        S.lora.v = l->v;
        S.lora.b_gu = l->b_gu;
        S.lora.a_d = l->a_d;
        S.lora.b_d = l->b_d;
        S.lora.vd = l->vd;
        return launch_split(S, h->sp, s) == cudaSuccess ? QMLP_OK : QMLP_ERR_CUDA;
    }
    if (lora_expand_few(l, false, ids, M, nullptr, nullptr, s) != cudaSuccess) return QMLP_ERR_CUDA;
    float* raw_d = l->raw;
    {
        // the two projections on their own, then the activation
        float* rg = l->raw + (size_t)kMaxGemvM * h->K;
        float* ru = rg + (size_t)kMaxGemvM * h->I;
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
// `inner`: the one slot of a training workspace, which makes the images of its own
// calls and needs the added terms for few tokens alone unless `added`.
static qmlp_status lora_create(qmlp_lora_t** out, qmlp_t* h, int slots, int max_rank, bool inner, bool added,
                               qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
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
        get(&l->vw, inner ? 16 : kLrWords * M * 2 * R, false);
        l->y_elems = (inner && !added ? std::min<size_t>(M, kPairMinM) : M) * std::max(2 * I, K);
        get(&l->y, l->y_elems, false);
        get(&l->raw, (size_t)kMaxGemvM * (2 * I + K), false);
        get(&l->vd, (size_t)std::max(1, h->sp.G) * kMaxGemvM * R, false);
        get(&l->perm, M, false);
        l->T = h->fmt == kFP8 ? 3 : 2;
        l->e_gu = word_ld(2 * (int)R, l->T) / 64;
        l->e_d = word_ld((int)R, l->T) / 64;
        const size_t ig = S * (I / 128) * l->e_gu * kImage, id = S * (K / 256) * l->e_d * kImage;
        bool ok = false;
        if (e == cudaSuccess && !inner && h->wdec && h->side && ig + id <= kMostImages) e = factors_divide(h, &ok, s);
        l->steps = ok;
        if (l->steps) {
            const size_t ents = (size_t)lr_max_entries((int)M, slots);
            get(&l->img_gu, ig, false);
            get(&l->img_d, id, false);
            l->ev_elems = ents * 256 * 64 * std::max(l->e_gu, l->e_d);
            get(&l->ev_v, l->ev_elems, false);
            get(reinterpret_cast<uint8_t**>(&l->x_rows), M * K * 2, false);
            get(&l->ents, (M + 255) / 256, false);
            get(&l->ent_slot, ents, false);
            get(&l->odd, S, true);
            get(&l->odd_rows, M, false);
        }
        get(&l->tiles, tiles, false);
        get(&l->n_tiles, 1, true);
        if (e == cudaSuccess) e = cudaEventCreateWithFlags(&l->ev, cudaEventDisableTiming);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) {
            cudaStreamSynchronize(s);
            if (l->ev) cudaEventDestroy(l->ev);
            l->mem.release();
            delete l;
            return from_cuda(e);
        }
        *out = l;
        return QMLP_OK;
    });
}

qmlp_status qmlp_lora_create(qmlp_lora_t** out, qmlp_t* h, int slots, int max_rank, qmlp_stream_t stream) {
    return lora_create(out, h, slots, max_rank, false, true, stream);
}

void qmlp_lora_destroy(qmlp_lora_t* l) {
    if (!l) return;
    cudaDeviceSynchronize();
    cudaEventDestroy(l->ev);
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
    if (launch_lr_pack(pack_of(l, slot, a), s) != cudaSuccess) return QMLP_ERR_CUDA;
    return l->steps && lora_images(l, slot, a, s) != cudaSuccess ? QMLP_ERR_CUDA : QMLP_OK;
}

qmlp_status qmlp_lora_forward(qmlp_lora_t* l, const void* x, const int32_t* ids, int M, void* out,
                              qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
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
            const int block = h->sp.G ? split_max_m(h) : kMaxGemvM;
            for (int m0 = 0; m0 < M; m0 += block) {
                const qmlp_status st =
                    lora_block(l, static_cast<const uint8_t*>(x) + (size_t)m0 * h->K * 2, ids + m0, std::min(block, M - m0),
                               static_cast<uint8_t*>(out) + (size_t)m0 * h->K * 2, s);
                if (st != QMLP_OK) return st;
            }
            return QMLP_OK;
        }
        const bool few = M <= kLrFew, steps = lora_steps(l, M);
        auto terms = [&](bool down, const void* z, cudaStream_t st) {
            cudaError_t e = few ? lora_shrink_few(l, down, z, ids, M, st, true) : lora_shrink(l, down, z, M, st);
            if (e == cudaSuccess)
                e = few ? lora_expand_few(l, down, ids, M, nullptr, nullptr, st) : lora_expand(l, down, M, st);
            return e;
        };
        GemmTerms t;
        t.ev = l->ev;
        if (steps) {
            t.ext = l->e_gu;
            t.ext_down = l->e_d;
            t.v = l->ev_v;
            t.img = l->img_gu;
            t.img_down = l->img_d;
            t.ents = l->ents;
            t.ent_slot = l->ent_slot;
            t.entries = lr_max_entries(M, l->slots);
            t.slots = l->slots;
            t.rows = l->perm;
            t.add = t.add_down = l->y;
            t.add_elems = l->y_elems;
            t.add_rows = l->odd_rows;
            t.before = [&](cudaStream_t st) {
                cudaError_t e = launch_lr_plan(ids, M, l->slots, l->rank, l->perm, l->tiles, l->n_tiles, l->ents,
                                               l->ent_slot, l->odd, l->odd_rows, st);
                if (e == cudaSuccess) e = launch_lr_gather(x, l->perm, M, h->K, l->x_rows, st);
                return e == cudaSuccess ? lora_shrink_steps(l, false, l->x_rows, M, st) : e;
            };
            t.between = [&](cudaStream_t st) { return lora_shrink_steps(l, true, h->act, M, st); };
            return run_gemm(h, QMLP_PATH_AUTO, 3, l->x_rows, M, out, s, nullptr, &t);
        }
        t.before = [&](cudaStream_t st) {
            const cudaError_t e = few ? cudaSuccess
                                      : launch_lr_plan(ids, M, l->slots, l->rank, l->perm, l->tiles, l->n_tiles, nullptr,
                                                       nullptr, nullptr, nullptr, st);
            return e == cudaSuccess ? terms(false, x, st) : e;
        };
        t.add = l->y;
        t.add_down = l->y;
        t.add_elems = l->y_elems;
        t.between = [&](cudaStream_t st) { return terms(true, h->act, st); };
        return run_gemm(h, QMLP_PATH_AUTO, 3, x, M, out, s, nullptr, &t);
    });
}

// ---------------------------------------------------------------------------
// training
// ---------------------------------------------------------------------------
extern "C++" {
namespace {

// What a forward keeps (see qmlp_train_saved_bytes).
struct Saved {
    uint8_t *g, *u;          // fp32 gate and up, in quads of 32 rows
    __nv_bfloat16* act;      // [M][I]
    __nv_bfloat16* act_lo;   // likewise, its second word (M < kTwoWordM), or null
    Words vgu, vd;           // c A z of gate and up, of down
    size_t bytes;
};
Saved saved_of(const qmlp_train_s* t, int M, const void* base) {
    const size_t I = t->h->I, R = t->l->Rp, m = M;
    Saved v;
    size_t at = reinterpret_cast<size_t>(base);
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) / 256 * 256;
        return reinterpret_cast<uint8_t*>(p);
    };
    v.g = take(gemm_gu_bytes(M, (int)I));
    v.u = take(gemm_gu_bytes(M, (int)I));
    v.act = reinterpret_cast<__nv_bfloat16*>(take(m * I * 2));
    // room for the second word at any M: a buffer for M tokens serves every
    // smaller M too
    uint8_t* lo = take(std::min<size_t>(m, kTwoWordM - 1) * I * 2);
    v.act_lo = M < kTwoWordM ? reinterpret_cast<__nv_bfloat16*>(lo) : nullptr;
    const bool ext = t->steps && M >= kPairMinM;
    v.vgu = words_of(reinterpret_cast<__nv_bfloat16*>(take(words_room(m, 2 * (int)R) * 2)), 2 * (int)R, ext, t->T);
    v.vd = words_of(reinterpret_cast<__nv_bfloat16*>(take(words_room(m, (int)R) * 2)), (int)R, ext, t->T);
    v.bytes = at - reinterpret_cast<size_t>(base);
    return v;
}

int tiles_for(int M) { return (M + kLrTile - 1) / kLrTile; }

// v = c z W^T for every token (one adapter), W [nc][D] or, trans, [D][nc].
LrShrink shrink_all(const qmlp_adapter* ad, const void* z, int M, int D, const Words& w) {
    LrShrink a;
    a.scale_all = ad->scale;
    a.tok.M = M;
    a.x = static_cast<const __nv_bfloat16*>(z);
    a.ldx = D;
    a.D = D;
    a.v = w.p;
    a.v_elems = (size_t)M * w.ld;
    a.v_word = w.nc;
    a.ldv = w.ld;
    a.words = w.T;
    a.again = w.ext && w.T == 3;
    a.pad = w.ld - w.nc * w.T;
    return a;
}
// The adapter's terms into l->y: v W^T, W [N][rc] or, trans, [rc][N].
cudaError_t expand_all(const qmlp_train_s* t, const Words& v, int M, int rc, int zs, const __nv_bfloat16* w,
                       size_t w_z, int N, bool trans, cudaStream_t s) {
    LrExpand a;
    a.tok.M = M;
    a.v = v.p;
    a.ldv = v.ld;
    a.v_word = v.nc;
    a.w = w;
    a.w_z = w_z;
    a.N = N;
    a.y = t->l->y;
    a.y_elems = t->l->y_elems;
    a.ldy = (size_t)N * zs;
    return launch_lr_expand(a, rc, trans, tiles_for(M), zs, s);
}

GemmLaunch dq_gemm(const qmlp_train_s* t, int M) {
    qmlp_t* h = t->h;
    GemmLaunch g;
    g.M = M;
    g.pair = kDqPair && M >= kPairMinM;
    g.err = h->err;
    g.a16 = h->a16;
    g.sig = h->sig;
    g.ws = h->gemm_ws;
    g.wait_ns = h->wait_ns;
    g.withhold = h->withhold;
    g.images_ready = true;
    g.split_tail = g.pair;
    return g;
}

// The adapter's terms of a GEMM: further steps, or added by its epilogue.
void extend(GemmLaunch& g, const Words& w, const uint8_t* img) {
    g.ext = w.steps();
    g.ext_a = w.p;
    g.ext_b = img;
}
void add_terms(GemmLaunch& g, const qmlp_lora_t* l, size_t ld) {
    g.add = l->y;
    g.ldadd = ld;
    g.add_elems = l->y_elems;
}

// Work on the handle's side stream between the events: `fork` follows all that
// is on s, and the caller waits for ev_join.
template <typename F>
cudaError_t beside(qmlp_t* h, cudaStream_t s, F&& f) {
    cudaError_t e = cudaEventRecord(h->ev_fork, s);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(h->side, h->ev_fork, 0);
    if (e == cudaSuccess) e = f(h->side);
    if (e == cudaSuccess) e = cudaEventRecord(h->ev_join, h->side);
    return e;
}

#define TRY(call)                                          \
    do {                                                   \
        const cudaError_t try_e = (call);                  \
        if (try_e != cudaSuccess) return try_e;            \
    } while (0)

// Whether the kernels can read the adapter's own arrays: the A's rows where
// they start at 16 bytes, the B's where, besides, their rank is the padded one.
bool own_a(const qmlp_adapter* a) { return aligned16(a->gate_a) && aligned16(a->up_a) && aligned16(a->down_a); }
bool own_b(const qmlp_train_s* t, const qmlp_adapter* a) {
    return a->rank == t->l->Rp && aligned16(a->gate_b) && aligned16(a->up_b) && aligned16(a->down_b) && a->gate_b &&
           a->up_b && a->down_b;
}

// What the low-rank kernels read of the adapter, padded: the A parts for the
// forward, the B parts (gate's and up's over the factor that their gradients
// carry) for the backward pass; both where expand_all adds the other side.
LrPack pack_train(const qmlp_train_s* t, const qmlp_adapter* a, bool back, bool both) {
    const qmlp_lora_t* l = t->l;
    LrPack p = pack_of(l, 0, a);
    p.first = back && !both ? 3 : 0;
    p.count = both ? 6 : 3;
    if (!back) return p;
    const size_t n = (size_t)t->h->I * l->Rp;
    for (int i = 0; i < 2; ++i) {
        LrPackPart& q = p.part[3 + i];
        q.dst_h = t->bq + i * n;
        q.dst_l = t->bq + (2 + i) * n;
        q.div = t->eff ? t->eff + (size_t)i * t->h->I : nullptr;
        q.div_all = t->h->gv[i].inv_g;
    }
    return p;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }

// The images of `rows` rows (interleaved: of each part) for words w.
LrImage image_of(const qmlp_train_s* t, const qmlp_adapter* a, const Words& w, int rows, bool interleaved, int parts,
                 uint8_t* img) {
    LrImage g;
    g.r = a->rank;
    g.R = t->l->Rp;
    g.parts = parts;
    g.T = w.T;
    g.N = rows;
    g.interleaved = interleaved;
    g.tiles = interleaved ? rows / 128 : (rows + 255) / 256;
    g.ext = w.steps();
    g.img = img;
    g.img_bytes = (size_t)g.tiles * g.ext * kImage;
    return g;
}

cudaError_t train_forward(qmlp_train_s* t, const qmlp_adapter* ad, const void* x, int M, void* out, const Saved& v,
                          cudaStream_t s) {
    qmlp_t* h = t->h;
    const qmlp_lora_t* l = t->l;
    const int K = h->K, I = h->I, R = l->Rp;
    const bool ext = v.vgu.ext, fp8 = h->fmt == kFP8;
    bool own = false;
    // few tokens: the decoder warps' GEMM, which reads the packed weights and no
    // images (the backward pass has no such form: its weights lie transposed),
    // unless the weights are so few that the twelve epilogue warps count
    const bool dq = M >= kPairMinM || (size_t)K * I < kFewWeights;
    // beside: the adapter's images, then down's weights
    TRY(beside(h, s, [&](cudaStream_t b) {
        if (ad && ext) {
            LrImage m = image_of(t, ad, v.vgu, I, true, 2, t->img_gu);
            m.src[0] = bf(ad->gate_b);
            m.src[1] = bf(ad->up_b);
            m.sn = ad->rank;
            m.sj = 1;
            m.div[0] = t->eff;
            m.div[1] = t->eff + I;
            TRY(launch_lr_image(m, b));
            m = image_of(t, ad, v.vd, K, false, 1, t->img_d);
            m.src[0] = bf(ad->down_b);
            m.sn = ad->rank;
            m.sj = 1;
            m.div[0] = h->gv[2].chs;
            TRY(launch_lr_image(m, b));
            TRY(cudaEventRecord(t->ev_img, b));
        }
        return dq ? launch_gemm_predecode(h->gm_d, h->wdec2, h->wdec2_bytes, h->num_sms, b) : cudaSuccess;
    }));
    if (dq) TRY(launch_gemm_predecode(h->gm_gu, h->wdec, h->wdec_bytes, h->num_sms, s));
    else TRY(launch_gemm_prescale(x, M, K, h->a16, h->sig, h->num_sms, s));
    if (ad) {
        own = own_a(ad);
        if (!own || !ext) TRY(launch_lr_pack(pack_train(t, ad, false, !ext), s));
        LrShrink a = shrink_all(ad, x, M, K, v.vgu);
        if (own) {
            a.wa[0] = bf(ad->gate_a);
            a.wa[1] = bf(ad->up_a);
            a.r = ad->rank;
            a.R = R;
        } else {
            a.w = l->a_gu;
        }
        if (ext && !fp8) {
            a.mul0 = 1.0f / h->gv[0].inv_g;
            a.mul1 = 1.0f / h->gv[1].inv_g;
            a.half = R;
        }
        TRY(launch_lr_shrink(a, 2 * R, false, tiles_for(M), 1, h->num_sms, s));
        if (ext) TRY(cudaStreamWaitEvent(s, t->ev_img, 0));
        else TRY(expand_all(t, v.vgu, M, R, 2, l->b_gu, (size_t)I * R, I, false, s));
    }
    GemmLaunch g = dq_gemm(t, M);
    g.epi = kEpiSwiGLU;
    g.w = h->gm_gu;
    g.wdec = dq ? h->wdec : nullptr;
    g.wdec_bytes = h->wdec_bytes;
    g.prescaled = !dq;
    g.early = ad && !ext;
    g.a = x;
    g.out = v.act;
    g.gu_g = v.g;
    g.gu_u = v.u;
    if (ad) {
        g.out_lo = v.act_lo;
        if (ext) extend(g, v.vgu, t->img_gu);
        else add_terms(g, l, (size_t)2 * I);
    }
    TRY(launch_gemm(g, h->num_sms, s));
    TRY(cudaStreamWaitEvent(s, h->ev_join, 0));
    if (!dq) TRY(launch_gemm_prescale(v.act, M, I, h->a16, h->sig, h->num_sms, s));
    if (ad) {
        LrShrink a = shrink_all(ad, v.act, M, I, v.vd);
        a.x_lo = v.act_lo;
        if (own) {
            a.wa[0] = bf(ad->down_a);
            a.r = ad->rank;
            a.R = R;
        } else {
            a.w = l->a_d;
        }
        if (ext && !fp8) a.mul0 = 1.0f / h->gv[2].inv_g;
        TRY(launch_lr_shrink(a, R, false, tiles_for(M), 1, h->num_sms, s));
        if (!ext) TRY(expand_all(t, v.vd, M, R, 1, l->b_d, 0, K, false, s));
    }
    g = dq_gemm(t, M);
    g.prescaled = !dq;
    g.early = ad && !ext;
    g.epi = kEpiPlain;
    g.w = h->gm_d;
    g.wdec = dq ? h->wdec2 : nullptr;
    g.wdec_bytes = h->wdec2_bytes;
    g.a = v.act;
    g.out = out;
    if (ad && ext) extend(g, v.vd, t->img_d);
    else if (ad) add_terms(g, l, K);
    return launch_gemm(g, h->num_sms, s);
}

cudaError_t train_backward(qmlp_train_s* t, const qmlp_adapter* ad, const void* x, int M, const Saved& v,
                           const void* dout, void* dx, const qmlp_adapter* gr, cudaStream_t s) {
    qmlp_t* h = t->h;
    const qmlp_lora_t* l = t->l;
    const int K = h->K, I = h->I, R = l->Rp;
    const bool fp8 = h->fmt == kFP8;
    // d act's GEMM of FP8 has fp16 operands: its adapter terms are added
    const bool ext = v.vgu.ext, ext_d = ext && !fp8;
    bool own = false;
    const Words wd = words_of(t->dvd, R, ext_d, 2), wv = words_of(t->dv, 2 * R, ext, 2);
    const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(dout);
    // the transposed images: down's (FP8: in fp16 with its per-channel factors,
    // which lie along the contraction here; dout is then prescaled to fp16, so
    // that neither costs a rounding to 8 bits: dx was 2.8e-3 off with bf16
    // images, 2.3e-3 with these), then gate's and up's beside the first GEMM
    TRY(beside(h, s, [&](cudaStream_t b) {
        if (ad && ext_d) {
            LrImage m = image_of(t, ad, wd, I, false, 1, t->img_d);
            m.src[0] = bf(ad->down_a);
            m.sn = 1;
            m.sj = I;
            TRY(launch_lr_image(m, b));
        }
        if (ad && ext) {
            LrImage m = image_of(t, ad, wv, K, false, 2, t->img_gu);
            m.src[0] = bf(ad->gate_a);
            m.src[1] = bf(ad->up_a);
            m.sn = 1;
            m.sj = K;
            TRY(launch_lr_image(m, b));
            TRY(cudaEventRecord(t->ev_img, b));
        }
        return launch_gemm_predecode_t(h->gm_gu, t->row, t->row ? t->row + I : nullptr, false, h->wdec, h->wdec_bytes, b);
    }));
    TRY(launch_gemm_predecode_t(h->gm_d, t->mul_d, nullptr, fp8, t->img_t, t->img_t_bytes, s));
    if (fp8) TRY(launch_gemm_prescale(dy, M, K, h->a16, h->sig, h->num_sms, s));
    if (ad) {
        own = own_b(t, ad) && !fp8 && ext;
        if (!own) TRY(launch_lr_pack(pack_train(t, ad, true, !ext_d || !ext), s));
        LrShrink a = shrink_all(ad, dy, M, K, wd);
        a.w = own ? bf(ad->down_b) : l->b_d;
        if (ext_d) a.mul0 = 1.0f / h->gv[2].inv_g;
        TRY(launch_lr_shrink(a, R, true, tiles_for(M), 1, h->num_sms, s));
        if (!ext_d) TRY(expand_all(t, wd, M, R, 1, l->a_d, 0, I, true, s));
        if (ext) TRY(cudaStreamWaitEvent(s, t->ev_img, 0));
    }
    // d act, and through the activation d gate and d up
    GemmLaunch g = dq_gemm(t, M);
    g.epi = kEpiSwiGLUGrad;
    g.w.fmt = kNVFP4;  // one factor for all columns
    g.w.inv_g0 = fp8 ? t->fac_d : h->gv[2].inv_g;
    g.f16 = g.prescaled = fp8;
    g.early = ad && !ext_d;
    g.w.N = (I + 255) / 256 * 256;
    g.w.K = K;
    g.wdec = t->img_t;
    g.wdec_bytes = t->img_t_bytes;
    g.a = dy;
    g.out = t->dgu;
    g.gu_g = v.g;
    g.gu_u = v.u;
    g.ncols = I;
    g.gf0 = h->gv[0].inv_g;
    g.gf1 = h->gv[1].inv_g;
    g.gc0 = t->eff;
    g.gc1 = t->eff ? t->eff + I : nullptr;
    __nv_bfloat16* lo = ad && M < kTwoWordM ? t->dgu_lo : nullptr;
    if (ad) {
        g.out_lo = lo;
        if (ext_d) extend(g, wd, t->img_d);
        else add_terms(g, l, I);
    }
    TRY(launch_gemm(g, h->num_sms, s));
    TRY(cudaStreamWaitEvent(s, h->ev_join, 0));
    if (ad) {
        LrShrink a = shrink_all(ad, t->dgu, M, I, wv);
        a.x_lo = lo;
        a.ldx = (size_t)2 * I;
        a.x_z = I;
        if (own) {  // d gate and d up carry NVFP4's factors: taken out of the products
            a.w = bf(ad->gate_b);
            a.w_z = (size_t)(bf(ad->up_b) - bf(ad->gate_b));
            a.mul0 = 1.0f / h->gv[0].inv_g;
            a.mul1 = 1.0f / h->gv[1].inv_g;
            a.half = R;
        } else {
            a.w = t->bq;
            a.w_lo = t->bq + (size_t)2 * I * R;
            a.w_z = (size_t)I * R;
        }
        TRY(launch_lr_shrink(a, R, true, tiles_for(M), 2, h->num_sms, s));
        if (!ext) TRY(expand_all(t, wv, M, 2 * R, 1, l->a_gu, 0, K, true, s));
    }
    g = dq_gemm(t, M);
    g.early = ad && !ext;
    g.epi = kEpiPlain;
    g.w.fmt = kNVFP4;
    g.w.N = K;
    g.w.K = 2 * I;
    g.wdec = h->wdec;
    g.wdec_bytes = h->wdec_bytes;
    g.a = t->dgu;
    g.out = dx;
    if (ad && ext) extend(g, wv, t->img_gu);
    else if (ad) add_terms(g, l, K);
    TRY(launch_gemm(g, h->num_sms, s));
    if (!gr) return cudaSuccess;
    // every gradient in one launch: B's = c dy^T (z A^T), A's = c (dy B)^T z
    LrTokGrads all;
    auto add = [&](const void* out, const void* z, const __nv_bfloat16* z_lo, int ldz, int D, const Words& w, int col,
                   bool rows_d, float mul, const float* div) {
        if (!out) return;
        LrTokGrad& q = all.job[all.count++];
        q.x = bf(z);
        q.x_lo = z_lo;
        q.ldx = ldz;
        q.D = D;
        q.M = M;
        q.v = w.p + col;
        q.ldv = w.ld;
        q.v_word = w.nc;
        q.rows_d = rows_d;
        q.r = ad->rank;
        q.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out));
        q.mul = mul;
        q.div = div;
    };
    // v lacks NVFP4's factor where it is a GEMM's operand; d gate and d up carry
    // theirs (FP8: eff)
    const float fd = ext && !fp8 ? h->gv[2].inv_g : 1.0f;
    const float fg = ext && !fp8 ? 1.0f : 1.0f / h->gv[0].inv_g, fu = ext && !fp8 ? 1.0f : 1.0f / h->gv[1].inv_g;
    add(gr->gate_b, t->dgu, lo, 2 * I, I, v.vgu, 0, true, fg, t->eff);
    add(gr->up_b, t->dgu + I, lo ? lo + I : nullptr, 2 * I, I, v.vgu, R, true, fu, t->eff ? t->eff + I : nullptr);
    add(gr->down_a, v.act, v.act_lo, I, I, wd, 0, false, ext_d ? h->gv[2].inv_g : 1.0f, nullptr);
    add(gr->gate_a, x, nullptr, K, K, wv, 0, false, 1.0f, nullptr);
    add(gr->up_a, x, nullptr, K, K, wv, R, false, 1.0f, nullptr);
    add(gr->down_b, dy, nullptr, K, K, v.vd, 0, true, fd, nullptr);
    return launch_lr_tokgrad(all, R, h->num_sms, s);
}
#undef TRY

}  // namespace
}  // extern "C++"

qmlp_status qmlp_train_create(qmlp_train_t** out, qmlp_t* h, int max_rank, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        if (!out) return QMLP_ERR_INVALID_ARG;
        *out = nullptr;
        if (!h) return QMLP_ERR_INVALID_ARG;
        if (!h->has_gemm || !h->wdec || !h->side || max_rank < 1 || max_rank > kLrMaxRank) return QMLP_ERR_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (h->fmt == kNVFP4 && !(fabsf(h->gv[i].inv_g) >= kLeastFactor)) return QMLP_ERR_INVALID_ARG;
        qmlp_train_t* t = new qmlp_train_t();
        t->h = h;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        qmlp_status st = from_cuda(factors_divide(h, &t->steps, s));
        // FP8's d act, and every GEMM where the factors cannot be divided by, add
        // the adapter's terms at any number of tokens
        if (st == QMLP_OK) st = lora_create(&t->l, h, 1, max_rank, true, h->fmt == kFP8 || !t->steps, stream);
        if (st != QMLP_OK) {
            delete t;
            return st;
        }
        const size_t I = h->I, K = h->K, M = h->max_M, R = t->l->Rp;
        t->img_t_bytes = gemm_decoded_t_bytes((int)K, (int)I);
        cudaError_t e = cudaSuccess;
        auto get = [&](auto** p, size_t count) {
            if (e == cudaSuccess) e = t->mem.alloc(reinterpret_cast<void**>(p), count * sizeof(**p));
        };
        get(&t->img_t, t->img_t_bytes);
        get(&t->bq, 4 * I * R);
        get(&t->dgu, M * 2 * I);
        get(&t->dgu_lo, std::min<size_t>(M, kTwoWordM) * 2 * I);
        get(&t->dv, words_room(M, 2 * (int)R));
        get(&t->dvd, words_room(M, (int)R));
        t->T = h->fmt == kFP8 ? 3 : 2;
        // gate/up: I / 128 tiles, or K / 256 of the transposed; down: K / 256 or I / 256
        const size_t tg = std::max(I / 128, K / 256), td = std::max(K / 256, (I + 255) / 256);
        get(&t->img_gu, tg * (size_t)(word_ld(2 * (int)R, 3) / 64) * 32768);
        get(&t->img_d, td * (size_t)(word_ld((int)R, 3) / 64) * 32768);
        if (h->fmt == kFP8) {
            get(&t->eff, 2 * I);
            get(&t->row, 2 * I);
            if (e == cudaSuccess) {
                factors_kernel<<<(unsigned)((2 * I + 255) / 256), 256, 0, s>>>(h->gv[0].chs, h->gv[1].chs, (int)I, t->eff,
                                                                              t->row);
                e = cudaPeekAtLastError();
            }
        }
        if (e == cudaSuccess && h->fmt == kFP8) {
            // e4m3 (at most 448) times a factor under fac_d, times 2^6: under 2^15
            std::vector<float> f(K);
            e = cudaMemcpyAsync(f.data(), h->gv[2].chs, K * sizeof(float), cudaMemcpyDeviceToHost, s);
            if (e == cudaSuccess) e = cudaStreamSynchronize(s);
            float top = 0.0f;
            for (float v : f)
                if (isfinite(v)) top = std::max(top, fabsf(v));
            int ex = 0;
            frexpf(top, &ex);
            ex = std::max(-100, std::min(100, ex - 6));
            t->fac_d = ldexpf(1.0f, ex);
            for (float& v : f) v = ldexpf(v, -ex);
            get(&t->mul_d, K);
            if (e == cudaSuccess) e = cudaMemcpyAsync(t->mul_d, f.data(), K * sizeof(float), cudaMemcpyHostToDevice, s);
            if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        }
        if (e == cudaSuccess) e = cudaEventCreateWithFlags(&t->ev_img, cudaEventDisableTiming);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) {
            cudaStreamSynchronize(s);
            if (t->ev_img) cudaEventDestroy(t->ev_img);
            qmlp_lora_destroy(t->l);
            t->mem.release();
            delete t;
            return from_cuda(e);
        }
        *out = t;
        return QMLP_OK;
    });
}

void qmlp_train_destroy(qmlp_train_t* t) {
    if (!t) return;
    cudaDeviceSynchronize();
    cudaEventDestroy(t->ev_img);
    qmlp_lora_destroy(t->l);
    t->mem.release();
    delete t;
}

size_t qmlp_train_saved_bytes(qmlp_train_t* t, int M) {
    return !t || M < 1 || M > t->h->max_M ? 0 : saved_of(t, M, nullptr).bytes;
}

// The checks that forward and backward share.
static qmlp_status check_train(const qmlp_train_t* t, const qmlp_adapter* a, int M) {
    if (M < 1 || M > t->h->max_M) return QMLP_ERR_SHAPE;
    return a ? check_adapter(a, t->l->max_rank) : QMLP_OK;
}

qmlp_status qmlp_train_forward(qmlp_train_t* t, const qmlp_adapter* adapter, const void* x, int M, void* out,
                               void* saved, qmlp_stream_t stream) {
    if (!t || !x || !out || !saved) return QMLP_ERR_INVALID_ARG;
    const qmlp_status st = check_train(t, adapter, M);
    if (st != QMLP_OK) return st;
    if (!aligned16(x) || !aligned16(out) || !aligned16(saved)) return QMLP_ERR_ALIGNMENT;
    const size_t xb = (size_t)M * t->h->K * 2, sb = saved_of(t, M, nullptr).bytes;
    if (overlaps(out, xb, x, xb) || overlaps(saved, sb, x, xb) || overlaps(saved, sb, out, xb)) return QMLP_ERR_ALIAS;
    if (fault("launch")) return QMLP_ERR_CUDA;
    return train_forward(t, adapter, x, M, out, saved_of(t, M, saved), reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? QMLP_OK
               : QMLP_ERR_CUDA;
}

qmlp_status qmlp_train_backward(qmlp_train_t* t, const qmlp_adapter* adapter, const void* x, int M, const void* saved,
                                const void* dout, void* dx, const qmlp_adapter* grads, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
        if (!t || !x || !saved || !dout || !dx || (grads && !adapter)) return QMLP_ERR_INVALID_ARG;
        const qmlp_status st = check_train(t, adapter, M);
        if (st != QMLP_OK) return st;
        if (!aligned16(x) || !aligned16(saved) || !aligned16(dout) || !aligned16(dx)) return QMLP_ERR_ALIGNMENT;
        const size_t K = t->h->K, I = t->h->I, xb = (size_t)M * K * 2;
        std::vector<Range> r;
        auto add = [&](const void* p, size_t bytes, bool w) {
            if (p) r.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, w});
        };
        add(x, xb, false);
        add(dout, xb, false);
        add(saved, saved_of(t, M, nullptr).bytes, false);
        add(dx, xb, true);
        if (adapter) {
            const size_t rk = (size_t)adapter->rank * 2;
            const size_t bytes[6] = {rk * K, rk * I, rk * K, rk * I, rk * I, rk * K};
            const void* p[6] = {adapter->gate_a, adapter->gate_b, adapter->up_a, adapter->up_b, adapter->down_a, adapter->down_b};
            for (int i = 0; i < 6; ++i) add(p[i], bytes[i], false);
            if (grads) {
                const void* g[6] = {grads->gate_a, grads->gate_b, grads->up_a, grads->up_b, grads->down_a, grads->down_b};
                for (int i = 0; i < 6; ++i) {
                    if (g[i] && !p[i]) return QMLP_ERR_INVALID_ARG;
                    if (!aligned(g[i], 2)) return QMLP_ERR_ALIGNMENT;
                    add(g[i], bytes[i], true);
                }
            }
        }
        if (any_alias(r)) return QMLP_ERR_ALIAS;
        if (fault("launch")) return QMLP_ERR_CUDA;
        return train_backward(t, adapter, x, M, saved_of(t, M, saved), dout, dx, grads,
                              reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? QMLP_OK
                   : QMLP_ERR_CUDA;
    });
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
qmlp_status qmlp_adamw_create(qmlp_adamw_t** out, const qmlp_adamw_tensor* ts, int count, qmlp_dtype pdt,
                              qmlp_dtype gdt, qmlp_state state, qmlp_stream_t stream) {
    return guarded([&]() -> qmlp_status {
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
        h->num_sms = sms;
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
    });
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
    return launch_adamw(h->chunks, h->count, h->param_bf16, h->master, h->grad_bf16, h->s8, k, h->num_sms,
                        reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QMLP_OK
               : QMLP_ERR_CUDA;
}

}  // extern "C"
