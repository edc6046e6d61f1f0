// moe_layer.cu -- a whole mixture-of-experts layer: router, selection, routed and
// shared experts, weighted sum.
//
// For every token x, with E routed experts and S shared ones (the last S of the
// B = E + S banks; W13, W2 as in moe_awq.cu):
//   l[e] = router[e] . x            e < E, fp32
//   p    = softmax(l) or sigmoid(l);  the topk largest p (+ bias) are selected,
//          ties to the lowest index
//   w[e] = route_scale p[e] (over the sum of the selected p, if renormed)
//   w[E + j] = 1, or sigmoid(shared_gate[j] . x)
//   act  = SiLU(W13[e][:I] x) (W13[e][I:] x)
//   out  = sum over the selected and shared e of w[e] W2[e] act
//
// Few tokens (at most 16): one cooperative kernel, a CTA an SM, in three parts with
// a grid barrier between them. With one token all of it is latency: the reads of
// each part depend on the part before.
//  1. Router: a row for five warps; x goes to shared memory meanwhile.
//  2. Every CTA selects by itself (a warp a token, from the logits in L2), lists
//     the experts that any token named, and takes its share of their (expert,
//     eight gate and eight up rows) tiles, ten warps a tile as in moe_awq.cu. All
//     tokens are columns of the MMAs, whether they named the expert or not: the
//     weights bound the time, and no token has to be gathered. act is kept in
//     fp32, a row a (token, choice).
//  3. A warp a (16 output rows, expert): act as fp16 times a power of two of the
//     (token, expert) (its largest value, known now, goes to [2^14, 2^15): off by
//     2^-11 of a value at most, the only rounding between x and out), W2 times it;
//     a token's choices are added in their order, fp32. So a token's result does
//     not depend on the other tokens of the call.
// More tokens: the same router and selection as two kernels, then the grouped
// kernels (moe_grouped.cu) with the shared experts as further routes.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kTeams = 2;                           // tiles that a CTA has in hand
constexpr int kWarps = kTeams * kMoeKSplit;         // 20
constexpr int kThreads = kWarps * 32;
constexpr int kRowTeams = 4;                        // router rows that a CTA has in hand
constexpr int kRowWarps = kWarps / kRowTeams;       // 5
constexpr int kC13 = 4;                             // 64-k chunks that a W13 warp loads at once
constexpr int kG2 = 10;                             // k16 groups that a W2 warp loads at once
constexpr uint64_t kWaitNs = 2000000000ull;         // 2 s
constexpr int kSmemMax = 224 * 1024;
constexpr uint16_t kNone = 0xFFFF;

// Bytes of the shared-memory tables (slots: experts that the tokens can name).
struct Layout {
    int x, coef, ridx, expo, slot_e, mask, sel_e, sel_w, part, bytes;
};
__host__ __device__ inline Layout layout(int M, int K, int E, int slots, int NT) {
    Layout l;
    auto up = [](int b) { return (b + 15) / 16 * 16; };
    int at = 0;
    l.x = at, at += M * K * 2;
    l.coef = at, at += up(slots * M * 4);
    l.ridx = at, at += up(slots * M * 2);
    l.expo = at, at += up(slots * M);
    l.slot_e = at, at += up(slots * 4);
    l.mask = at, at += up(E * 4);
    l.sel_e = at, at += 16 * 16 * 4;
    l.sel_w = at, at += 16 * 16 * 4;
    l.part = at, at += 2 * kWarps * 16 * 8 * NT * 4;  // (parts 1 and 3 need less)
    l.bytes = at;
    return l;
}

template <typename T>
QMLP_DEV void load8f(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
}
// Eight values of a type known at run time (0 fp32, 1 bf16, 2 fp16).
QMLP_DEV void load8t(const void* p, int type, size_t at, float (&v)[8]) {
    if (type == 0) load8f(static_cast<const float*>(p) + at, v);
    else if (type == 1) load8f(static_cast<const __nv_bfloat16*>(p) + at, v);
    else load8f(static_cast<const __half*>(p) + at, v);
}

QMLP_DEV float wsum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Row `row` of the router, then of the shared gates, times up to 16 tokens, over
// the chunks of 8 k of `threads` threads: this thread's sums.
QMLP_DEV void row_dots(const MoeLayerArgs& a, const void* x, int M, int row, int tid, int threads, float (&acc)[16]) {
#pragma unroll
    for (int m = 0; m < 16; ++m) acc[m] = 0.0f;
    const bool sh = row >= a.E;
    const void* w = sh ? a.sgate : a.router;
    const size_t base = (size_t)(sh ? row - a.E : row) * a.K;
    for (int c = tid; c < a.K / 8; c += threads) {
        float wv[8];
        load8t(w, a.rdt, base + 8 * c, wv);
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            if (m < M) {
                float xv[8];
                load8t(x, a.x_bf16 ? 1 : 2, (size_t)m * a.K + 8 * c, xv);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m] = fmaf(wv[e], xv[e], acc[m]);
            }
        }
    }
}

// A float as an unsigned number of the same order, above 1; NaN is 1, the lowest.
QMLP_DEV uint32_t order_key(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return max(k, 2u);
}

// One warp selects for one token: logits l[0..E) (then the shared gates'), its
// choices to sel_e / sel_w in order (the shared experts after the routed ones).
template <int NPL>
QMLP_DEV void select(const MoeLayerArgs& a, const float* l, int lane, int* sel_e, float* sel_w) {
    float v[NPL];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < a.E ? __ldcg(l + e) : -INFINITY;
        mx = fmaxf(mx, v[i]);
    }
    float lsh = 0.0f;
    if (a.sgate && lane < a.S) lsh = __ldcg(l + a.E + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float total = 1.0f;  // softmax, without renorming or with a bias: p itself is wanted
    if (a.softmax && (!a.renorm || a.bias)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (i * 32 + lane < a.E) s += expf(v[i] - mx);
        total = wsum(s);
    }
    auto score = [&](float t) { return a.softmax ? expf(t - mx) / total : 1.0f / (1.0f + expf(-t)); };
    uint32_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        // without a bias the logits have the scores' order
        key[i] = e < a.E ? order_key(a.bias ? score(v[i]) + __ldg(a.bias + e) : v[i]) : 0u;
    }
    float mine = 0.0f;  // lane r: the score of choice r
    for (int r = 0; r < a.topk; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
        float s = 0.0f;
        if ((int)(e & 31u) == lane) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (i == (int)(e >> 5)) {
                    s = score(v[i]);
                    key[i] = 0u;
                }
        }
        s = __shfl_sync(0xffffffffu, s, (int)(e & 31u));
        if (lane == r) {
            mine = s;
            sel_e[r] = (int)e;
        }
    }
    const float sum = a.renorm ? wsum(lane < a.topk ? mine : 0.0f) : 1.0f;
    if (lane < a.topk) sel_w[lane] = mine / sum * a.rscale;
    if (lane < a.S) {
        sel_e[a.topk + lane] = a.E + lane;
        sel_w[a.topk + lane] = a.sgate ? 1.0f / (1.0f + expf(-lsh)) : 1.0f;
    }
}
QMLP_DEV void select_any(const MoeLayerArgs& a, const float* l, int lane, int* sel_e, float* sel_w) {
    if (a.E <= 64) select<2>(a, l, lane, sel_e, sel_w);
    else if (a.E <= 256) select<8>(a, l, lane, sel_e, sel_w);
    else if (a.E <= 512) select<16>(a, l, lane, sel_e, sel_w);
    else select<32>(a, l, lane, sel_e, sel_w);
}

// ---------------------------------------------------------------------------
// Weight decode, as moe_awq.cu: {half_fma(q_lo, s, b), half_fma(q_hi, s, b)}
// ---------------------------------------------------------------------------
QMLP_DEV uint32_t lfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
template <int MB>
QMLP_DEV void meta2(uint32_t m, uint32_t& s2, uint32_t& b2) {
    const uint32_t s = m & 0xFFFFu;
    uint32_t b;
    if (MB == 4) {
        b = m >> 16;
    } else {
        const float bf = -(float)((m >> 16) & 0xFFu) * __half2float(__ushort_as_half((unsigned short)s));
        b = __half_as_ushort(__float2half_rn(bf));
    }
    s2 = s | (s << 16);
    b2 = b | (b << 16);
}
template <int T>  // byte T of the word
QMLP_DEV uint32_t pair_of(uint32_t w, uint32_t s2, uint32_t b2) {
    const uint32_t m = __byte_perm(w, 0u, (uint32_t)(T | 4 << 4 | T << 8 | 4 << 12));
    const uint32_t q = lfma2((m & 0x00F0000Fu) | 0x64006400u, 0x2C003C00u, 0xD400E400u);
    return lfma2(q, s2, b2);
}

// A warp's batch of a W13 tile: its four chunks' codes and records (lane-sliced
// banks in warp blocks, internal.h).
template <int MB>
struct Batch13 {
    uint32_t c[kC13][2][2];  // [chunk][gate, up][unit]
    uint32_t m[kC13][2][2];
};
template <int MB>
QMLP_DEV void load13(Batch13<MB>& b, const MoeLayerArgs& a, size_t blk, int at, int lane) {
    const int g = lane >> 2, np = moe_w13_pairs(a.K), ms = moe_w13_meta_stride(a.K, MB);
    const uint8_t* codes = a.w13 + blk * moe_w13_block_bytes(a.K);
    if (!QMLP_INB((blk + 1) * moe_w13_block_bytes(a.K) - 1, a.w13_bytes, 101) ||
        !QMLP_INB((blk + 1) * moe_w13_meta_block_bytes(a.K, MB) - 1, a.w13_meta_bytes, 102))
        return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int pi = 0; pi < kC13 / 2; ++pi) {
            const int pp = at / 2 + pi;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (pp < np) u = __ldg(reinterpret_cast<const uint4*>(codes + (size_t)(q * np + pp) * 512) + lane);
            b.c[2 * pi][q][0] = u.x;
            b.c[2 * pi][q][1] = u.y;
            b.c[2 * pi + 1][q][0] = u.z;
            b.c[2 * pi + 1][q][1] = u.w;
        }
        const uint8_t* slot =
            a.w13_meta + blk * moe_w13_meta_block_bytes(a.K, MB) + (q * 8 + g) * ms + (size_t)at * 2 * MB;
        if (MB == 4) {
            const uint4 m0 = __ldg(reinterpret_cast<const uint4*>(slot)), m1 = __ldg(reinterpret_cast<const uint4*>(slot) + 1);
            const uint32_t mr[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
            for (int i = 0; i < kC13; ++i) b.m[i][q][0] = mr[2 * i], b.m[i][q][1] = mr[2 * i + 1];
        } else {
            uint32_t mr[3 * kC13 / 2 + 1];
#pragma unroll
            for (int j = 0; j < 3 * kC13 / 4; ++j) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(slot) + j);
                mr[2 * j] = v.x;
                mr[2 * j + 1] = v.y;
            }
            mr[3 * kC13 / 2] = 0u;
#pragma unroll
            for (int i = 0; i < kC13; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int o = 3 * (2 * i + h);
                    b.m[i][q][h] = __funnelshift_r(mr[o / 4], mr[o / 4 + 1], 8 * (o % 4)) & 0xFFFFFFu;
                }
        }
    }
}

// A warp's batch of W2: rows g and g + 8 of 16, kG2 groups of 16 k.
template <int MB>
struct Batch2 {
    uint32_t c[kG2 / 2][2], m[kG2 / 2][2];
};
template <int MB>
QMLP_DEV void load2(Batch2<MB>& b, const MoeLayerArgs& a, int e, int n0, int gb, int lane) {
    const int g = lane >> 2, t = lane & 3, gpr = a.I / 32;
    const size_t row0 = (size_t)e * a.K + n0 + g;
    if (!QMLP_INB((row0 + 9) * (a.I / 2) - 1, a.w2_bytes, 103) ||
        !QMLP_INB((row0 + 9) * gpr * MB - 1, a.w2_meta_bytes, 104))
        return;
#pragma unroll
    for (int i = 0; i < kG2 / 2; ++i) {
        const int u = gb / 2 + i;  // unit of 32 k
        b.c[i][0] = b.c[i][1] = b.m[i][0] = b.m[i][1] = 0u;
        if (u < gpr) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const size_t row = row0 + 8 * h;
                b.c[i][h] = __ldg(reinterpret_cast<const unsigned int*>(a.w2 + row * (a.I / 2) + 16 * u) + t);
                const uint8_t* mp = a.w2_meta + (row * gpr + u) * MB;
                if (MB == 4) {
                    b.m[i][h] = __ldg(reinterpret_cast<const unsigned int*>(mp));
                } else {
                    b.m[i][h] = (uint32_t)__ldg(mp) | (uint32_t)__ldg(mp + 1) << 8 | (uint32_t)__ldg(mp + 2) << 16;
                }
            }
        }
    }
}

QMLP_DEV unsigned long long ld_acq(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// Grid barrier: what the CTAs wrote before it is visible after it. False, for the
// whole CTA, after the bounded wait (recorded in a.err).
QMLP_DEV bool grid_barrier(const MoeLayerArgs& a, int* s_pass) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned long long tk;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(tk) : "l"(a.ticket) : "memory");
        const unsigned long long G = gridDim.x, target = (tk / G + 1ull) * G;
        int pass = 1;
        if (tk + 1ull != target) {
            const uint64_t t0 = globaltimer_ns();
            while (ld_acq(a.ticket) < target)
                if (globaltimer_ns() - t0 > a.limit) {
                    atomicExch(a.err, 101);
                    pass = 0;
                    break;
                }
        }
        *s_pass = pass;
    }
    __syncthreads();
    return *s_pass != 0;
}

QMLP_DEV void store_any(void* p, int type, size_t at, float v) {
    if (type == 0) static_cast<float*>(p)[at] = v;
    else if (type == 1) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[at] = __float2half_rn(v);
}

template <int MB, int NT>
__global__ void __launch_bounds__(kThreads, 1) moe_layer_kernel(const MoeLayerArgs a) {
    constexpr int kC = 8 * NT;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_pass, s_n, s_sig[16], s_cnt[kWarps];
    const int M = a.M, K = a.K, I = a.I, rows = a.E + (a.sgate ? a.S : 0), nsel = a.topk + a.S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Layout L = layout(M, K, a.E, a.slots, NT);
    uint4* xsm = reinterpret_cast<uint4*>(sm + L.x);
    float* coef = reinterpret_cast<float*>(sm + L.coef);          // [slot][M]
    uint16_t* ridx = reinterpret_cast<uint16_t*>(sm + L.ridx);    // [slot][M]: row of act
    int8_t* expo = reinterpret_cast<int8_t*>(sm + L.expo);        // [slot][M]
    int* slot_e = reinterpret_cast<int*>(sm + L.slot_e);
    uint32_t* mask = reinterpret_cast<uint32_t*>(sm + L.mask);    // [E]: tokens that named it, then its slot
    int* sel_e = reinterpret_cast<int*>(sm + L.sel_e);            // [16][16]
    float* sel_w = reinterpret_cast<float*>(sm + L.sel_w);
    float* part = reinterpret_cast<float*>(sm + L.part);

    // ---------------- 1: router ----------------
    {
        const int rt = warp / kRowWarps, tid = threadIdx.x - rt * kRowWarps * 32;
        for (int row = blockIdx.x + rt * gridDim.x; row < rows; row += kRowTeams * gridDim.x) {
            float acc[16];
            row_dots(a, a.x, M, row, tid, kRowWarps * 32, acc);
            float* pr = part + rt * kRowWarps * 16;
#pragma unroll
            for (int m = 0; m < 16; ++m)
                if (m < M) {
                    const float s = wsum(acc[m]);
                    if (lane == 0) pr[(warp % kRowWarps) * 16 + m] = s;
                }
            named_bar_sync(1 + rt, kRowWarps * 32);
            if (tid < M) {
                float s = 0.0f;
                for (int w = 0; w < kRowWarps; ++w) s += pr[w * 16 + tid];
                if (QMLP_INB((size_t)tid * (a.E + a.S) + row, a.logit_elems, 105)) a.logits[(size_t)tid * (a.E + a.S) + row] = s;
            }
            named_bar_sync(1 + rt, kRowWarps * 32);
        }
    }
    // the largest |act| of each row of act, for part 2
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < M * nsel; i += gridDim.x * kThreads) a.amax[i] = 0;
    for (int e = threadIdx.x; e < a.E; e += kThreads) mask[e] = 0;
    // x -> fp16 in the order of the MMAs: slot ((c 2 + jj) M + m) 4 + t has, of chunk
    // c (64 k) and its steps 2jj and 2jj + 1, k pairs 2t.. and 8 + 2t.. of token m
    if (a.x_bf16) {
        for (int m = warp; m < M; m += kWarps) {
            float mx = 0.0f;
            for (int c = lane; c < K / 8; c += 32) {
                float v[8];
                load8t(a.x, 1, (size_t)m * K + 8 * c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) s_sig[m] = prescale_exponent(mx);
        }
    } else if (threadIdx.x < 16) {
        s_sig[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (K / 64) * 2 * M * 4; i += kThreads) {
        const int tt = i & 3, m = (i >> 2) % M, cj = (i >> 2) / M;
        const uint32_t* row = static_cast<const uint32_t*>(a.x) + (size_t)m * (K / 2) + cj * 16 + tt;
        uint32_t v[4] = {__ldg(row), __ldg(row + 4), __ldg(row + 8), __ldg(row + 12)};
        if (a.x_bf16) {
            const int sg = s_sig[m];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = __floats2half2_rn(scalbnf(__uint_as_float(v[j] << 16), sg),
                                                    scalbnf(__uint_as_float(v[j] & 0xFFFF0000u), sg));
                v[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        xsm[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
    if (!grid_barrier(a, &s_pass)) {
        if (threadIdx.x == 0) atomicAdd(a.ticket, 1ull);  // the second barrier's count
        return;
    }

    // ---------------- 2: selection, W13 ----------------
    if (warp < M) select_any(a, a.logits + (size_t)warp * (a.E + a.S), lane, sel_e + warp * 16, sel_w + warp * 16);
    __syncthreads();
    for (int i = threadIdx.x; i < M * a.topk; i += kThreads) atomicOr(&mask[sel_e[(i / a.topk) * 16 + i % a.topk]], 1u << (i / a.topk));
    __syncthreads();
    // the experts named, in their order, then the shared ones
    const int per = (a.E + kWarps - 1) / kWarps;  // experts a warp, its lanes side by side
    {
        int n = 0;
        for (int b = 0; b < per; b += 32) {
            const int e = warp * per + b + lane;
            n += __popc(__ballot_sync(0xffffffffu, b + lane < per && e < a.E && mask[e] != 0));
        }
        if (lane == 0) s_cnt[warp] = n;
    }
    __syncthreads();
    {
        int at = 0;
        for (int w = 0; w < warp; ++w) at += s_cnt[w];
        for (int b = 0; b < per; b += 32) {
            const int e = warp * per + b + lane;
            const bool on = b + lane < per && e < a.E && mask[e] != 0;
            const uint32_t vote = __ballot_sync(0xffffffffu, on);
            if (on) {
                const int s = at + __popc(vote & ((1u << lane) - 1));
                slot_e[s] = e;
                mask[e] = (uint32_t)s;
            }
            at += __popc(vote);
        }
        if (warp == kWarps - 1 && lane == 0) s_n = at;
    }
    __syncthreads();
    const int named = s_n, slots = named + a.S;
    for (int i = threadIdx.x; i < slots * M; i += kThreads) {
        ridx[i] = kNone;
        coef[i] = 0.0f;
    }
    for (int j = threadIdx.x; j < a.S; j += kThreads) slot_e[named + j] = a.E + j;
    __syncthreads();
    for (int i = threadIdx.x; i < M * nsel; i += kThreads) {
        const int m = i / nsel, r = i % nsel, e = sel_e[m * 16 + r];
        const int s = r < a.topk ? (int)mask[e] : named + r - a.topk;
        ridx[s * M + m] = (uint16_t)i;
        coef[s * M + m] = sel_w[m * 16 + r];
        if (blockIdx.x == 0 && r < a.topk) {
            if (a.ids_out) a.ids_out[m * a.topk + r] = e;
            if (a.w_out) a.w_out[m * a.topk + r] = sel_w[m * 16 + r];
        }
    }
    __syncthreads();
    {
        const int team = warp / kMoeKSplit, ks = warp % kMoeKSplit, tid = threadIdx.x - team * kMoeKSplit * 32;
        const int no = I / 8, items = slots * no, stride = kTeams * gridDim.x;
        const int Kc = K / 64, cpw = moe_w13_cpw(K), c0 = ks * cpw, nc = max(0, min(Kc, c0 + cpw) - c0);
        Batch13<MB> b;
        int item = blockIdx.x + team * gridDim.x;
        auto block = [&](int it) { return ((size_t)slot_e[it / no] * no + it % no) * kMoeKSplit + ks; };
        if (item < items && nc > 0) load13<MB>(b, a, block(item), 0, lane);
        for (int turn = 0; item < items; item += stride, turn ^= 1) {
            const int s = item / no, oct = item % no;
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
            for (int cb = 0; cb < nc; cb += kC13) {
                if (cb > 0) load13<MB>(b, a, block(item), cb, lane);
#pragma unroll
                for (int i = 0; i < kC13; ++i) {
                    if (cb + i < nc) {
                        uint32_t s2[2][2], b2[2][2];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int h = 0; h < 2; ++h) meta2<MB>(b.m[i][q][h], s2[q][h], b2[q][h]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // steps 2h and 2h + 1: record h
                            uint32_t f[2][4];
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                f[q][0] = pair_of<0>(b.c[i][q][h], s2[q][h], b2[q][h]);
                                f[q][1] = pair_of<1>(b.c[i][q][h], s2[q][h], b2[q][h]);
                                f[q][2] = pair_of<2>(b.c[i][q][h], s2[q][h], b2[q][h]);
                                f[q][3] = pair_of<3>(b.c[i][q][h], s2[q][h], b2[q][h]);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint4 x = xsm[(((c0 + cb + i) * 2 + h) * M + min(8 * n + g, M - 1)) * 4 + t];
                                mma_f16_16816(d[n], f[0][0], f[1][0], f[0][1], f[1][1], x.x, x.y);
                                mma_f16_16816(d[n], f[0][2], f[1][2], f[0][3], f[1][3], x.z, x.w);
                            }
                        }
                    }
                }
            }
            // the next tile's weights are on their way while this one's sums are added
            if (item + stride < items && nc > 0) load13<MB>(b, a, block(item + stride), 0, lane);
            float* pt = part + ((turn * kTeams + team) * kMoeKSplit) * 16 * kC;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(pt + (ks * 16 + g) * kC + 8 * n + 2 * t) = make_float2(d[n][0], d[n][1]);
                *reinterpret_cast<float2*>(pt + (ks * 16 + g + 8) * kC + 8 * n + 2 * t) = make_float2(d[n][2], d[n][3]);
            }
            named_bar_sync(1 + team, kMoeKSplit * 32);
            if (tid < 8 * kC) {
                const int row = tid & 7, m = tid >> 3;
                float v = 0.0f;
                if (m < M && ridx[s * M + m] != kNone) {
                    float hg = 0.0f, hu = 0.0f;
#pragma unroll
                    for (int w = 0; w < kMoeKSplit; ++w) {
                        hg += pt[(w * 16 + row) * kC + m];
                        hu += pt[(w * 16 + 8 + row) * kC + m];
                    }
                    const int sg = s_sig[m], r = ridx[s * M + m];
                    v = silu_f32(scalbnf(hg, -sg)) * scalbnf(hu, -sg);
                    if (QMLP_INB((size_t)r * I + 8 * oct + row, a.act_elems, 106)) a.act[(size_t)r * I + 8 * oct + row] = v;
                    v = fabsf(v);
                    // the eight rows of a token are neighbours in a warp; the largest
                    // of them does not depend on the order of the tiles
                    uint32_t top = __float_as_uint(v);
                    const uint32_t lanes = 0xFFu << (lane & 24);
                    top = __reduce_max_sync(lanes, top);
                    if (row == 0) atomicMax(a.amax + r, (int)top);
                }
            }
        }
    }
    if (!grid_barrier(a, &s_pass)) return;

    // ---------------- 3: W2 and the weighted sum ----------------
    for (int i = threadIdx.x; i < slots * M; i += kThreads) {
        int e = 0;
        if (ridx[i] != kNone) {
            e = max(-113, min(126, prescale_exponent(__int_as_float(__ldcg(a.amax + ridx[i])))));
            coef[i] *= __int_as_float((127 - e) << 23);
        }
        expo[i] = (int8_t)e;
    }
    __syncthreads();
    const int ng = I / 16;
    for (int tile = blockIdx.x; tile < K / 16; tile += gridDim.x) {
        __syncthreads();  // the sums of the tile before are read
        for (int s = warp; s < slots; s += kWarps) {
            int col[NT];
            float up[NT];
            const float* row[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int m = 8 * n + g;
                col[n] = m < M ? ridx[s * M + m] : kNone;
                up[n] = m < M ? __int_as_float((127 + expo[s * M + m]) << 23) : 1.0f;
                row[n] = a.act + (size_t)(col[n] == kNone ? 0 : col[n]) * I;
            }
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
            for (int gb = 0; gb < ng; gb += kG2) {
                Batch2<MB> b;
                load2<MB>(b, a, slot_e[s], 16 * tile, gb, lane);
                uint32_t xb[NT][kG2][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < kG2; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float2 v = make_float2(0.0f, 0.0f);
                            if (gb + i < ng && col[n] != kNone &&
                                QMLP_INB((size_t)col[n] * I + 16 * (gb + i) + 8 * h + 2 * t + 1, a.act_elems, 107))
                                v = __ldcg(reinterpret_cast<const float2*>(row[n] + 16 * (gb + i) + 8 * h + 2 * t));
                            const __half2 p = __floats2half2_rn(v.x * up[n], v.y * up[n]);
                            xb[n][i][h] = *reinterpret_cast<const uint32_t*>(&p);
                        }
#pragma unroll
                for (int i = 0; i < kG2 / 2; ++i) {
                    if (gb + 2 * i < ng) {
                        uint32_t s2[2], b2[2], f[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            meta2<MB>(b.m[i][h], s2[h], b2[h]);
                            f[h][0] = pair_of<0>(b.c[i][h], s2[h], b2[h]);
                            f[h][1] = pair_of<1>(b.c[i][h], s2[h], b2[h]);
                            f[h][2] = pair_of<2>(b.c[i][h], s2[h], b2[h]);
                            f[h][3] = pair_of<3>(b.c[i][h], s2[h], b2[h]);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16_16816(d[n], f[0][0], f[1][0], f[0][1], f[1][1], xb[n][2 * i][0], xb[n][2 * i][1]);
                            mma_f16_16816(d[n], f[0][2], f[1][2], f[0][3], f[1][3], xb[n][2 * i + 1][0],
                                          xb[n][2 * i + 1][1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = 8 * n + 2 * t + e;
                    const int r = m < M ? ridx[s * M + m] : kNone;
                    if (r != kNone) {  // a choice of token m: its rows g and g + 8
                        const float w = coef[s * M + m];
                        part[r * 16 + g] = w * d[n][e];
                        part[r * 16 + g + 8] = w * d[n][2 + e];
                    }
                }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * M; i += kThreads) {
            const int r = i & 15, m = i >> 4;
            float v = 0.0f;
            for (int c = 0; c < nsel; ++c) v += part[(m * nsel + c) * 16 + r];
            store_any(a.out, a.odt, (size_t)m * K + 16 * tile + r, v);
        }
    }
}

// ---------------------------------------------------------------------------
// More tokens: router and selection for the grouped kernels
// ---------------------------------------------------------------------------
// One CTA eight rows (a warp a row) for 16 tokens.
__global__ void __launch_bounds__(256) router_kernel(const MoeLayerArgs a) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int m0 = blockIdx.y * 16, M = min(16, a.M - m0);
    if (row >= a.E + (a.sgate ? a.S : 0)) return;
    float acc[16];
    row_dots(a, static_cast<const uint16_t*>(a.x) + (size_t)m0 * a.K, M, row, lane, 32, acc);
#pragma unroll
    for (int m = 0; m < 16; ++m)
        if (m < M) {
            const float s = wsum(acc[m]);
            const size_t at = (size_t)(m0 + m) * (a.E + a.S) + row;
            if (lane == 0 && QMLP_INB(at, a.logit_elems, 108)) a.logits[at] = s;
        }
}
// A warp a token.
__global__ void __launch_bounds__(128) select_kernel(const MoeLayerArgs a) {
    __shared__ int se[4][16];
    __shared__ float sw[4][16];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, m = blockIdx.x * 4 + w, nsel = a.topk + a.S;
    if (m >= a.M) return;
    select_any(a, a.logits + (size_t)m * (a.E + a.S), lane, se[w], sw[w]);
    __syncwarp();
    if (lane < nsel) {
        a.ids[(size_t)m * nsel + lane] = se[w][lane];
        a.weights[(size_t)m * nsel + lane] = sw[w][lane];
    }
    if (lane < a.topk) {
        if (a.ids_out) a.ids_out[(size_t)m * a.topk + lane] = se[w][lane];
        if (a.w_out) a.w_out[(size_t)m * a.topk + lane] = sw[w][lane];
    }
}

template <int MB, int NT>
cudaError_t launch_few(const MoeLayerArgs& a, int bytes, int num_sms, cudaStream_t s) {
    static bool attr = false;
    if (!attr) {
        const cudaError_t e =
            cudaFuncSetAttribute(moe_layer_kernel<MB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        attr = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once, or the launch waits
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_layer_kernel<MB, NT>, a);
}

}  // namespace

bool moe_layer_few(int M, int K, int E, int slots) {
    return M <= kMoeLayerFew && E <= kMoeLayerMaxE &&
           layout(M, K, E, slots, M <= 8 ? 1 : 2).bytes <= kSmemMax;
}

cudaError_t launch_moe_layer_few(MoeLayerArgs a, int meta_bytes, int num_sms, cudaStream_t s) {
    a.slots = std::min(a.E, a.M * a.topk) + a.S;
    a.limit = kWaitNs;
    const int bytes = layout(a.M, a.K, a.E, a.slots, a.M <= 8 ? 1 : 2).bytes;
    if (bytes > kSmemMax) return cudaErrorInvalidValue;
    if (meta_bytes == 4)
        return a.M <= 8 ? launch_few<4, 1>(a, bytes, num_sms, s) : launch_few<4, 2>(a, bytes, num_sms, s);
    return a.M <= 8 ? launch_few<3, 1>(a, bytes, num_sms, s) : launch_few<3, 2>(a, bytes, num_sms, s);
}

cudaError_t launch_moe_router(const MoeLayerArgs& a, cudaStream_t s) {
    const int rows = a.E + (a.sgate ? a.S : 0);
    router_kernel<<<dim3((unsigned)((rows + 7) / 8), (unsigned)((a.M + 15) / 16)), 256, 0, s>>>(a);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    select_kernel<<<(unsigned)((a.M + 3) / 4), 128, 0, s>>>(a);
    return cudaPeekAtLastError();
}

QMLP_BOUNDS_UNIT(moe_layer)

}  // namespace qmlp
