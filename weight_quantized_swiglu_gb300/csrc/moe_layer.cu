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
//  1. x goes to shared memory as fp16 in the order of the MMAs (bf16 times a power of
//     two a token: exact within 2^29 of its largest value), and the router is a
//     product on the same MMAs: its rows are kept as fp16 times a power of two a row
//     (bf16, fp16: exact within 2^29 of the row's largest; fp32: two fp16 words, 22
//     bits), in fragments. Sixteen rows a CTA, k split over CTAs and warps; the
//     CTAs' shares of a logit are added in order by who reads them.
//  2. Every CTA selects by itself (a warp a token, from the logits in L2), lists
//     the experts that any token named, and takes its share of their (expert,
//     eight gate and eight up rows) tiles, ten warps a tile as in moe_awq.cu. All
//     tokens are columns of the MMAs, whether they named the expert or not: the
//     weights bound the time, and no token has to be gathered. act is kept in
//     fp32, a row a (token, choice).
//  3. A warp a (16 output rows, expert): act as fp16 times a power of two of the
//     (token, expert) (its largest value, known now, goes to [2^14, 2^15): off by
//     2^-11 of a value at most, the only rounding between x and out; with an fp32 out
//     what that leaves is taken as well, another fp16), W2 times it;
//     a token's choices are added in their order, fp32. So a token's result does
//     not depend on the other tokens of the call.
// The weights of parts 2 and 3 come through a ring in shared memory that a producer
// warp fills with bulk copies: a W13 tile is one run of codes and one of records in
// the bank, 16 rows of W2 likewise. W2's first ones are on their way before the second
// barrier. (Where the ring does not fit beside x, the warps load for themselves.)
// More tokens: router and selection as two kernels, then the grouped kernels
// (moe_grouped.cu) with the shared experts as further routes, act in fp32 and scaled
// as here.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kTeams = 2;                           // W13 tiles that a CTA has in hand
constexpr int kWarps = kTeams * kMoeKSplit;         // 20
constexpr int kThreads = kWarps * 32;               // and a producer warp
constexpr int kMaxStages = 8;
constexpr uint64_t kWaitNs = 2000000000ull;         // 2 s
constexpr int kSmemMax = 225 * 1024;
constexpr uint16_t kNone = 0xFFFF;

QMLP_DEV uint32_t u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// What the warps of a token's selection share.
struct Pick {
    uint32_t top[32];  // largest keys of 32 groups of experts
    uint32_t key[32];  // candidates: key, expert, logit
    int e[32];
    float l[32];
    float part[16];
    int n;
};
// Splits of the router's k over CTAs.
__host__ __device__ inline int router_splits(int rows, int K, int ctas) {
    const int tiles = (rows + 15) / 16;
    int s = ctas / (tiles > 0 ? tiles : 1);
    if (s > kMoeRouterSplits) s = kMoeRouterSplits;
    while (s > 1 && K / 32 < 2 * s) --s;
    return s < 1 ? 1 : s;
}

// W2's rows of I / 2 bytes would meet on a bank: four units at a time (w2_quads).
__host__ __device__ inline bool quads(int I) { return I % 128 == 0; }
// Shared memory of the kernel (slots: experts that the tokens can name).
struct Layout {
    int x, coef, ridx, slot_e, mask, sel_e, sel_w, cand, part, part_bytes, act16, ring;
    int stage, stages;  // bytes of a ring stage (0: no ring), stages
    int n2, sp;         // W2: experts of a stage, parts of I that different warps take
    int bytes;
};
__host__ __device__ inline Layout layout(int M, int K, int I, int E, int nsel, int slots, int MB, int NT, bool lo) {
    Layout l;
    auto up = [](int b) { return (b + 127) / 128 * 128; };
    int at = 0;
    l.x = at, at += up(M * K * 2);
    l.coef = at, at += up(slots * M * 4);
    l.ridx = at, at += up(slots * M * 2);
    l.slot_e = at, at += up(slots * 4);
    l.mask = at, at += up(E * 4);
    l.sel_e = at, at += 16 * 16 * 4;
    l.sel_w = at, at += 16 * 16 * 4;
    l.cand = at, at += up(M * (int)sizeof(Pick));  // (what follows is read 8 and copied 16 bytes at a time)
    l.part = at, l.part_bytes = 2 * kWarps * 16 * 8 * NT * 4, at += l.part_bytes;
    l.act16 = -1;  // fp16 act of the routes (lo: and what it leaves), where it is small (else in device memory)
    const int act = M * nsel * I * (lo ? 4 : 2);
    if (act <= 32 * 1024) l.act16 = at, at += up(act);
    l.ring = at;
    const int item13 = (int)(kMoeKSplit * (moe_w13_block_bytes(K) + moe_w13_meta_block_bytes(K, MB)));
    const int item2 = 16 * (I / 2) + 16 * (I / 32) * MB;
    l.stage = up(item13 > item2 ? item13 : item2);
    l.stages = (kSmemMax - at) / l.stage;
    if (l.stages > kMaxStages) l.stages = kMaxStages;
    if (l.stages < 2) l.stage = l.stages = 0;
    l.n2 = l.stage ? l.stage / item2 : slots;
    if (l.n2 > 32) l.n2 = 32;
    // where the experts of a stage are few, parts of I go to different warps
    l.sp = 1;
    const int per = l.n2 < slots ? l.n2 : slots;
    while (l.sp < 8 && 2 * l.sp * per <= kWarps && I / 32 >= 4 * l.sp && 2 * M * nsel * 2 * l.sp * 64 <= l.part_bytes) l.sp *= 2;
    l.bytes = at + l.stage * l.stages;
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

// A float as an unsigned number of the same order, above 1; NaN is 1, the lowest.
QMLP_DEV uint32_t order_key(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return max(k, 2u);
}

// Selection for M tokens from their logits lg (rows of E routed experts, then the
// shared gates; shared or global memory) by `wt` warps a token (a power of two): to
// sel_e / sel_w [token][16] in order, the shared experts after the routed ones.
// The topk-th largest of the 32 groups' largest keys is at most the topk-th largest
// key: only the keys from it on are candidates, seldom more than 32 of them, one a lane
// then, whose rank is how many are above it. One token is all latency: its experts go
// over 16 warps, and the code is loops instead of registers (512 experts: 5.8 us by one
// warp in topk rounds of a warp-wide maximum, 5.3 by one warp with candidates).
// sync: a barrier of all warps that call it.
template <typename Sync>
QMLP_DEV void select_tokens(const MoeLayerArgs& a, const float* lg, int M, int wt, Pick* picks, int* sel_e, float* sel_w, Sync sync) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = warp / wt, w = warp % wt;
    const bool on = m < M;
    const float* l = lg + (size_t)(on ? m : 0) * (a.E + a.S);
    Pick& c = picks[on ? m : 0];
    const int e0 = w * 32 + lane, hop = wt * 32, E = on ? a.E : 0;
    if (on && w == 0 && lane == 0) c.n = 0;
    float mx = 0.0f, total = 1.0f;
    if (a.softmax && (!a.renorm || a.bias)) {  // p itself is wanted
        mx = -INFINITY;
        for (int e = e0; e < E; e += hop) mx = fmaxf(mx, l[e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (on && lane == 0) c.part[w] = mx;
        sync();
        for (int i = 0; i < wt; ++i) mx = fmaxf(mx, c.part[i]);
        float s = 0.0f;
        for (int e = e0; e < E; e += hop) s += expf(l[e] - mx);
        s = wsum(s);
        sync();
        if (on && lane == 0) c.part[w] = s;
        sync();
        total = 0.0f;
        for (int i = 0; i < wt; ++i) total += c.part[i];
    }
    auto score = [&](float t) { return a.softmax ? expf(t - mx) / total : 1.0f / (1.0f + expf(-t)); };
    // without a bias the logits have the scores' order
    auto key_of = [&](int e) {
        const float t = l[e];
        return order_key(a.bias ? score(t) + __ldg(a.bias + e) : t);
    };
    uint32_t best = 0;
#pragma unroll 4
    for (int e = e0; e < E; e += hop) best = max(best, key_of(e));
    for (int o = 1; o < wt; o <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (on && lane % wt == 0) c.top[w * (32 / wt) + lane / wt] = best;
    sync();
    {
        const uint32_t mine = c.top[lane];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
            const uint32_t o = c.top[j];
            rank += o > mine || (o == mine && j < lane);
        }
        const uint32_t at = __ballot_sync(0xffffffffu, rank == a.topk - 1);
        const uint32_t least = max(__shfl_sync(0xffffffffu, mine, __ffs(at) - 1), 1u);
#pragma unroll 4
        for (int e = e0; e < E; e += hop) {
            const uint32_t k = key_of(e);
            if (k >= least) {
                const int pos = atomicAdd(&c.n, 1);
                if (pos < 32) {
                    c.key[pos] = k;
                    c.e[pos] = e;
                    c.l[pos] = l[e];
                }
            }
        }
    }
    sync();
    if (!on || w != 0) return;
    int* se = sel_e + m * 16;
    float* sw = sel_w + m * 16;
    float mine = 0.0f;  // lane r: the logit of choice r
    const int n = c.n;
    if (n <= 32) {
        const uint32_t k = lane < n ? c.key[lane] : 0u;
        const int e = lane < n ? c.e[lane] : 0;
        const float f = c.l[lane];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += c.key[j] > k || (c.key[j] == k && c.e[j] < e);
        __syncwarp();
        if (lane < n && rank < a.topk) {
            se[rank] = e;
            c.l[rank] = f;
        }
        __syncwarp();
        mine = c.l[lane];
    } else {  // (many equal ones) round after round
        for (int r = 0; r < a.topk; ++r) {
            uint32_t top = 0;
            int at = 0;
            for (int e = lane; e < E; e += 32) {
                const uint32_t k = key_of(e);
                bool taken = false;
                for (int q = 0; q < r; ++q) taken = taken || se[q] == e;
                if (!taken && k > top) {
                    top = k;
                    at = e;
                }
            }
            const uint32_t all = __reduce_max_sync(0xffffffffu, top);
            const uint32_t e = __reduce_min_sync(0xffffffffu, top == all ? (uint32_t)at : 0xffffffffu);
            if (lane == 0) se[r] = (int)e;
            __syncwarp();
            if (lane == r) mine = l[e];
        }
    }
    // renormed, only the selected scores' ratios count: what they share goes before it
    // underflows. Of softmax any shift will do, the largest selected logit
    if (a.softmax && a.renorm) {
        mx = lane < a.topk ? mine : -INFINITY;
        total = 1.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    // of sigmoids whose logits are all far below zero the largest one's: p = 1 / (1 + exp(-l))
    // is taken over exp(shift)
    float shift = 0.0f;
    if (!a.softmax && a.renorm) {
        shift = lane < a.topk ? mine : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) shift = fmaxf(shift, __shfl_xor_sync(0xffffffffu, shift, o));
        shift = shift < -60.0f ? shift : 0.0f;
    }
    const float p = lane < a.topk ? (a.softmax ? expf(mine - mx) / total : 1.0f / (expf(shift) + expf(shift - mine))) : 0.0f;
    const float sum = a.renorm ? wsum(p) : 1.0f;
    if (lane < a.topk) sw[lane] = p / sum * a.rscale;
    if (lane < a.S) {
        se[a.topk + lane] = a.E + lane;
        sw[a.topk + lane] = a.sgate ? 1.0f / (1.0f + expf(-l[a.E + lane])) : 1.0f;
    }
}

// The MMAs' accumulators to sums of their own: an MMA cuts off what passes its last
// bit, always downward in size, and a chain of 128 of them was 1.4e-6 off, eight at a time 5e-7.
template <int NT>
QMLP_DEV void flush(float (&d)[NT][4], float (&sum)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[n][e] += d[n][e], d[n][e] = 0.0f;
}
// Sixteen rows of the router times NT tiles of eight tokens over pairs of steps
// (32 k) j0 + w, w + hop, ... < j1, both planes of an fp32 router: fragments of 1 KB a
// pair, [plane][tile][pair][2][lane] of 16 bytes. SUM: for long shares of k; the MMAs'
// accumulators, which lose their last bits at every step, go to fp32 sums every eight MMAs (a
// chain over k = 8192: weights 8e-6 to 3.4e-5 off, fp32 arithmetic 4e-7).
template <int NT, bool SUM>
QMLP_DEV void router_tile(const MoeLayerArgs& a, const uint4* xsm, int M, int tile, int j0, int j1, int hop, int lane,
                          float (&d)[NT][4]) {
    const int g = lane >> 2, t = lane & 3, n32 = a.K / 32;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
    float sum[SUM ? NT : 1][4] = {};
    for (int pl = 0; pl < a.planes; ++pl) {
        const uint4* f = a.rfrag + ((size_t)(pl * a.rtiles + tile) * n32) * 64 + lane;
#pragma unroll 2
        for (int j = j0; j < j1; j += hop) {
            if (!QMLP_INB((size_t)(f - a.rfrag) + (size_t)j * 64 + 32, a.rfrag_elems, 105)) continue;
            const uint4 a0 = __ldg(f + (size_t)j * 64), a1 = __ldg(f + (size_t)j * 64 + 32);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x = xsm[(j * M + min(8 * n + g, M - 1)) * 4 + t];
                mma_f16_16816(d[n], a0.x, a0.y, a0.z, a0.w, x.x, x.y);
                mma_f16_16816(d[n], a1.x, a1.y, a1.z, a1.w, x.z, x.w);
            }
            if constexpr (SUM)
                if ((((j - j0) / hop) & 3) == 3 || j + hop >= j1) flush<NT>(d, sum);
        }
    }
    if constexpr (SUM)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[n][e] = sum[n][e];
}
// The order of a lane's eight k of a unit of 32, for A and B alike: a byte of the
// lane-sliced banks holds two neighbours, and the codes are taken as nibbles p and p +
// 4 of the word, so pairs (2t, 16 + 2t), (2t + 1, 17 + 2t), (8 + 2t, 24 + 2t),
// (9 + 2t, 25 + 2t); the first two are one MMA's, the others the next one's.
// From v[i] = k 8 i + 2t and its neighbour (packed halves) to that order.
QMLP_DEV uint4 unit_order(uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
    return make_uint4(__byte_perm(v0, v2, 0x5410), __byte_perm(v0, v2, 0x7632), __byte_perm(v1, v3, 0x5410),
                      __byte_perm(v1, v3, 0x7632));
}
// x [M, K] -> fp16 in that order, by `threads` threads: slot (j M + m) 4 + t has unit j
// of token m for lanes t; the tokens' exponents to sig. A thread stays with a token:
// the row's largest value falls out of the copy, which is then scaled in place.
template <typename Sync>
QMLP_DEV void stage_x(const MoeLayerArgs& a, const void* x, int M, uint4* xsm, int* s_max, int* sig, int threads, Sync sync) {
    const int K = a.K, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = threads >> 5;
    const int wpt = max(1, nw / M);  // warps a token
    if (threadIdx.x < 16) s_max[threadIdx.x] = 0;
    sync();
    for (int m = warp / wpt; m < M; m += nw / wpt) {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(x) + (size_t)m * K);
        float mx = 0.0f;
        // lane t of unit j: word t of its four pieces (16 bytes in four places at once met on
        // a bank: 8 tokens of 2560 4.1 us). All loads of a batch are under way together (the
        // rest of an unrolled loop goes one by one).
        constexpr int kBatch = 6;
        for (int q0 = (warp % wpt) * 32 + lane; q0 < K / 8; q0 += 32 * wpt * kBatch) {
            uint32_t w[kBatch][4];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int q = q0 + 32 * wpt * b, at = 16 * (q >> 2) + (q & 3);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[b][i] = q < K / 8 ? row[at + 4 * i] : 0u;
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int q = q0 + 32 * wpt * b;
                if (q >= K / 8) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[b][i] << 16)), fabsf(__uint_as_float(w[b][i] & 0xFFFF0000u))));
                xsm[((q >> 2) * M + m) * 4 + (q & 3)] = a.x_bf16 ? make_uint4(w[b][0], w[b][1], w[b][2], w[b][3])
                                                                 : unit_order(w[b][0], w[b][1], w[b][2], w[b][3]);
            }
        }
        if (a.x_bf16) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) atomicMax(s_max + m, __float_as_int(mx));
        }
    }
    sync();
    if (threadIdx.x < 16) sig[threadIdx.x] = a.x_bf16 ? prescale_exponent(__int_as_float(s_max[threadIdx.x])) : 0;
    if (a.x_bf16)  // a thread's own pieces again
        for (int m = warp / wpt; m < M; m += nw / wpt) {
            const int sg = prescale_exponent(__int_as_float(s_max[m]));
            const float p0 = __int_as_float((127 + (sg >> 1)) << 23), p1 = __int_as_float((127 + sg - (sg >> 1)) << 23);
#pragma unroll 2
            for (int q = (warp % wpt) * 32 + lane; q < K / 8; q += 32 * wpt) {
                uint4* at = xsm + ((q >> 2) * M + m) * 4 + (q & 3);
                const uint4 u = *at;
                uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = u32(__floats2half2_rn(__uint_as_float(v[j] << 16) * p0 * p1, __uint_as_float(v[j] & 0xFFFF0000u) * p0 * p1));
                *at = unit_order(v[0], v[1], v[2], v[3]);
            }
        }
    sync();
}

// ---------------------------------------------------------------------------
// Weight decode with the values of moe_awq.cu: half_fma(q, s, b)
// ---------------------------------------------------------------------------
QMLP_DEV uint32_t lfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
QMLP_DEV uint32_t ladd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// {scale, scale} and {bias, bias} of a record: the bias is stored (4 bytes) or
// half(-zero scale): -(1024 + z) + 1024 is exact, and the product rounds once.
template <int MB>
QMLP_DEV void meta2(uint32_t m, uint32_t& s2, uint32_t& b2) {
    s2 = __byte_perm(m, 0, 0x1010);
    if (MB == 4) b2 = __byte_perm(m, 0, 0x3232);
    else b2 = hmul2_u32(ladd2(__byte_perm(m, 0xE4E4E4E4u, 0x4242), 0x64006400u), s2);
}
// (w & mask) | magic in one instruction (the compiler took two)
QMLP_DEV uint32_t and_or(uint32_t w, uint32_t mask) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x64006400u));
    return d;
}
// A lane's word of a unit (eight weights of a row) in the order above: nibbles p and p +
// 4 are pair p; 0x6400 | q is 1024 + q, 0x6400 | 16 q is 1024 + 16 q; q comes out exact
// and half_fma rounds once. (Byte by byte, PRMT and LOP3 for two weights: 8 integer
// instructions a word instead of 5.)
QMLP_DEV void word_weights(uint32_t w, uint32_t s2, uint32_t b2, uint32_t (&f)[4]) {
    const uint32_t v = w >> 8;
    f[0] = lfma2(ladd2(and_or(w, 0x000F000Fu), 0xE400E400u), s2, b2);
    f[1] = lfma2(lfma2(and_or(w, 0x00F000F0u), 0x2C002C00u, 0xD400D400u), s2, b2);
    f[2] = lfma2(ladd2(and_or(v, 0x000F000Fu), 0xE400E400u), s2, b2);
    f[3] = lfma2(lfma2(and_or(v, 0x00F000F0u), 0x2C002C00u, 0xD400D400u), s2, b2);
}
// One unit of 32 k of sixteen rows (words and records of rows g and g + 8) times NT
// tiles of tokens.
// LO: xl, what x's rounding left, as well.
template <int NT, bool LO = false>
QMLP_DEV void words_mma(uint32_t w0, uint32_t w8, uint32_t s0, uint32_t b0, uint32_t s8, uint32_t b8, const uint4 (&x)[NT],
                        const uint4 (&xl)[NT], float (&d)[NT][4]) {
    uint32_t f0[4], f8[4];
    word_weights(w0, s0, b0, f0);
    word_weights(w8, s8, b8, f8);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mma_f16_16816(d[n], f0[0], f8[0], f0[1], f8[1], x[n].x, x[n].y);
        mma_f16_16816(d[n], f0[2], f8[2], f0[3], f8[3], x[n].z, x[n].w);
        if (LO) {
            mma_f16_16816(d[n], f0[0], f8[0], f0[1], f8[1], xl[n].x, xl[n].y);
            mma_f16_16816(d[n], f0[2], f8[2], f0[3], f8[3], xl[n].z, xl[n].w);
        }
    }
}
template <int MB, int NT, bool LO = false>
QMLP_DEV void unit_mma(uint32_t w0, uint32_t w8, uint32_t m0, uint32_t m8, const uint4 (&x)[NT], const uint4 (&xl)[NT],
                       float (&d)[NT][4]) {
    uint32_t s0, b0, s8, b8;
    meta2<MB>(m0, s0, b0);
    meta2<MB>(m8, s8, b8);
    words_mma<NT, LO>(w0, w8, s0, b0, s8, b8, x, xl, d);
}
template <int MB>
QMLP_DEV uint32_t record(const uint8_t* p) {
    if (MB == 4) return *reinterpret_cast<const uint32_t*>(p);
    return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
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

// Sixteen bytes of device memory, where `on`: else zeros, without a branch.
QMLP_DEV uint4 ldcg4_if(const uint4* p, bool on) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)on));
    return v;
}

// act (fp32, rows of I) -> fp16 times the row's power of two, in the order of the
// MMAs: piece (r I / 32 + unit) 4 + t, to `out` (shared or device memory), by threads
// i0, i0 + hop, ...
template <bool QUAD, bool LO>
QMLP_DEV void convert_act(const MoeLayerArgs& a, int rows, uint4* out, size_t out_elems, int i0, int hop) {
    const bool quad = QUAD && quads(a.I);
    const int nu = a.I / 32;
    constexpr int kBatch = LO ? 2 : 3;  // (88 rows of 160: all loads under way together)
    for (int b0 = i0; b0 < rows * nu * 4; b0 += hop * kBatch) {
        float2 v[kBatch][4];
        int top[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = b0 + b * hop, t = i & 3;
            const bool in = i < rows * nu * 4 && QMLP_INB((size_t)(i >> 2) * 32 + 31, a.act_elems, 107);
            const float* p = a.act + (size_t)(in ? i >> 2 : 0) * 32 + 2 * t;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[b][j] = in ? __ldcg(reinterpret_cast<const float2*>(p + 8 * j)) : make_float2(0.0f, 0.0f);
            top[b] = in ? __ldcg(a.amax + (i >> 2) / nu) : 0;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = b0 + b * hop, t = i & 3, u = (i >> 2) % nu;
            if (i >= rows * nu * 4 || !QMLP_INB((LO ? rows * nu * 4 : 0) + i, out_elems, 109)) continue;
            const float up = __int_as_float((127 + act_exponent(top[b])) << 23);
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 w = make_float2(v[b][j].x * up, v[b][j].y * up);
                const __half2 q = __floats2half2_rn(w.x, w.y);
                h[j] = u32(q);
                if (LO) {  // (nothing of what is not finite)
                    const float2 f = __half22float2(q);
                    l[j] = u32(__floats2half2_rn(isfinite(f.x) ? w.x - f.x : 0.0f, isfinite(f.y) ? w.y - f.y : 0.0f));
                }
            }
            // (of four units: lane t's pieces are unit t's, see w2_quads)
            const int at = quad ? i + 3 * (t - (u & 3)) : i;
            out[at] = unit_order(h[0], h[1], h[2], h[3]);
            if (LO) out[rows * nu * 4 + at] = unit_order(l[0], l[1], l[2], l[3]);
        }
    }
}

// A unit's results, times the weights, to part.
template <int NT>
QMLP_DEV void unit_out(const float (&d)[NT][4], int M, int t, int g, const uint16_t* ridx, const float* coef, float* part) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = 8 * n + 2 * t + e, r = m < M ? ridx[m] : kNone;
            if (r != kNone) {  // a choice of token m: its rows g and g + 8
                const float w = coef[m];
                part[r * 16 + g] = w * d[n][e];
                part[r * 16 + g + 8] = w * d[n][2 + e];
            }
        }
}

// Part 3's share of one expert: sixteen rows (codes, meta) times the tokens' act (fp16,
// converted; SH: in shared memory) over units u0..u1 of 32 k, times the weights, to
// part (choice r of the call: r 16 + row).
template <int MB, int NT, bool SH, bool LO>
QMLP_DEV void w2_unit(const MoeLayerArgs& a, const uint8_t* codes, const uint8_t* meta, const uint4* act16, int u0, int u1,
                      const uint16_t* ridx, const float* coef, float* part, size_t lo, int lane) {
    const int M = a.M, I = a.I, nu = I / 32, g = lane >> 2, t = lane & 3;
    float d[NT][4], sum[NT][4];
    const uint4* row[NT];
    bool on[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g, r = m < M ? ridx[m] : kNone;
        on[n] = r != kNone;
        row[n] = act16 + (size_t)(on[n] ? r : 0) * nu * 4 + t;
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = sum[n][e] = 0.0f;
    }
    const uint8_t *c0 = codes + g * (I / 2) + 4 * t, *c8 = c0 + 4 * I;
    const uint8_t *m0 = meta + g * nu * MB, *m8 = m0 + 8 * nu * MB;
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
        uint4 x[NT], xl[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (SH) x[n] = on[n] ? row[n][u * 4] : make_uint4(0, 0, 0, 0);
            else x[n] = ldcg4_if(row[n] + u * 4, on[n]);
            if (!LO) continue;
            if (SH) xl[n] = on[n] ? row[n][lo + u * 4] : make_uint4(0, 0, 0, 0);
            else xl[n] = ldcg4_if(row[n] + lo + u * 4, on[n]);
        }
        uint32_t r0, r8;
        if (MB == 4) {
            r0 = *reinterpret_cast<const uint32_t*>(m0 + u * 4);
            r8 = *reinterpret_cast<const uint32_t*>(m8 + u * 4);
        } else {
            r0 = (uint32_t)m0[u * 3] | (uint32_t)m0[u * 3 + 1] << 8 | (uint32_t)m0[u * 3 + 2] << 16;
            r8 = (uint32_t)m8[u * 3] | (uint32_t)m8[u * 3 + 1] << 8 | (uint32_t)m8[u * 3 + 2] << 16;
        }
        unit_mma<MB, NT, LO>(*reinterpret_cast<const uint32_t*>(c0 + 16 * u), *reinterpret_cast<const uint32_t*>(c8 + 16 * u), r0,
                         r8, x, xl, d);
        if (LO && (u & 1)) flush<NT>(d, sum);
    }
    if (LO) flush<NT>(d, sum);
    unit_out<NT>(LO ? sum : d, M, t, g, ridx, coef, part);
}

// The same with act in device memory, four units at a time: lane t takes unit u + t whole, a
// word of it a step, one read of 16 bytes a row and a record for the four. (A word a unit
// has four or eight rows on one bank where I is a multiple of 128: 4 tokens of 64 experts
// of 4096 x 1024 103 us instead of 87; elsewhere it is ahead, I = 704 84 to 88 us.) act lies
// in that order, and is asked for PF steps ahead.
template <int MB, int NT, bool LO>
QMLP_DEV void w2_quads(const MoeLayerArgs& a, const uint8_t* codes, const uint8_t* meta, const uint4* act16, int u0, int u1,
                       const uint16_t* ridx, const float* coef, float* part, size_t lo, int lane) {
    constexpr int PF = 4 / (NT * (LO ? 2 : 1));
    const int M = a.M, I = a.I, nu = I / 32, g = lane >> 2, t = lane & 3;
    float d[NT][4], sum[NT][4];
    const uint4* row[NT];
    bool on[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g, r = m < M ? ridx[m] : kNone;
        on[n] = r != kNone;
        row[n] = act16 + (size_t)(on[n] ? r : 0) * nu * 4 + t;
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = sum[n][e] = 0.0f;
    }
    const uint8_t *c0 = codes + g * (I / 2) + 16 * t, *c8 = c0 + 4 * I;
    const uint8_t *m0 = meta + (g * nu + t) * MB, *m8 = m0 + 8 * nu * MB;
    uint4 x[PF][NT], xl[PF][NT];
    auto ask = [&](int u, uint4 (&v)[NT], uint4 (&vl)[NT]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            v[n] = ldcg4_if(row[n] + u * 4, on[n] && u < u1);
            if (LO) vl[n] = ldcg4_if(row[n] + lo + u * 4, on[n] && u < u1);
        }
    };
#pragma unroll
    for (int j = 0; j < PF; ++j) ask(u0 + j, x[j], xl[j]);
#pragma unroll 1
    for (int u = u0; u < u1; u += 4) {
        const uint4 p = *reinterpret_cast<const uint4*>(c0 + 16 * u), q = *reinterpret_cast<const uint4*>(c8 + 16 * u);
        const uint32_t w0[4] = {p.x, p.y, p.z, p.w}, w8[4] = {q.x, q.y, q.z, q.w};
        uint32_t s0, b0, s8, b8;
        meta2<MB>(record<MB>(m0 + u * MB), s0, b0);
        meta2<MB>(record<MB>(m8 + u * MB), s8, b8);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            words_mma<NT, LO>(w0[j], w8[j], s0, b0, s8, b8, x[j % PF], xl[j % PF], d);
            ask(u + j + PF, x[j % PF], xl[j % PF]);
            if (LO && (j & 1)) flush<NT>(d, sum);
        }
    }
    unit_out<NT>(LO ? sum : d, M, t, g, ridx, coef, part);
}

template <int MB, int NT, bool RING, bool LO>
__global__ void __launch_bounds__(kThreads + 32, 1) moe_layer_kernel(const MoeLayerArgs a) {
    constexpr int kC = 8 * NT;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int s_pass, s_n, s_max[16], s_sig[16], s_cnt[kWarps];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
    const int M = a.M, K = a.K, I = a.I, rows = a.E + (a.sgate ? a.S : 0), nsel = a.topk + a.S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Layout L = layout(M, K, I, a.E, nsel, a.slots, MB, NT, LO);
    uint4* xsm = reinterpret_cast<uint4*>(sm + L.x);
    float* coef = reinterpret_cast<float*>(sm + L.coef);          // [slot][M]
    uint16_t* ridx = reinterpret_cast<uint16_t*>(sm + L.ridx);    // [slot][M]: row of act
    int* slot_e = reinterpret_cast<int*>(sm + L.slot_e);
    uint32_t* mask = reinterpret_cast<uint32_t*>(sm + L.mask);    // [E]: tokens that named it, then its slot
    int* sel_e = reinterpret_cast<int*>(sm + L.sel_e);            // [16][16]
    float* sel_w = reinterpret_cast<float*>(sm + L.sel_w);
    Pick* picks = reinterpret_cast<Pick*>(sm + L.cand);           // [M]
    float* part = reinterpret_cast<float*>(sm + L.part);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    // (one split where the logits have no room in shared memory)
    const int splits = M * (a.E + a.S) * 4 <= L.part_bytes ? router_splits(rows, K, gridDim.x) : 1, ctile = (rows + 15) / 16;
    const size_t hop = (size_t)M * (a.E + a.S);  // between the splits' shares of the logits
    if (RING && threadIdx.x == 0) {
        for (int s = 0; s < L.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kMoeKSplit);  // a team; W2's stages: every warp, see below
        }
        fence_mbar_init();
    }

    // ---------------- 1: x, router ----------------
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < M * nsel; i += gridDim.x * kThreads) a.amax[i] = 0;
    for (int e = threadIdx.x; e < a.E; e += kThreads) mask[e] = 0;
    if (warp < kWarps) {
        stage_x(a, a.x, M, xsm, s_max, s_sig, kThreads, [] { named_bar_sync(1, kThreads); });
        const int n32 = K / 32;
        for (int u = blockIdx.x; u < ctile * splits; u += gridDim.x) {
            const int tile = u / splits, sp = u % splits;
            const int j0 = (int)((long)sp * n32 / splits), j1 = (int)((long)(sp + 1) * n32 / splits);
            float d[NT][4];
            router_tile<NT, false>(a, xsm, M, tile, j0 + warp, j1, kWarps, lane, d);
            if (u != (int)blockIdx.x) named_bar_sync(1, kThreads);  // the sums before are read
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(part + (warp * 16 + g) * kC + 8 * n + 2 * t) = make_float2(d[n][0], d[n][1]);
                *reinterpret_cast<float2*>(part + (warp * 16 + g + 8) * kC + 8 * n + 2 * t) = make_float2(d[n][2], d[n][3]);
            }
            named_bar_sync(1, kThreads);
            for (int i = threadIdx.x; i < 16 * M; i += kThreads) {
                const int r = i & 15, m = i >> 4, row = tile * 16 + r;
                if (row < rows) {
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += part[(w * 16 + r) * kC + m];
                    const size_t at = sp * hop + (size_t)m * (a.E + a.S) + row;
                    if (QMLP_INB(at, a.logit_elems, 105)) a.logits[at] = scalbnf(v, -s_sig[m] - a.rexp[row]);
                }
            }
        }
    }
    // (a barrier that ran out: the CTA still counts for those that it will not reach)
    const unsigned long long further = L.act16 < 0 ? 2ull : 1ull;
    if (!grid_barrier(a, &s_pass)) {
        if (threadIdx.x == 0) atomicAdd(a.ticket, further);
        return;
    }

    // ---------------- 2: selection, W13 ----------------
    {
        // the logits: the splits' shares in order, in shared memory where there is room
        const int all = M * (a.E + a.S);
        const bool room = all * 4 <= L.part_bytes;
        float* lg = room ? part : a.logits;
        if (warp < kWarps && room) {
            constexpr int kBatch = 7;  // (8 tokens of 512 experts: all loads under way together)
            for (int i0 = threadIdx.x; i0 < all; i0 += kThreads * kBatch) {
                float v[kBatch][kMoeRouterSplits];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
#pragma unroll
                    for (int s = 0; s < kMoeRouterSplits; ++s)
                        v[b][s] = s < splits && i0 + b * kThreads < all ? __ldcg(a.logits + s * hop + i0 + b * kThreads) : 0.0f;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
#pragma unroll
                    for (int s = 1; s < kMoeRouterSplits; ++s)
                        if (s < splits) v[b][0] += v[b][s];
                    if (i0 + b * kThreads < all) part[i0 + b * kThreads] = v[b][0];
                }
            }
        }
        if (warp < kWarps) {
            named_bar_sync(1, kThreads);
            select_tokens(a, lg, M, M == 1 ? 16 : M == 2 ? 8 : M <= 4 ? 4 : M <= 8 ? 2 : 1, picks, sel_e, sel_w,
                          [] { named_bar_sync(1, kThreads); });
        }
    }
    __syncthreads();
    int slots;
    if (M == 1) {  // the choices are the list
        slots = nsel;
        if ((int)threadIdx.x < nsel) {
            slot_e[threadIdx.x] = sel_e[threadIdx.x];
            ridx[threadIdx.x] = (uint16_t)threadIdx.x;
            coef[threadIdx.x] = sel_w[threadIdx.x];
        }
    } else {
        for (int i = threadIdx.x; i < M * a.topk; i += kThreads + 32)
            atomicOr(&mask[sel_e[(i / a.topk) * 16 + i % a.topk]], 1u << (i / a.topk));
        __syncthreads();
        // the experts named, in their order, then the shared ones: experts a warp, its
        // lanes side by side
        const int per = (a.E + kWarps - 1) / kWarps;
        if (warp < kWarps) {
            int n = 0;
            for (int b = 0; b < per; b += 32) {
                const int e = warp * per + b + lane;
                n += __popc(__ballot_sync(0xffffffffu, b + lane < per && e < a.E && mask[e] != 0));
            }
            if (lane == 0) s_cnt[warp] = n;
        }
        __syncthreads();
        if (warp < kWarps) {
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
        const int named = s_n;
        slots = named + a.S;
        for (int i = threadIdx.x; i < slots * M; i += kThreads + 32) {
            ridx[i] = kNone;
            coef[i] = 0.0f;
        }
        for (int j = threadIdx.x; j < a.S; j += kThreads + 32) slot_e[named + j] = a.E + j;
        __syncthreads();
        for (int i = threadIdx.x; i < M * nsel; i += kThreads + 32) {
            const int m = i / nsel, r = i % nsel;
            const int s = r < a.topk ? (int)mask[sel_e[m * 16 + r]] : named + r - a.topk;
            ridx[s * M + m] = (uint16_t)i;
            coef[s * M + m] = sel_w[m * 16 + r];
        }
    }
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < M * a.topk; i += kThreads + 32) {
            const int m = i / a.topk, r = i % a.topk;
            if (a.ids_out) a.ids_out[i] = sel_e[m * 16 + r];
            if (a.w_out) a.w_out[i] = sel_w[m * 16 + r];
        }
    __syncthreads();

    const int no = I / 8, items = slots * no, np = moe_w13_pairs(K), ms = moe_w13_meta_stride(K, MB), cpw = moe_w13_cpw(K);
    const int cb = (int)moe_w13_block_bytes(K), mb = (int)moe_w13_meta_block_bytes(K, MB);  // a warp's blocks
    const int cb2 = 16 * (I / 2), mb2 = 16 * (I / 32) * MB;                                  // 16 rows of W2
    const int n13 = items > (int)blockIdx.x ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;  // this CTA's tiles
    const int tiles2 = K / 16 > (int)blockIdx.x ? (K / 16 - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const int st2 = (slots + L.n2 - 1) / L.n2, n2 = tiles2 * st2;  // stages of W2: an expert group of a tile each
    // ---------------- the producer's side of the ring ----------------
    bool ok = true;
    auto claim = [&](int it) {  // stage it % L.stages is free
        if (it < L.stages) return true;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(it % L.stages), (uint32_t)((it / L.stages - 1) & 1), a.limit))) {
            if (lane == 0) atomicExch(a.err, 102);
            ok = false;
        }
        return ok;
    };
    auto send13 = [&](int it) {
        const int s = it % L.stages, item = blockIdx.x + it * gridDim.x;
        const size_t blk = ((size_t)slot_e[item / no] * no + item % no) * kMoeKSplit;
        if (lane == 0) mbar_arrive_expect_tx(full(s), (uint32_t)(kMoeKSplit * (cb + mb)));
        __syncwarp();
        const uint32_t dst = smem_u32(sm + L.ring) + (uint32_t)(s * L.stage);
        if (lane == 0) {
            const uint8_t* p = a.w13 + blk * cb;
            if (!QMLP_INB((blk + kMoeKSplit) * cb - 1, a.w13_bytes, 101)) p = a.w13;
            bulk_g2s(dst, p, (uint32_t)(kMoeKSplit * cb), full(s));
        } else if (lane == 1) {
            const uint8_t* p = a.w13_meta + blk * mb;
            if (!QMLP_INB((blk + kMoeKSplit) * mb - 1, a.w13_meta_bytes, 102)) p = a.w13_meta;
            bulk_g2s(dst + (uint32_t)(kMoeKSplit * cb), p, (uint32_t)(kMoeKSplit * mb), full(s));
        }
    };
    auto send2 = [&](int it) {  // it counts on from W13's
        const int s = it % L.stages, j = it - n13, s0 = j % st2 * L.n2, n = min(L.n2, slots - s0);
        const int tile = blockIdx.x + j / st2 * gridDim.x;
        if (lane == 0) mbar_arrive_expect_tx(full(s), (uint32_t)(n * (cb2 + mb2)));
        __syncwarp();
        if (lane < n) {
            const size_t row = (size_t)slot_e[s0 + lane] * K + 16 * tile;
            const uint32_t dst = smem_u32(sm + L.ring) + (uint32_t)(s * L.stage + lane * (cb2 + mb2));
            const uint8_t *p = a.w2 + row * (I / 2), *q = a.w2_meta + row * (I / 32) * MB;
            if (!QMLP_INB((row + 16) * (I / 2) - 1, a.w2_bytes, 103)) p = a.w2;
            if (!QMLP_INB((row + 16) * (I / 32) * MB - 1, a.w2_meta_bytes, 104)) q = a.w2_meta;
            bulk_g2s(dst, p, (uint32_t)cb2, full(s));
            bulk_g2s(dst + (uint32_t)cb2, q, (uint32_t)mb2, full(s));
        }
    };
    int sent = 0;
    if (RING && warp == kWarps) {
        for (; sent < n13 && claim(sent); ++sent) send13(sent);
        // what fits of W2 (every stage of W13 is consumed before the barrier)
        for (; ok && sent < n13 + min(n2, L.stages) && claim(sent); ++sent) send2(sent);
    }
    bool late = false;
    auto arrived = [&](int it) {
        const uint32_t bar = full(it % L.stages), par = (uint32_t)((it / L.stages) & 1);
        if (mbar_try_wait(bar, par)) return;
        if (!mbar_wait_bounded(bar, par, late ? 0 : a.limit)) {
            atomicExch(a.err, 103);  // (what is then read lies in the ring; out is not valid)
            late = true;
        }
    };

    if (warp < kWarps) {
        const int team = warp / kMoeKSplit, ks = warp % kMoeKSplit, tid = threadIdx.x - team * kMoeKSplit * 32;
        const int Kc = K / 64, c0 = ks * cpw, nc = max(0, min(Kc, c0 + cpw) - c0);
        int turn = 0;
        for (int it = team; it < n13; it += kTeams, turn ^= 1) {
            const int item = blockIdx.x + it * gridDim.x, s = item / no, oct = item % no;
            const uint8_t *codes, *meta;
            bool in = true;
            if (RING) {
                arrived(it);
                codes = sm + L.ring + (it % L.stages) * L.stage + ks * cb;
                meta = sm + L.ring + (it % L.stages) * L.stage + kMoeKSplit * cb + ks * mb;
            } else {
                const size_t blk = ((size_t)slot_e[s] * no + oct) * kMoeKSplit + ks;
                codes = a.w13 + blk * cb;
                meta = a.w13_meta + blk * mb;
                in = QMLP_INB((blk + 1) * cb - 1, a.w13_bytes, 101) && QMLP_INB((blk + 1) * mb - 1, a.w13_meta_bytes, 102);
            }
            float d[NT][4], sum[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = sum[n][e] = 0.0f;
            // pairs of 64-k chunks: four units of the gate row g and of the up row g
            const uint4* cp = reinterpret_cast<const uint4*>(codes) + lane;
            const uint8_t* mp = meta + g * ms;
#pragma unroll 2
            for (int pr = 0; pr < (nc + 1) / 2; ++pr) {
                if (!in) break;
                const uint4 cg = cp[pr * 32], cu = cp[(np + pr) * 32];
                const uint32_t wg[4] = {cg.x, cg.y, cg.z, cg.w}, wu[4] = {cu.x, cu.y, cu.z, cu.w};
                uint32_t rg[4], ru[4];
                if (MB == 4) {
                    const uint4 p = *reinterpret_cast<const uint4*>(mp + pr * 16), q = *reinterpret_cast<const uint4*>(mp + 8 * ms + pr * 16);
                    rg[0] = p.x, rg[1] = p.y, rg[2] = p.z, rg[3] = p.w;
                    ru[0] = q.x, ru[1] = q.y, ru[2] = q.z, ru[3] = q.w;
                } else {
                    const uint32_t *p = reinterpret_cast<const uint32_t*>(mp + pr * 12), *q = reinterpret_cast<const uint32_t*>(mp + 8 * ms + pr * 12);
                    const uint32_t a0 = p[0], a1 = p[1], a2 = p[2], e0 = q[0], e1 = q[1], e2 = q[2];
                    rg[0] = a0, rg[1] = __funnelshift_r(a0, a1, 24), rg[2] = __funnelshift_r(a1, a2, 16), rg[3] = a2 >> 8;
                    ru[0] = e0, ru[1] = __funnelshift_r(e0, e1, 24), ru[2] = __funnelshift_r(e1, e2, 16), ru[3] = e2 >> 8;
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (2 * pr + (h >> 1) < nc) {
                        uint4 x[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            x[n] = xsm[(((c0 + 2 * pr) * 2 + h) * M + min(8 * n + g, M - 1)) * 4 + t];
                        unit_mma<MB, NT>(wg[h], wu[h], rg[h], ru[h], x, x, d);
                    }
                }
                if (LO) flush<NT>(d, sum);
            }
            if (RING) {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(it % L.stages));
            }
            float (&v)[NT][4] = LO ? sum : d;
            float* pt = part + ((turn * kTeams + team) * kMoeKSplit) * 16 * kC;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(pt + (ks * 16 + g) * kC + 8 * n + 2 * t) = make_float2(v[n][0], v[n][1]);
                *reinterpret_cast<float2*>(pt + (ks * 16 + g + 8) * kC + 8 * n + 2 * t) = make_float2(v[n][2], v[n][3]);
            }
            named_bar_sync(1 + team, kMoeKSplit * 32);
            if (tid < 8 * kC) {
                const int row = tid & 7, m = tid >> 3;
                if (m < M && ridx[s * M + m] != kNone) {
                    float hg = 0.0f, hu = 0.0f;
#pragma unroll
                    for (int w = 0; w < kMoeKSplit; ++w) {
                        hg += pt[(w * 16 + row) * kC + m];
                        hu += pt[(w * 16 + 8 + row) * kC + m];
                    }
                    const int sg = s_sig[m], r = ridx[s * M + m];
                    const float v = silu_f32(scalbnf(hg, -sg)) * scalbnf(hu, -sg);
                    if (QMLP_INB((size_t)r * I + 8 * oct + row, a.act_elems, 106)) a.act[(size_t)r * I + 8 * oct + row] = v;
                    // the eight rows of a token are neighbours in a warp; the largest
                    // of them does not depend on the order of the tiles
                    const uint32_t top = __reduce_max_sync(0xFFu << (lane & 24), __float_as_uint(fabsf(v)));
                    if (row == 0) atomicMax(a.amax + r, (int)top);
                }
            }
        }
    }
    if (!grid_barrier(a, &s_pass)) {
        if (threadIdx.x == 0 && further > 1) atomicAdd(a.ticket, 1ull);
        // (copies in flight end before the CTA does)
        if (RING && warp == kWarps)
            for (int q = sent - 1; q >= 0 && q >= sent - L.stages; --q)
                mbar_wait_bounded(full(q % L.stages), (uint32_t)((q / L.stages) & 1), a.limit);
        return;
    }

    if (L.act16 < 0) {  // act has no room in shared memory: converted once, a third barrier
        if (warp < kWarps)
            convert_act<true, LO>(a, M * nsel, a.act16, a.act16_elems, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
        if (!grid_barrier(a, &s_pass)) {
            if (RING && warp == kWarps)
                for (int q = sent - 1; q >= 0 && q >= sent - L.stages; --q)
                    mbar_wait_bounded(full(q % L.stages), (uint32_t)((q / L.stages) & 1), a.limit);
            return;
        }
    }

    // ---------------- 3: W2 and the weighted sum ----------------
    if (warp == kWarps) {
        if (RING) {
            for (; ok && sent < n13 + n2 && claim(sent); ++sent) send2(sent);
            if (!ok)
                for (int q = sent - 1; q >= 0 && q >= sent - L.stages; --q)
                    mbar_wait_bounded(full(q % L.stages), (uint32_t)((q / L.stages) & 1), a.limit);
        }
        return;
    }
    const int nu = I / 32, prow = M * nsel;
    const bool quad = L.act16 < 0 && quads(I);
    const int step = quad ? 4 : 1;
    const int first_r = (int)threadIdx.x < slots * M ? ridx[threadIdx.x] : kNone;
    const int first_max = first_r != kNone ? __ldcg(a.amax + first_r) : 0;  // (on its way while act is converted)
    const uint4* act16 = a.act16;
    if (L.act16 >= 0) {  // every CTA for itself
        convert_act<false, LO>(a, prow, reinterpret_cast<uint4*>(sm + L.act16), (size_t)prow * nu * (LO ? 8 : 4), threadIdx.x, kThreads);
        act16 = reinterpret_cast<const uint4*>(sm + L.act16);
    }
    for (int i = threadIdx.x; i < slots * M; i += kThreads) {
        const int r = ridx[i];
        if (r == kNone) continue;
        coef[i] *= __int_as_float((127 - act_exponent(i == (int)threadIdx.x ? first_max : __ldcg(a.amax + r))) << 23);
    }
    named_bar_sync(1, kThreads);
    int first = 0;  // the warp that takes the next unit: the units of all stages go round
    for (int tl = 0; tl < tiles2; tl += 2) {  // two tiles between barriers
        const int nt = min(2, tiles2 - tl);
        for (int q = 0; q < nt; ++q)
            for (int j = 0; j < st2; ++j) {
                const int tile = blockIdx.x + (tl + q) * gridDim.x;
                const int it = n13 + (tl + q) * st2 + j, s0 = j * L.n2, n = min(L.n2, slots - s0);
                const uint8_t* stage = sm + L.ring + (RING ? it % L.stages * L.stage : 0);
                if (RING) arrived(it);
                int u = warp - first;
                for (u += u < 0 ? kWarps : 0; u < n * L.sp; u += kWarps) {
                    const int s = s0 + u / L.sp, ip = u % L.sp, u0 = ip * (nu / step) / L.sp * step;
                    const int u1 = ip + 1 < L.sp ? (ip + 1) * (nu / step) / L.sp * step : nu;
                    float* pp = part + (q * L.sp + ip) * prow * 16;
                    const uint8_t *codes, *meta;
                    bool in = true;
                    if (RING) {
                        codes = stage + (u / L.sp) * (cb2 + mb2);
                        meta = codes + cb2;
                    } else {
                        const size_t row = (size_t)slot_e[s] * K + 16 * tile;
                        codes = a.w2 + row * (I / 2);
                        meta = a.w2_meta + row * (I / 32) * MB;
                        in = QMLP_INB((row + 16) * (I / 2) - 1, a.w2_bytes, 103) &&
                             QMLP_INB((row + 16) * (I / 32) * MB - 1, a.w2_meta_bytes, 104);
                    }
                    if (!in) continue;
                    if (quad)
                        w2_quads<MB, NT, LO>(a, codes, meta, act16, u0, u1, ridx + s * M, coef + s * M, pp, (size_t)prow * nu * 4, lane);
                    else if (L.act16 >= 0)
                        w2_unit<MB, NT, true, LO>(a, codes, meta, act16, u0, u1, ridx + s * M, coef + s * M, pp, (size_t)prow * nu * 4, lane);
                    else
                        w2_unit<MB, NT, false, LO>(a, codes, meta, act16, u0, u1, ridx + s * M, coef + s * M, pp, (size_t)prow * nu * 4, lane);
                }
                first = (first + n * L.sp) % kWarps;
                if (RING) {  // ten arrivals a stage: one for two warps
                    named_bar_sync(2 + warp / 2, 64);
                    if (lane == 0 && (warp & 1) == 0) mbar_arrive(empty(it % L.stages));
                }
            }
        named_bar_sync(1, kThreads);
        for (int i = threadIdx.x; i < 16 * M * nt; i += kThreads) {
            const int r = i & 15, m = (i >> 4) % M, q = (i >> 4) / M;
            float v = 0.0f;
            for (int c = 0; c < nsel; ++c)
                for (int ip = 0; ip < L.sp; ++ip) v += part[((q * L.sp + ip) * prow + m * nsel + c) * 16 + r];
            store_any(a.out, a.odt, (size_t)m * K + 16 * (blockIdx.x + (tl + q) * gridDim.x) + r, v);
        }
        named_bar_sync(1, kThreads);
    }
}

// ---------------------------------------------------------------------------
// More tokens: router and selection for the grouped kernels
// ---------------------------------------------------------------------------
// Eight tokens and eight tiles of rows a CTA, a warp a tile.
__global__ void __launch_bounds__(256) router_kernel(const MoeLayerArgs a) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int s_max[16], s_sig[16];
    uint4* xsm = reinterpret_cast<uint4*>(sm);
    const int m0 = blockIdx.x * 8, M = min(8, a.M - m0), rows = a.E + (a.sgate ? a.S : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    stage_x(a, static_cast<const uint16_t*>(a.x) + (size_t)m0 * a.K, M, xsm, s_max, s_sig, 256, [] { __syncthreads(); });
    const int tile = blockIdx.y * 8 + warp;
    if (tile * 16 >= rows) return;
    float d[1][4];
    router_tile<1, true>(a, xsm, M, tile, 0, a.K / 32, 1, lane, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = tile * 16 + g + 4 * (e & 2), m = 2 * t + (e & 1);
        const size_t at = (size_t)(m0 + m) * (a.E + a.S) + row;
        if (row < rows && m < M && QMLP_INB(at, a.logit_elems, 108)) a.logits[at] = scalbnf(d[0][e], -s_sig[m] - a.rexp[row]);
    }
}
// A warp a token.
__global__ void __launch_bounds__(128) select_kernel(const MoeLayerArgs a) {
    __shared__ int se[4][16];
    __shared__ float sw[4][16];
    __shared__ Pick picks[4];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, m0 = blockIdx.x * 4, m = m0 + w, nsel = a.topk + a.S;
    select_tokens(a, a.logits + (size_t)m0 * (a.E + a.S), min(4, a.M - m0), 1, picks, &se[0][0], &sw[0][0], [] { __syncwarp(); });
    if (m >= a.M) return;
    __syncwarp();
    if (lane < nsel) {
        a.ids[(size_t)m * nsel + lane] = se[w][lane];
        a.weights[(size_t)m * nsel + lane] = sw[w][lane];
        a.amax[(size_t)m * nsel + lane] = 0;  // (W13's kernel takes maxima into it)
    }
    if (lane < a.topk) {
        if (a.ids_out) a.ids_out[(size_t)m * a.topk + lane] = se[w][lane];
        if (a.w_out) a.w_out[(size_t)m * a.topk + lane] = sw[w][lane];
    }
}

// The router (and shared gates) [rows, K] of a type -> fragments, and the rows'
// exponents. A warp a row for the exponent, then a thread a 16-byte piece.
__global__ void __launch_bounds__(256) router_exp_kernel(const void* w, const void* sg, int type, int E, int rows, int K, int* rexp,
                                                         int padded) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= padded) return;
    float mx = 0.0f;
    if (row < rows)
        for (int c = lane; c < K / 8; c += 32) {
            float v[8];
            load8t(row < E ? w : sg, type, (size_t)(row < E ? row : row - E) * K + 8 * c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) rexp[row] = prescale_exponent(mx);
}
__global__ void __launch_bounds__(256) router_frag_kernel(const void* w, const void* sg, int type, int E, int rows, int K,
                                                          const int* rexp, int tiles, int planes, uint4* out) {
    const size_t n32 = K / 32, items = (size_t)planes * tiles * n32 * 64;
    for (size_t it = (size_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (size_t)gridDim.x * 256) {
        const int lane = (int)(it & 31), st = (int)(it >> 5) & 1, g = lane >> 2, t = lane & 3;
        const size_t rest = it >> 6;
        const int j = (int)(rest % n32), tile = (int)(rest / n32 % tiles), pl = (int)(rest / n32 / tiles);
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // rows g, g + 8 of pair 2 st, then of 2 st + 1 (unit_order)
            const int row = tile * 16 + g + 8 * (q & 1), k = 32 * j + 8 * st + 2 * t + (q >> 1);
            float v[2] = {0.0f, 0.0f};
            if (row < rows) {
                const void* p = row < E ? w : sg;
                const size_t at = (size_t)(row < E ? row : row - E) * K + k;
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // k and k + 16
                    const float f = type == 0   ? static_cast<const float*>(p)[at + 16 * e]
                                    : type == 1 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at + 16 * e])
                                                : __half2float(static_cast<const __half*>(p)[at + 16 * e]);
                    v[e] = scalbnf(f, rexp[row]);
                    if (pl) v[e] -= __half2float(__float2half_rn(v[e]));  // what the first plane leaves
                }
            }
            o[q] = u32(__floats2half2_rn(v[0], v[1]));
        }
        out[it] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int MB, int NT, bool RING, bool LO>
cudaError_t launch_few(const MoeLayerArgs& a, int bytes, int num_sms, cudaStream_t s) {
    static unsigned long done = 0;
    if (const cudaError_t e = smem_once(moe_layer_kernel<MB, NT, RING, LO>, kSmemMax, done); e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms);
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once, or the launch waits
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_layer_kernel<MB, NT, RING, LO>, a);
}

Layout layout_of(int M, int K, int I, int E, int S, int topk, int MB, bool lo) {
    return layout(M, K, I, E, topk + S, std::min(E, M * topk) + S, MB, M <= 8 ? 1 : 2, lo);
}
template <int MB, bool LO>
cudaError_t launch_few_of(const MoeLayerArgs& a, const Layout& l, int num_sms, cudaStream_t s) {
    if (l.bytes > kSmemMax) return cudaErrorInvalidValue;
    if (l.stage)
        return a.M <= 8 ? launch_few<MB, 1, true, LO>(a, l.bytes, num_sms, s) : launch_few<MB, 2, true, LO>(a, l.bytes, num_sms, s);
    return a.M <= 8 ? launch_few<MB, 1, false, LO>(a, l.bytes, num_sms, s) : launch_few<MB, 2, false, LO>(a, l.bytes, num_sms, s);
}

}  // namespace

// The one kernel wherever it fits: it is ahead at every number of tokens that it takes. One
// kernel / router, selection and grouped kernels, 2, 8 and 16 tokens, us: 512 experts of
// 2560 x 160, top 10 and a shared one 31, 55, 88 / 51, 82, 114; 128 of 2048 x 768, top 8
// 37, 75, 125 / 96, 166, 176; 64 of 2048 x 704, top 6 and two shared 35, 55, 80 / 86, 138, 152.
bool moe_layer_few(int M, int K, int I, int E, int S, int topk, int meta_bytes) {
    return M <= kMoeLayerFew && layout_of(M, K, I, E, S, topk, meta_bytes, false).bytes <= kSmemMax &&
           layout_of(M, K, I, E, S, topk, meta_bytes, true).bytes <= kSmemMax;
}

cudaError_t launch_moe_layer_few(MoeLayerArgs a, int meta_bytes, int num_sms, cudaStream_t s) {
    a.slots = std::min(a.E, a.M * a.topk) + a.S;
    a.limit = kWaitNs;
    const bool lo = a.odt == 0;
    const Layout l = layout_of(a.M, a.K, a.I, a.E, a.S, a.topk, meta_bytes, lo);
    if (meta_bytes == 4) return lo ? launch_few_of<4, true>(a, l, num_sms, s) : launch_few_of<4, false>(a, l, num_sms, s);
    return lo ? launch_few_of<3, true>(a, l, num_sms, s) : launch_few_of<3, false>(a, l, num_sms, s);
}

cudaError_t launch_moe_router(const MoeLayerArgs& a, cudaStream_t s) {
    const int tiles = (a.E + (a.sgate ? a.S : 0) + 15) / 16;
    const size_t smem = (size_t)std::min(8, a.M) * a.K * 2;
    static unsigned long done = 0;
    if (const cudaError_t e = smem_once(router_kernel, kSmemMax, done); e != cudaSuccess) return e;
    if (smem > kSmemMax) return cudaErrorInvalidValue;
    // (tokens along x: a grid's second dimension ends at 65535)
    router_kernel<<<dim3((unsigned)((a.M + 7) / 8), (unsigned)((tiles + 7) / 8)), 256, smem, s>>>(a);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    select_kernel<<<(unsigned)((a.M + 3) / 4), 128, 0, s>>>(a);
    return cudaPeekAtLastError();
}

cudaError_t launch_router_layout(const MoeLayerArgs& a, const void* w, const void* sg, int type, uint4* frag, int* rexp,
                                 cudaStream_t s) {
    const int rows = a.E + (sg ? a.S : 0), padded = a.rtiles * 16;
    router_exp_kernel<<<(unsigned)((padded + 7) / 8), 256, 0, s>>>(w, sg, type, a.E, rows, a.K, rexp, padded);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return e;
    router_frag_kernel<<<(unsigned)std::min<size_t>((a.rfrag_elems + 255) / 256, 65535), 256, 0, s>>>(
        w, sg, type, a.E, rows, a.K, rexp, a.rtiles, a.planes, frag);
    return cudaPeekAtLastError();
}

QMLP_BOUNDS_UNIT(moe_layer)

}  // namespace qmlp
