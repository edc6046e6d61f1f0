// linear.cu -- one projection with 4-bit weights and group scales:
//   y[m, n] = c sum_k x[m, k] W[n, k] + bias[n]
//   NVFP4: W = E2M1(code) E4M3(scale[n, k / 16]), c = 1 / global
//   INT4:  W = (code - zero[n, k / G]) scale[n, k / G], G = 32, 64 or 128, c = 1
// for a few tokens (here) or many (images for the tensor-core GEMM, below).
//
// Few tokens (at most 64): the weights are read once.
//  * Weights are laid out once, in records of 16 rows x 128 k (kRec bytes: codes
//    in the order in which the lanes of an mma.sync m16n8k16 take them as the A
//    operand, then the groups' scales). k is summed in any order that both
//    operands share, so a lane's share of a step is four neighbours, and the 16
//    bytes that it loads for a row are all its eight steps.
//  * The tokens are the columns of the B operand (eight a tile), kept in shared
//    memory in the order of the steps. x is fp16 there: fp16 as it is, bf16 times
//    a power of two a token that takes the row's largest value to [2^14, 2^15),
//    exact for every value within 2^29 of it.
//  * NVFP4: E2M1 x E4M3 has six significant bits, exact in fp16: the weights are
//    multiplied out and all of k summed by the MMAs. INT4: code - zero is an
//    integer, exact in fp16; a group's sum is taken by itself and multiplied by
//    its scale in fp32, so no weight is ever rounded.
//  * A producer warp keeps a ring of records in shared memory full with bulk copies
//    (loads into registers, two records a warp, ran at one record's latency after
//    the other: 4.2 TB/s at 128000 x 5120). Its CTA's warps each take a record of the
//    ring at a time: a tile of 16 rows to several warps that share its k and whose
//    sums are added in their order, or a warp a tile.
//  * A cluster of up to eight CTAs splits k where x would not fit in shared memory or
//    the rows are too few for the GPU; its CTAs add their sums through distributed
//    shared memory, in their order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kCh = kLinearChunk;   // k of a record
constexpr int kPitch = 20;          // rows of a column of the warps' sums, padded
constexpr int kSmemMax = 226 * 1024;
constexpr int kMaxStages = 16;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s

// Kinds of weights: NVFP4 (group 16) or INT4 with its group.
template <int G>
struct Rec {
    static constexpr bool kNv = G == 16;
    static constexpr int kPer = kCh / G;  // groups a row and record
    static constexpr int kScales = kNv ? 16 * kPer : 16 * kPer * 2;
    static constexpr int kZeros = kNv ? 0 : 16 * kPer;
    static constexpr int kBytes = 16 * kCh / 2 + kScales + kZeros;
    static_assert(kBytes % 16 == 0 && kBytes == linear_rec_bytes(G), "records of whole 16 bytes");
};

// A lane's part of a record: codes of rows g and g + 8, and their scales and zeros,
// which lie together for the two rows: [8 g][2 rows][kPer].
template <int G>
struct Frag {
    uint4 c[2];
    uint32_t s[2][G >= 64 ? 1 : 2];  // NVFP4: 8 E4M3; INT4: the groups' fp16 scales (G = 128: both rows in s[0])
    uint32_t z[2];                   // INT4: the groups' zeros, a byte each (G >= 64: both rows in z[0])
};
QMLP_DEV uint4 lds4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
QMLP_DEV uint2 lds2(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
QMLP_DEV uint32_t lds1(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
QMLP_DEV uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
// at: the lane's codes of row g; sc: its g's scales, ze: zeros (shared memory).
template <int G>
QMLP_DEV void load_frag(Frag<G>& f, uint32_t at, uint32_t sc, uint32_t ze) {
    f.c[0] = lds4(at);
    f.c[1] = lds4(at + 512);
    if constexpr (G <= 32) {
        const uint4 v = lds4(sc);
        f.s[0][0] = v.x, f.s[0][1] = v.y, f.s[1][0] = v.z, f.s[1][1] = v.w;
        if constexpr (G == 32) {
            const uint2 z = lds2(ze);
            f.z[0] = z.x, f.z[1] = z.y;
        }
    } else if constexpr (G == 64) {
        const uint2 v = lds2(sc);
        f.s[0][0] = v.x, f.s[1][0] = v.y;
        f.z[0] = lds1(ze);
    } else {
        f.s[0][0] = lds1(sc);
        f.z[0] = lds16(ze);
    }
}
// fp16 scale of row half h and group q, in place 0 or 1 of its word.
template <int G>
QMLP_DEV __half scale_of(const Frag<G>& f, int h, int q) {
    const uint32_t w = G == 128 ? f.s[0][0] : f.s[h][q >> 1];
    const __half2 p = *reinterpret_cast<const __half2*>(&w);
    return (G == 128 ? h : q & 1) ? __high2half(p) : __low2half(p);
}

QMLP_DEV uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
QMLP_DEV __half2 h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
QMLP_DEV uint32_t u2(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
// Byte i of z as {-(1024 + z)} twice: 0xE400 is -1024, whose last place is one.
QMLP_DEV uint32_t zero2(uint32_t z, int i) { return __byte_perm(z, 0xE4E4E4E4u, 0x4040u | (uint32_t)(i | i << 8)); }
template <int G>
QMLP_DEV uint32_t zero_of(const Frag<G>& f, int h, int q) {
    return G == 32 ? zero2(f.z[h], q) : zero2(f.z[0], G == 64 ? 2 * h + q : h);
}
// (w & mask) | magic in one instruction (the compiler took two)
QMLP_DEV uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}
// Eight codes (two steps of a row) less their zero: nibbles p and p + 4 of the word
// are pair p; 0x6400 | q is 1024 + q, 0x6400 | 16 q is 1024 + 16 q; both steps exact.
// z1 = -(1024 + z), z16 = -(64 + z).
QMLP_DEV void int4x8(uint32_t w, __half2 z1, __half2 z16, uint32_t (&p)[4]) {
    const uint32_t v = w >> 8;
    const __half2 six = h2(0x2C002C00u);  // 1/16
    p[0] = u2(__hadd2(h2(and_or(w, 0x000F000Fu, 0x64006400u)), z1));
    p[1] = u2(__hfma2(h2(and_or(w, 0x00F000F0u, 0x64006400u)), six, z16));
    p[2] = u2(__hadd2(h2(and_or(v, 0x000F000Fu, 0x64006400u)), z1));
    p[3] = u2(__hfma2(h2(and_or(v, 0x00F000F0u, 0x64006400u)), six, z16));
}
// Eight E2M1 codes (two steps of a row) times the E4M3 scales of their two groups
// (sp, as fp16): pair p is byte p of the word.
QMLP_DEV void e2m1x8(uint32_t w, __half2 sp, uint32_t (&p)[4]) {
    e2m1x4_to_f16x2x4(w, p[0], p[1], p[2], p[3]);
    const __half2 lo = __low2half2(sp), hi = __high2half2(sp);
    p[0] = u2(__hmul2(h2(p[0]), lo));
    p[1] = u2(__hmul2(h2(p[1]), lo));
    p[2] = u2(__hmul2(h2(p[2]), hi));
    p[3] = u2(__hmul2(h2(p[3]), hi));
}

// One record times one tile of eight tokens. xb: this lane's x of the record in shared
// memory, 16 bytes a pair of steps, `xs` apart. The steps go to two accumulators in
// turn: a warp's MMAs would otherwise wait for one another. NVFP4's are all of the warp's
// k, or (SUM, for an fp32 out) a record's, added in fp32: an MMA cuts off what passes its last
// bit, and chains over k = 17408 were 6e-7 off (8 tokens of 17408 x 5120 take 17.4 us with
// it, 16.7 without; one of 128000 x 5120 72 and 73).
template <int G, bool ONE, bool SUM>
QMLP_DEV void mma_record(const Frag<G>& f, uint32_t xb, uint32_t xs, float (&acc)[2][4]) {
    using R = Rec<G>;
    if constexpr (R::kNv) {
        float sum[SUM ? 2 : 1][4];
        float (&d0)[4] = SUM ? sum[0] : acc[0];
        float (&d1)[4] = SUM ? sum[SUM ? 1 : 0] : acc[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // two steps: groups 2i and 2i + 1 of both rows
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t s01, s23;
                e4m3x4_to_f16x2x2(f.s[h][i >> 1], s01, s23);
                e2m1x8(word_of(f.c[h], i), h2((i & 1) ? s23 : s01), a[h]);
            }
            const uint4 x = lds4(xb + i * xs);
            if (SUM && i == 0) {
                mma_f16_16816_zc(d0, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                mma_f16_16816_zc(d1, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
            } else {
                mma_f16_16816(d0, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                mma_f16_16816(d1, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
            }
        }
        if constexpr (SUM)
#pragma unroll
            for (int e = 0; e < 4; e += ONE ? 2 : 1) acc[0][e] += sum[0][e] + sum[1][e];
    } else {
#pragma unroll
        for (int q = 0; q < R::kPer; ++q) {
            __half2 z1[2], z16[2];
            float s[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                z1[h] = h2(zero_of<G>(f, h, q));
                z16[h] = __hadd2(z1[h], h2(0x63806380u));  // -(1024 + z) + 960
                s[h] = __half2float(scale_of<G>(f, h, q));
            }
            float d[2][4];
#pragma unroll
            for (int i = q * (4 / R::kPer); i < (q + 1) * (4 / R::kPer); ++i) {
                uint32_t a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) int4x8(word_of(f.c[h], i), z1[h], z16[h], a[h]);
                const uint4 x = lds4(xb + i * xs);
                if (i == q * (4 / R::kPer)) {
                    mma_f16_16816_zc(d[0], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                    mma_f16_16816_zc(d[1], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                } else {
                    mma_f16_16816(d[0], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                    mma_f16_16816(d[1], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; e += ONE ? 2 : 1) acc[0][e] = fmaf(s[e >> 1], d[0][e] + d[1][e], acc[0][e]);
        }
    }
}
// One record times NT tiles; INT4's sums of 32 k are scaled one by one, which keeps
// few of them in registers. NVFP4's are all of k's, or (SUM, for an fp32 out) a record's:
// an MMA cuts off what passes its last bit, and chains over k = 17408 were 1.3e-6 off (64
// tokens of 17408 x 5120 take 54 us with it, 40 without). xn: this lane's place in the record's x (xb) by tile.
template <int G, int NT, bool SUM>
QMLP_DEV void mma_record_tiles(const Frag<G>& f, uint32_t xb, uint32_t xs, const uint32_t (&xn)[NT], float (&acc)[NT][4]) {
    using R = Rec<G>;
    __half2 z1[2], z16[2];
    float s[2], sum[SUM ? NT : 1][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[2][4];
        if constexpr (R::kNv) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t s01, s23;
                e4m3x4_to_f16x2x2(f.s[h][i >> 1], s01, s23);
                e2m1x8(word_of(f.c[h], i), h2((i & 1) ? s23 : s01), a[h]);
            }
        } else {
            if (i % (4 / R::kPer) == 0)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = i / (4 / R::kPer);
                    z1[h] = h2(zero_of<G>(f, h, q));
                    z16[h] = __hadd2(z1[h], h2(0x63806380u));
                    s[h] = __half2float(scale_of<G>(f, h, q));
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) int4x8(word_of(f.c[h], i), z1[h], z16[h], a[h]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 x = lds4(xb + xn[n] + i * xs);
            if constexpr (R::kNv) {
                float (&d)[4] = SUM ? sum[n] : acc[n];
                if (SUM && i == 0) mma_f16_16816_zc(d, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                else mma_f16_16816(d, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                mma_f16_16816(d, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                if (SUM && i == 3)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][e] += sum[n][e];
            } else {
                float d[4];
                mma_f16_16816_zc(d, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                mma_f16_16816(d, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] = fmaf(s[e >> 1], d[e], acc[n][e]);
            }
        }
    }
}

QMLP_DEV void lin_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QMLP_DEV void peer_arrive(uint32_t bar, uint32_t rank) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(bar), "r"(rank));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(ra) : "memory");
}
// Bounded wait for a phase of a barrier that CTAs of the cluster arrive on.
QMLP_DEV bool wait_peers(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    auto once = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (once()) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!once())
        if (globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}
QMLP_DEV float4 peer_f4(const float* p, int rank) {
    uint32_t ra;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(ra));
    return v;
}
QMLP_DEV void add4(float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
// The sum over the S CTAs of a cluster of what they have at p, in their order.
QMLP_DEV float4 peer_sum(const float* p, int S) {
    float4 q[8], v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < S) q[r] = peer_f4(p, r);
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < S) add4(v, q[r]);
    return v;
}

QMLP_DEV int peer_s32(const int* p, int rank) {
    uint32_t ra;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

// Outputs n..n + 3 of token m from their sums, which are times 2^sig.
QMLP_DEV void store4(const LinearArgs& a, int m, int n, const float4& s, int sig) {
    const float p0 = __int_as_float((127 - (sig >> 1)) << 23), p1 = __int_as_float((127 - sig + (sig >> 1)) << 23);
    float v[4] = {s.x, s.y, s.z, s.w};
    const size_t at = (size_t)m * a.N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = v[e] * p0 * a.factor * p1;  // (a sum past fp32's range that the factor brings back)
        if (a.bias && n + e < a.N) v[e] += __ldg(a.bias + n + e);
    }
    if (n + 3 < a.N && (a.N & 3) == 0) {
        if (!QMLP_INB(at + 3, (size_t)a.M * a.N, 92)) return;
        if (a.odt == 0) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else if (a.odt == 1) {
            __nv_bfloat162 p[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = *reinterpret_cast<const uint2*>(p);
        } else {
            __half2 p[2] = {__floats2half2_rn(v[0], v[1]), __floats2half2_rn(v[2], v[3])};
            *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = *reinterpret_cast<const uint2*>(p);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (n + e >= a.N || !QMLP_INB(at + e, (size_t)a.M * a.N, 92)) continue;
        if (a.odt == 0) static_cast<float*>(a.out)[at + e] = v[e];
        else if (a.odt == 1) static_cast<__nv_bfloat16*>(a.out)[at + e] = __float2bfloat16_rn(v[e]);
        else static_cast<__half*>(a.out)[at + e] = __float2half_rn(v[e]);
    }
}

// The meeting of the consumers of a cluster's CTAs: what they wrote to their shared
// memory is visible to all of them behind it (the producers have no part in it: they
// wait for the consumers, who would wait for them). Bounded.
struct Peers {
    uint32_t bar;
    int S, threads, count;
    int* err;
    bool ok;
    QMLP_DEV void meet() {
        named_bar_sync(1, threads);
        if ((int)threadIdx.x < S) peer_arrive(bar, threadIdx.x);
        if (ok && !wait_peers(bar, (uint32_t)(count & 1), kWaitNs)) {
            atomicExch(err, 93);
            ok = false;
        }
        ++count;
        named_bar_sync(1, threads);
    }
};

// A consumer's place in the ring of stages.
struct Place {
    uint32_t slot, first, end, stage, fb, fb0, parity;
    bool late;
    QMLP_DEV void wait(int* err) {
        if (mbar_try_wait(fb, parity)) return;
        if (!mbar_wait_bounded(fb, parity, late ? 0 : kWaitNs)) {
            atomicExch(err, 92);  // (what is then read lies in the ring; out is not valid)
            late = true;
        }
    }
    QMLP_DEV void release_and_step(int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(fb + 8u * kMaxStages);
        slot += stage;
        fb += 8;
        if (slot == end) {
            slot = first;
            fb = fb0;
            parity ^= 1;
        }
    }
};

// How a launch is cut.
struct FewPlan {
    int S;       // CTAs of a cluster: splits of k
    int wpt;     // few: warps that share a tile of 16 rows (its k), W / wpt tiles a group
    int tg;      // mid: tiles of a group
    int gy;      // clusters
    int stages;  // of the ring
    int batch;   // few: groups whose sums wait in shared memory (S > 1)
};
// Warps and CTAs an SM, one token and two to eight (5120 x 5120 / 17408 x 5120 / 128000 x
// 5120 NVFP4: one token 6.9 / 15.4 / 76 us, with 16 warps in one CTA 7.6 / 14.1 / 84; eight
// tokens 10.9 / 17.3 / 86, with 8 warps in two CTAs 12.1 / 22.6 / 111).
template <bool ONE>
constexpr int few_warps() { return ONE ? 8 : 16; }
template <bool ONE>
constexpr int few_ctas() { return ONE ? 3 : 1; }

// At most eight tokens. Grid (S, gy), clusters of S. A producer warp copies the
// groups' records into a ring in shared memory (bulk copies: the weights do not
// depend on anything before this launch, so they start at once), W warps consume
// them. Shared memory: x, the ring, the warps' sums (two buffers: one barrier a group
// is enough), this CTA's sums of a batch of groups where k is split.
template <int G, bool ONE, bool SUM>
__global__ void __launch_bounds__((few_warps<ONE>() + 1) * 32, few_ctas<ONE>())
    linear_few_kernel(const LinearArgs a, const FewPlan P) {
    using R = Rec<G>;
    constexpr int kC = ONE ? 1 : 8, W = few_warps<ONE>(), kT = W * 32, kRec = R::kBytes, kStage = W * kRec;
    extern __shared__ __align__(128) uint8_t few_sm[];
    __shared__ int s_max[8], s_sig[8];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 1];
    const int S = P.S, rank = blockIdx.x, M = ONE ? 1 : a.M, K = a.K;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int Kc = (K + kCh - 1) / kCh, Nt = (a.N + 15) / 16;
    const int cps = (Kc + S - 1) / S;                     // records of k a CTA
    const int kc0 = rank * cps, nch = min(cps, Kc - kc0);  // this one's
    const int wpt = P.wpt, TG = W / wpt, groups = (Nt + TG - 1) / TG, steps = (cps + wpt - 1) / wpt;
    uint4* xsm = reinterpret_cast<uint4*>(few_sm);
    uint8_t* ring = few_sm + (size_t)cps * 256 * M;
    float* red = reinterpret_cast<float*>(ring + (size_t)P.stages * kStage);  // [2][W][kC][kPitch], wpt > 1
    float* own = red + (wpt > 1 ? 2 * W * kC * kPitch : 0);                    // [batch][TG][kC][16], S > 1
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    const uint32_t peers = bar0 + 8u * (2 * kMaxStages);
    if (threadIdx.x == 0) {
        for (int s = 0; s < P.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), W);
        }
        mbar_init(peers, (uint32_t)S);
        fence_mbar_init();
    }
    if (threadIdx.x < 8) s_max[threadIdx.x] = s_sig[threadIdx.x] = 0;
    if (S > 1) lin_cluster_sync();  // the peers' barriers are there
    else __syncthreads();
    pdl_launch_dependents();

    if (warp == W) {
        // ---------------- producer: a lane a tile ----------------
        int it = 0;
        bool ok = true;
        for (int gr = blockIdx.y; gr < groups && ok; gr += gridDim.y) {
            const int tiles = min(TG, Nt - gr * TG);
            const uint8_t* src = a.w + (((size_t)gr * TG + lane) * Kc + kc0) * kRec;
            for (int st = 0; st < steps; ++st, ++it) {
                const int s = it % P.stages;
                if (it >= P.stages &&
                    !__all_sync(0xffffffffu, mbar_wait_bounded(empty(s), (uint32_t)((it / P.stages - 1) & 1), kWaitNs))) {
                    if (lane == 0) atomicExch(a.err, 91);
                    ok = false;
                    break;
                }
                const int n = max(0, min(wpt, nch - st * wpt));
                const uint32_t bytes = (uint32_t)(n * kRec);
                if (lane == 0) mbar_arrive_expect_tx(full(s), bytes * tiles);
                __syncwarp();
                if (n > 0 && lane < tiles) {
                    const uint8_t* p = src + (size_t)st * wpt * kRec;
                    if (!QMLP_INB(p - a.w + bytes - 1, a.w_bytes, 91)) p = a.w;
                    bulk_g2s(smem_u32(ring + (size_t)s * kStage + (size_t)lane * wpt * kRec), p, bytes, full(s));
                }
            }
        }
        // copies still in flight (only after a wait that ran out): wait for each
        // stage's last one
        if (!ok)
            for (int q = it - 1; q >= 0 && q >= it - P.stages; --q)
                mbar_wait_bounded(full(q % P.stages), (uint32_t)((q / P.stages) & 1), kWaitNs);
        __syncwarp();
        if (S > 1) lin_cluster_sync();  // see the end
        return;
    }

    // ---------------- x ----------------
    // of this CTA's k, in the order of the steps: slot ((c 4 + i) M + m) 4 + t has
    // k = 128 c + 32 i + 4 t.. (four) and 16 further (four) of token m. A thread
    // stays with one token: its largest value falls out of the copy, and the copy is
    // scaled in place once the row's exponent is known.
    pdl_wait();  // x is written, and out may be
    Peers cluster{peers, S, kT, 0, a.err, true};
    const int xt = threadIdx.x & 3, xm = ONE ? 0 : (threadIdx.x >> 2) & 7, hop = ONE ? kT / 4 : kT / 32;
    const int ci0 = ONE ? threadIdx.x >> 2 : threadIdx.x >> 5;
    if (xm < M) {
        float mx = 0.0f;
        const uint16_t* row = static_cast<const uint16_t*>(a.x) + (size_t)xm * K;
#pragma unroll 4
        for (int ci = ci0; ci < nch * 4; ci += hop) {
            const int k = kc0 * kCh + 32 * ci + 4 * xt;
            uint2 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)  // K is a multiple of 16
                v[h] = k + 16 * h < K ? *reinterpret_cast<const uint2*>(row + k + 16 * h) : make_uint2(0, 0);
            if (a.x_bf16)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(v[h].x << 16)), fabsf(__uint_as_float(v[h].x & 0xFFFF0000u))),
                                         fmaxf(fabsf(__uint_as_float(v[h].y << 16)), fabsf(__uint_as_float(v[h].y & 0xFFFF0000u)))));
            xsm[(ci * M + xm) * 4 + xt] = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
        }
        if (a.x_bf16) {  // lanes of the same token first
            const uint32_t on = __activemask();
#pragma unroll
            for (int o = 1; o < (ONE ? 32 : 4); o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(on, mx, o));
            if (ONE ? lane == 0 : xt == 0) atomicMax(s_max + xm, __float_as_int(mx));
        }
    }
    if (a.x_bf16) {
        if (S > 1) cluster.meet();
        else named_bar_sync(1, kT);
        if (threadIdx.x < M) {
            int mx = 0;
            for (int r = 0; r < S; ++r) mx = max(mx, S > 1 ? peer_s32(s_max + threadIdx.x, r) : s_max[threadIdx.x]);
            s_sig[threadIdx.x] = prescale_exponent(__int_as_float(mx));
        }
        named_bar_sync(1, kT);
        if (xm < M) {
            // 2^sig in two factors: it may pass fp32's range, they do not
            const int sg = s_sig[xm];
            const float p0 = __int_as_float((127 + (sg >> 1)) << 23), p1 = __int_as_float((127 + sg - (sg >> 1)) << 23);
            for (int ci = ci0; ci < nch * 4; ci += hop) {
                uint4& slot = xsm[(ci * M + xm) * 4 + xt];
                const uint4 u = slot;
                uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = u2(__floats2half2_rn(__uint_as_float(v[j] << 16) * p0 * p1,
                                                __uint_as_float(v[j] & 0xFFFF0000u) * p0 * p1));
                slot = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }
    named_bar_sync(1, kT);

    // ---------------- consumers ----------------
    const int wi = warp % wpt, wt = warp / wpt;  // place in the tile's k, tile of the group
    const uint32_t x0 = smem_u32(xsm) + (uint32_t)(wi * 256 * M + (min(g, M - 1) * 4 + t) * 16);
    const uint32_t xstep = (uint32_t)(wpt * 256 * M), xs = (uint32_t)(64 * M);
    const uint32_t at0 = smem_u32(ring) + (uint32_t)(warp * kRec);
    Place at{at0, at0, at0 + (uint32_t)(P.stages * kStage), (uint32_t)kStage, full(0), full(0), 0, false};
    const int nst = nch > wi ? (nch - wi + wpt - 1) / wpt : 0;  // steps that this warp has a record in
    int done = 0, b0 = blockIdx.y;  // groups done, the batch's first
    for (int gr = blockIdx.y; gr < groups; gr += gridDim.y, ++done) {
        float acc[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][e] = acc[1][e] = 0.0f;
        const int mst = gr * TG + wt < Nt ? nst : 0;
        uint32_t xb = x0;
#pragma unroll 1
        for (int st = 0; st < steps; ++st, xb += xstep) {
            at.wait(a.err);
            Frag<G> f;
            const bool has = st < mst;
            if (has)
                load_frag<G>(f, at.slot + lane * 16, at.slot + 1024 + g * (R::kScales / 8),
                             at.slot + 1024 + R::kScales + g * (R::kZeros / 8));
            at.release_and_step(lane);
            if (has) mma_record<G, ONE, SUM>(f, xb, xs, acc);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][e] += acc[1][e];
        float* ob = own + (size_t)(done % P.batch) * TG * kC * 16;
        if (wpt > 1) {
            float* rb = red + (done & 1) * W * kC * kPitch;
            // [warp][column][kPitch rows]: 20 puts the 32 lanes on 32 banks
            float* mine = rb + warp * kC * kPitch;
            if (!ONE || t == 0)
#pragma unroll
                for (int e = 0; e < 4; e += ONE ? 2 : 1) mine[(ONE ? 0 : 2 * t + (e & 1)) * kPitch + g + 4 * (e & 2)] = acc[0][e];
            named_bar_sync(1, kT);
            for (int i = threadIdx.x; i < 4 * M * TG; i += kT) {  // four rows of a token
                const int r4 = (i & 3) * 4, m = (i >> 2) % M, j = (i >> 2) / M;
                float4 v = make_float4(0, 0, 0, 0);
                for (int w = 0; w < wpt; ++w)
                    add4(v, *reinterpret_cast<const float4*>(rb + ((j * wpt + w) * kC + m) * kPitch + r4));
                if (S > 1) *reinterpret_cast<float4*>(ob + (j * kC + m) * 16 + r4) = v;
                else store4(a, m, 16 * (gr * TG + j) + r4, v, s_sig[m]);
            }
        } else {
            // the warp's own tile: through its place in `own`, four rows of a token at a time
            float* mine = ob + warp * kC * 16;
            __syncwarp();
            if (!ONE || t == 0)
#pragma unroll
                for (int e = 0; e < 4; e += ONE ? 2 : 1) mine[(ONE ? 0 : 2 * t + (e & 1)) * 16 + g + 4 * (e & 2)] = acc[0][e];
            __syncwarp();
            if (S == 1 && lane < 4 * M)
                store4(a, lane >> 2, 16 * (gr * TG + warp) + (lane & 3) * 4,
                       *reinterpret_cast<const float4*>(mine + (lane >> 2) * 16 + (lane & 3) * 4), s_sig[lane >> 2]);
        }
        // a batch of groups is done: the cluster's sums in order
        if (S > 1 && ((done + 1) % P.batch == 0 || gr + (int)gridDim.y >= groups)) {
            cluster.meet();  // every CTA's sums are written
            const int nb = done % P.batch + 1, items = nb * TG * 4 * M, per = (items + S - 1) / S;
            for (int i = rank * per + threadIdx.x; i < min(items, (rank + 1) * per); i += kT) {
                const int r4 = (i & 3) * 4, m = (i >> 2) % M, j = (i >> 2) / M;
                const float4 v = peer_sum(own + ((size_t)j * kC + m) * 16 + r4, S);
                store4(a, m, 16 * ((b0 + j / TG * (int)gridDim.y) * TG + j % TG) + r4, v, s_sig[m]);
            }
            cluster.meet();  // none writes its next sums while another reads
            b0 = gr + gridDim.y;
        }
    }
    if (S > 1) lin_cluster_sync();  // no CTA leaves while another may read its sums
}

// Nine to 64 tokens: x does not stay in shared memory but comes through the ring with
// the weights, in the order of the steps as linear_x_kernel wrote it. A warp takes a
// tile of 16 rows, up to 15 of them a group, and all of them the same k: a stage is CS
// records of each of the group's tiles and the x of their k.
template <int NT>
constexpr int mid_chunks() { return NT == 8 ? 1 : 2; }  // CS: 36 KB of weights a stage, 18 with 64 tokens
constexpr int kMidWarps = 15;  // with the producer four a scheduler: 128 registers each

template <int G, int NT, bool SUM>
__global__ void __launch_bounds__((kMidWarps + 1) * 32, 1) linear_mid_kernel(const LinearArgs a, const FewPlan P) {
    using R = Rec<G>;
    constexpr int kC = 8 * NT, W = kMidWarps, kT = W * 32, kRec = R::kBytes, CS = mid_chunks<NT>();
    extern __shared__ __align__(128) uint8_t few_sm[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 1];
    const int S = P.S, rank = blockIdx.x, M = a.M, K = a.K;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int Kc = (K + kCh - 1) / kCh, Nt = (a.N + 15) / 16, TG = P.tg, groups = (Nt + TG - 1) / TG;
    const int cps = (Kc + S - 1) / S, kc0 = rank * cps, nch = min(cps, Kc - kc0), steps = (cps + CS - 1) / CS;
    const int xbytes = 256 * M, stage = TG * CS * kRec + CS * xbytes;
    float* own = reinterpret_cast<float*>(few_sm + (size_t)P.stages * stage);  // [W][kC][16]
    const uint32_t bar0 = smem_u32(bars), ring = smem_u32(few_sm);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    const uint32_t peers = bar0 + 8u * (2 * kMaxStages);
    if (threadIdx.x == 0) {
        for (int s = 0; s < P.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), W);
        }
        mbar_init(peers, (uint32_t)S);
        fence_mbar_init();
    }
    if (S > 1) lin_cluster_sync();
    else __syncthreads();
    pdl_launch_dependents();

    if (warp == W) {
        // ---------------- producer: a lane a tile ----------------
        const uint8_t* xf = static_cast<const uint8_t*>(a.xf) + (size_t)kc0 * xbytes;
        const int all = (groups - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y * steps;
        // the first stages' weights, then, once x is there, their x
        auto weights = [&](int it) {
            const int s = it % P.stages, st = it % steps, gr = blockIdx.y + it / steps * gridDim.y;
            const int n = max(0, min(CS, nch - st * CS)), tiles = min(TG, Nt - gr * TG);
            if (lane == 0) mbar_arrive_expect_tx(full(s), (uint32_t)(n * (kRec * tiles + xbytes)));
            __syncwarp();
            if (n > 0 && lane < tiles) {
                const uint8_t* p = a.w + (((size_t)gr * TG + lane) * Kc + kc0 + st * CS) * kRec;
                if (!QMLP_INB(p - a.w + n * kRec - 1, a.w_bytes, 91)) p = a.w;
                bulk_g2s(ring + (uint32_t)(s * stage + lane * CS * kRec), p, (uint32_t)(n * kRec), full(s));
            }
        };
        auto tokens = [&](int it) {
            const int s = it % P.stages, st = it % steps, n = max(0, min(CS, nch - st * CS));
            if (n > 0 && lane == 0)
                bulk_g2s(ring + (uint32_t)(s * stage + TG * CS * kRec), xf + (size_t)st * CS * xbytes, (uint32_t)(n * xbytes),
                         full(s));
        };
        int it = 0;
        const int early = min(all, P.stages);
        for (; it < early; ++it) weights(it);
        pdl_wait();
        for (int q = 0; q < early; ++q) tokens(q);
        bool ok = true;
        for (; it < all; ++it) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(it % P.stages), (uint32_t)((it / P.stages - 1) & 1), kWaitNs))) {
                if (lane == 0) atomicExch(a.err, 91);
                ok = false;
                break;
            }
            weights(it);
            tokens(it);
        }
        if (!ok)
            for (int q = it - 1; q >= 0 && q >= it - P.stages; --q)
                mbar_wait_bounded(full(q % P.stages), (uint32_t)((q / P.stages) & 1), kWaitNs);
        __syncwarp();
        if (S > 1) lin_cluster_sync();
        return;
    }

    // ---------------- consumers ----------------
    pdl_wait();  // the exponents are written, and out may be
    Peers cluster{peers, S, kT, 0, a.err, true};
    uint32_t xn[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xn[n] = (uint32_t)((min(8 * n + g, M - 1) * 4 + t) * 16);
    const uint32_t xs = (uint32_t)(64 * M), xat = (uint32_t)(TG * CS * kRec - warp * CS * kRec);
    const uint32_t at0 = ring + (uint32_t)(warp * CS * kRec);
    Place at{at0, at0, at0 + (uint32_t)(P.stages * stage), (uint32_t)stage, full(0), full(0), 0, false};
    for (int gr = blockIdx.y; gr < groups; gr += gridDim.y) {
        const bool on = warp < TG && gr * TG + warp < Nt;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
            at.wait(a.err);
#pragma unroll
            for (int c = 0; c < CS; ++c)
                if (on && st * CS + c < nch) {
                    const uint32_t rec = at.slot + c * kRec;
                    Frag<G> f;
                    load_frag<G>(f, rec + lane * 16, rec + 1024 + g * (R::kScales / 8),
                                 rec + 1024 + R::kScales + g * (R::kZeros / 8));
                    mma_record_tiles<G, NT, SUM>(f, at.slot + xat + c * xbytes, xs, xn, acc);
                }
            at.release_and_step(lane);
        }
        // the tile's sums, [token][16 rows]
        float* mine = own + warp * kC * 16;
        __syncwarp();
        if (on)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[(8 * n + 2 * t + (e & 1)) * 16 + g + 4 * (e & 2)] = acc[n][e];
        __syncwarp();
        if (S == 1) {
            if (on)
                for (int i = lane; i < 4 * M; i += 32)
                    store4(a, i >> 2, 16 * (gr * TG + warp) + (i & 3) * 4,
                           *reinterpret_cast<const float4*>(mine + (i >> 2) * 16 + (i & 3) * 4), __ldcg(a.sig + (i >> 2)));
        } else {
            cluster.meet();  // every CTA's sums are written
            const int tiles = min(TG, Nt - gr * TG), items = tiles * 4 * M, per = (items + S - 1) / S;
            for (int i = rank * per + threadIdx.x; i < min(items, (rank + 1) * per); i += kT) {
                const int r4 = (i & 3) * 4, m = (i >> 2) % M, j = (i >> 2) / M;
                store4(a, m, 16 * (gr * TG + j) + r4, peer_sum(own + ((size_t)j * kC + m) * 16 + r4, S), __ldcg(a.sig + m));
            }
            cluster.meet();
        }
    }
    if (S > 1) lin_cluster_sync();
}

// x -> fp16 in the order of the steps, [record of k][pair of steps][token][t] of 16
// bytes (see linear_few_kernel), and the tokens' exponents. A CTA a token.
__global__ void __launch_bounds__(256) linear_x_kernel(const LinearArgs a) {
    __shared__ int s_max;
    const int m = blockIdx.x, M = a.M, K = a.K, n = (K + kCh - 1) / kCh * 16;  // 16-byte pieces of the token
    if (threadIdx.x == 0) s_max = 0;
    pdl_wait();
    pdl_launch_dependents();  // (only now: what comes next waits for this kernel alone)
    const uint16_t* row = static_cast<const uint16_t*>(a.x) + (size_t)m * K;
    uint4* out = static_cast<uint4*>(a.xf);
    auto piece = [&](int i) {  // i = 4 ci + t
        const int k = 32 * (i >> 2) + 4 * (i & 3);
        uint2 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) v[h] = k + 16 * h < K ? *reinterpret_cast<const uint2*>(row + k + 16 * h) : make_uint2(0, 0);
        return make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
    };
    constexpr int kKeep = 4;  // pieces a thread keeps between the two passes
    uint4 keep[kKeep];
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = threadIdx.x + j * 256;
        keep[j] = i < n ? piece(i) : make_uint4(0, 0, 0, 0);
    }
    auto largest = [&](const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
    };
    int sg = 0;
    __syncthreads();
    if (a.x_bf16) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j) largest(keep[j]);
#pragma unroll 4
        for (int i = threadIdx.x + kKeep * 256; i < n; i += 256) largest(piece(i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((threadIdx.x & 31) == 0) atomicMax(&s_max, __float_as_int(mx));
        __syncthreads();
        sg = prescale_exponent(__int_as_float(s_max));
    }
    if (threadIdx.x == 0) a.sig[m] = sg;
    const float p0 = __int_as_float((127 + (sg >> 1)) << 23), p1 = __int_as_float((127 + sg - (sg >> 1)) << 23);
    auto put = [&](int i, const uint4& u) {
        uint32_t v[4] = {u.x, u.y, u.z, u.w};
        if (a.x_bf16)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = u2(__floats2half2_rn(__uint_as_float(v[j] << 16) * p0 * p1, __uint_as_float(v[j] & 0xFFFF0000u) * p0 * p1));
        const size_t at = ((size_t)(i >> 2) * M + m) * 4 + (i & 3);
        if (QMLP_INB(at, a.xf_elems, 95)) out[at] = make_uint4(v[0], v[1], v[2], v[3]);
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
        if (threadIdx.x + j * 256 < n) put(threadIdx.x + j * 256, keep[j]);
#pragma unroll 4
    for (int i = threadIdx.x + kKeep * 256; i < n; i += 256) put(i, piece(i));
}

// Checkpoint rows -> records (one thread a lane's 16 bytes of a row half, the
// first also its row's scales).
template <int G>
__global__ void __launch_bounds__(256) repack_linear_kernel(const uint8_t* __restrict__ w,
                                                            const uint8_t* __restrict__ scale,
                                                            const uint8_t* __restrict__ zero, int N, int K, int Kc,
                                                            size_t items, uint8_t* __restrict__ out) {
    using R = Rec<G>;
    for (size_t it = (size_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (size_t)gridDim.x * 256) {
        const int lane = (int)(it & 31), h = (int)(it >> 5) & 1, g = lane >> 2, t = lane & 3;
        const size_t rec = it >> 6;
        const int kc = (int)(rec % Kc);
        const size_t row = rec / Kc * 16 + g + 8 * h;
        uint8_t* dst = out + rec * R::kBytes;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t b[4];  // the bytes of pairs 0..3 of steps 2i and 2i + 1
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int k = kc * kCh + 32 * i + 16 * (p >> 1) + 4 * t + 2 * (p & 1);
                b[p] = row < (size_t)N && k < K ? w[row * (K / 2) + k / 2] : 0u;
            }
            o[i] = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                o[i] |= R::kNv ? b[p] << (8 * p) : (b[p] & 15u) << (4 * p) | (b[p] >> 4) << (16 + 4 * p);
        }
        reinterpret_cast<uint4*>(dst + 512 * h)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
        if (t == 0) {
            const int groups = K / G;
            for (int q = 0; q < R::kPer; ++q) {
                const int gi = kc * R::kPer + q;
                const bool in = row < (size_t)N && gi < groups;
                const size_t at = row * groups + gi;
                const int to = (2 * g + h) * R::kPer + q;
                if (R::kNv) {
                    dst[1024 + to] = in ? scale[at] : 0;
                } else {
                    reinterpret_cast<uint16_t*>(dst + 1024)[to] =
                        in ? reinterpret_cast<const uint16_t*>(scale)[at] : (uint16_t)0;
                    dst[1024 + R::kScales + to] = in ? zero[at] : 0;
                }
            }
        }
    }
}

// Records -> stage images: a warp a record (16 rows x 128 k), each lane the four k
// of its two rows that it has of a step, 8 bytes of an image row at a time.
// An INT4 weight, 8 bits times 11, is rounded once to fp16 here: half a step, 2^-12 to 2^-11
// of itself. With a bf16 out that is not seen (relative error 1.67e-3, 1.66e-3 by the out's
// rounding alone), with an fp16 out it is (2.8e-4, 2.1e-4 alone); the second product that
// fp32 outs have takes the GEMM's time again (5120 x 17408, 2000 tokens 273 and 621 us).
template <int G>
__global__ void __launch_bounds__(256) linear_images_kernel(const uint8_t* __restrict__ w, size_t w_bytes,
                                                            const float* __restrict__ factors, int Nt, int Kc, int KS,
                                                            int tile0, long recs, bool rest, uint8_t* __restrict__ img,
                                                            size_t img_bytes) {
    using R = Rec<G>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (long rec = (long)blockIdx.x * 8 + (threadIdx.x >> 5); rec < recs; rec += (long)gridDim.x * 8) {
        const int kc = (int)(rec % Kc), lt = (int)(rec / Kc), tile = tile0 + lt;  // 16 rows, from the images' first
        const bool in = tile < Nt;
        const size_t at = ((size_t)(in ? tile : 0) * Kc + kc) * R::kBytes;
        uint32_t f[2][4], s[2][G <= 32 ? 2 : 1], z[2] = {0, 0};  // codes; scales and zeros of rows g and g + 8
        if (!QMLP_INB(at + R::kBytes - 1, w_bytes, 93)) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 c = ldg_stream_u4(reinterpret_cast<const uint4*>(w + at + 512 * h) + lane);
            f[h][0] = c.x, f[h][1] = c.y, f[h][2] = c.z, f[h][3] = c.w;
            const uint8_t* sp = w + at + 1024 + (2 * g + h) * (R::kScales / 16);
            const uint8_t* zp = w + at + 1024 + R::kScales + (2 * g + h) * R::kPer;
            if constexpr (G <= 32) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
                s[h][0] = v.x, s[h][1] = v.y;
                if constexpr (G == 32) z[h] = __ldg(reinterpret_cast<const unsigned int*>(zp));
            } else if constexpr (G == 64) {
                s[h][0] = __ldg(reinterpret_cast<const unsigned int*>(sp));
                z[h] = __ldg(reinterpret_cast<const unsigned short*>(zp));
            } else {
                s[h][0] = __ldg(reinterpret_cast<const unsigned short*>(sp));
                z[h] = __ldg(zp);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = lt * 16 + g + 8 * h, n = row & 255;
            // INT4: the images hold (code - zero) scale over the row's factor, a power of two
            const float rf = R::kNv || !in ? 1.0f : 1.0f / factors[tile * 16 + g + 8 * h];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // steps 2i, 2i + 1
                uint32_t a[4] = {0, 0, 0, 0};
                if (in) {
                    if constexpr (R::kNv) {
                        uint32_t s01, s23;
                        e4m3x4_to_f16x2x2(s[h][i >> 1], s01, s23);
                        e2m1x8(f[h][i], h2((i & 1) ? s23 : s01), a);
                    } else {
                        const int q = i * R::kPer / 4;
                        const __half2 z1 = h2(zero2(z[h], q));
                        int4x8(f[h][i], z1, __hadd2(z1, h2(0x63806380u)), a);
                        const float sc =
                            rf * __half2float(__ushort_as_half((unsigned short)(s[h][q >> 1] >> (16 * (q & 1)))));
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            float2 v = __half22float2(*reinterpret_cast<const __half2*>(&a[p]));
                            v.x *= sc, v.y *= sc;  // exact: 8 bits times 11
                            __half2 o = __floats2half2_rn(v.x, v.y);
                            if (rest) {  // what that leaves, exact as well (nothing of what is not finite)
                                const float2 r = __half22float2(o);
                                o = __floats2half2_rn(isfinite(r.x) ? v.x - r.x : 0.0f, isfinite(r.y) ? v.y - r.y : 0.0f);
                            }
                            a[p] = *reinterpret_cast<const uint32_t*>(&o);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int ks = 2 * kc + (i >> 1);                          // 64-k step
                    const int ch = 2 * (2 * (i & 1) + u) + (t >> 1);           // 16-byte chunk of its row
                    if (ks < KS) {
                        const size_t o = ((size_t)(row >> 8) * KS + ks) * 32768 + n * 128 + ((ch ^ (n & 7)) << 4) + 8 * (t & 1);
                        if (QMLP_INB(o + 7, img_bytes, 94)) *reinterpret_cast<uint2*>(img + o) = make_uint2(a[2 * u], a[2 * u + 1]);
                    }
                }
            }
        }
    }
}

// The factors of the images' rows, padded with ones.
__global__ void __launch_bounds__(256) linear_factors_kernel(const __half* __restrict__ scale, int groups, int N, float c,
                                                             float* __restrict__ factors, int padded) {
    const int lane = threadIdx.x & 31;
    for (int n = blockIdx.x * 8 + (threadIdx.x >> 5); n < padded; n += gridDim.x * 8) {
        float f = n < N ? c : 1.0f;
        if (scale && n < N) {
            float mx = 0.0f;
            for (int i = lane; i < groups; i += 32) mx = fmaxf(mx, fabsf(__half2float(scale[(size_t)n * groups + i])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // the largest scale to [2^5, 2^6): 255 of it stay below fp16's largest
            f = scalbnf(1.0f, 9 - prescale_exponent(mx));
        }
        if (lane == 0) factors[n] = f;
    }
}

// Bytes of x that one of S CTAs holds for M tokens.
size_t few_x_bytes(int K, int M, int S) {
    const int Kc = (K + kCh - 1) / kCh;
    return (size_t)((Kc + S - 1) / S) * 256 * M;
}

cudaLaunchConfig_t few_config(const FewPlan& P, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute* at) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P.S, (unsigned)P.gy);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)P.S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = P.S > 1 ? 2 : 1;
    return cfg;
}

template <int G, bool ONE, bool SUM>
cudaError_t launch_few(const LinearArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kC = ONE ? 1 : 8, W = few_warps<ONE>(), kStage = W * Rec<G>::kBytes, kCtas = few_ctas<ONE>();
    const int Kc = (a.K + kCh - 1) / kCh, Nt = (a.N + 15) / 16;
    const size_t room = kSmemMax / kCtas - 2048;  // of a CTA where the SM has all its CTAs
    FewPlan P = {};
    // k is split where x would take more than half of that, and where a warp would
    // have 16 records of a tile and more while half of the GPU has none (a cluster's
    // barriers cost 1.4 us: 1024 x 5120, 4.3 us without, 5.7 with two CTAs)
    P.S = 1;
    while (P.S < 8 && few_x_bytes(a.K, a.M, P.S) > room / 2) P.S *= 2;
    while (P.S < 8 && (long)Nt * P.S * 2 <= (long)num_sms * kCtas && Kc >= 16 * P.S * W) P.S *= 2;
    while (P.S > 1 && (P.S - 1) * ((Kc + P.S - 1) / P.S) >= Kc) P.S /= 2;  // every CTA has some of k
    // a tile's k is shared by as many warps as have two records or more of it: a copy
    // of the ring is their records of one tile, and small copies are slow (128000 x
    // 5120, one token: 78 us with eight records a copy, 84 with two or four, 112 with
    // one). Sixteen warps: by eight where that leaves every CTA two groups (17408 x
    // 5120, eight tokens: 17.3 us, 20.8 with sixteen).
    auto tile_groups = [&](int wpt) { return (Nt + W / wpt - 1) / (W / wpt); };
    P.wpt = W;
    while (P.wpt > 1 && ((Kc + P.S - 1) / P.S < 2 * P.wpt ||
                         (P.wpt > 8 && tile_groups(P.wpt / 2) * P.S >= 2 * kCtas * num_sms)))
        P.wpt /= 2;
    const int TG = W / P.wpt, groups = tile_groups(P.wpt);
    const size_t x = few_x_bytes(a.K, a.M, P.S);
    const size_t red = P.wpt > 1 ? (size_t)2 * W * kC * kPitch * 4 : 0;
    const size_t group_own = P.S > 1 || P.wpt == 1 ? (size_t)TG * kC * 16 * 4 : 0;
    if (x + red + group_own + 2 * kStage > kSmemMax - 2048) return cudaErrorInvalidValue;
    const bool one = x + red + group_own + 2 * kStage > room;  // one CTA an SM then
    const size_t all = one ? kSmemMax - 2048 : room;
    const int fit = one ? 1 : kCtas;
    P.gy = std::max(1, std::min(groups, num_sms * fit / P.S));
    const int mine = (groups + P.gy - 1) / P.gy;
    // Single CTAs fill every place, some with a group less (8192 x 5120 9.3 us; as many to
    // each in fewer CTAs 10.8). Clusters get as many each: the GPU does not hold as many
    // of them as its SMs would (5120 x 17408, eight tokens, S = 8: 21.4 us, 35.6 with all).
    if (P.S > 1) P.gy = (groups + mine - 1) / mine;
    P.batch = 1;
    if (P.S > 1) {  // a quarter of what is left for the sums that wait
        const size_t left = all - x - red - 2 * kStage;
        P.batch = (int)std::max<size_t>(1, std::min<size_t>(mine, left / 4 / group_own));
    }
    const size_t fixed = x + red + group_own * P.batch;
    P.stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(2, (all - fixed) / kStage));
    static unsigned long done = 0;
    if (const cudaError_t e = smem_once(linear_few_kernel<G, ONE, SUM>, kSmemMax, done); e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = few_config(P, (W + 1) * 32, fixed + (size_t)P.stages * kStage, s, at);
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<G, ONE, SUM>, a, P);
}

template <int G, int NT, bool SUM>
cudaError_t launch_mid(const LinearArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kC = 8 * NT, CS = mid_chunks<NT>(), kRec = Rec<G>::kBytes;
    const int Kc = (a.K + kCh - 1) / kCh, Nt = (a.N + 15) / 16;
    FewPlan P = {};
    // a CTA an SM, with eight tiles or more of its cluster's k where there are enough
    P.S = 1;
    while (P.S < 8 && Nt * P.S * 2 <= 12 * num_sms && Kc >= 4 * P.S * CS) P.S *= 2;
    while (P.S > 1 && (P.S - 1) * ((Kc + P.S - 1) / P.S) >= Kc) P.S /= 2;
    const int clusters = std::max(1, num_sms / P.S);
    P.tg = std::min(kMidWarps, (Nt + clusters - 1) / clusters);
    const int groups = (Nt + P.tg - 1) / P.tg;
    P.gy = std::min(groups, clusters);
    const size_t stage = (size_t)P.tg * CS * kRec + (size_t)CS * 256 * a.M, own = (size_t)kMidWarps * kC * 16 * 4;
    P.stages = (int)std::min<size_t>(kMaxStages, (kSmemMax - 2048 - own) / stage);
    if (P.stages < 2) return cudaErrorInvalidValue;
    static unsigned long done = 0;
    if (const cudaError_t e = smem_once(linear_mid_kernel<G, NT, SUM>, kSmemMax, done); e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    FewPlan X = {};
    X.S = 1;
    cudaLaunchConfig_t cfg = few_config(X, 256, 0, s, at);
    cfg.gridDim = dim3((unsigned)a.M);
    cudaError_t e = cudaLaunchKernelEx(&cfg, linear_x_kernel, a);
    if (e != cudaSuccess) return e;
    cfg = few_config(P, (kMidWarps + 1) * 32, own + (size_t)P.stages * stage, s, at);
    return cudaLaunchKernelEx(&cfg, linear_mid_kernel<G, NT, SUM>, a, P);
}

template <int G, bool SUM>
cudaError_t launch_tiles(const LinearArgs& a, int num_sms, cudaStream_t s) {
    if (a.M <= 16) return launch_mid<G, 2, SUM>(a, num_sms, s);
    return a.M <= 32 ? launch_mid<G, 4, SUM>(a, num_sms, s) : launch_mid<G, 8, SUM>(a, num_sms, s);
}
template <int G, bool SUM>
cudaError_t launch_sums(const LinearArgs& a, int num_sms, cudaStream_t s) {
    if (a.M == 1) return launch_few<G, true, SUM>(a, num_sms, s);
    if (a.M <= kLinearFew) return launch_few<G, false, SUM>(a, num_sms, s);
    return launch_tiles<G, SUM>(a, num_sms, s);
}
template <int G>
cudaError_t launch_g(const LinearArgs& a, int num_sms, cudaStream_t s) {
    if (a.M > kLinearMid) return cudaErrorInvalidValue;  // (the GEMM's)
    if (Rec<G>::kNv && a.odt == 0) return launch_sums<G, Rec<G>::kNv>(a, num_sms, s);
    return launch_sums<G, false>(a, num_sms, s);
}

}  // namespace

size_t linear_x_bytes(int K, int M) { return few_x_bytes(K, std::min(M, kLinearMid), 1); }

size_t linear_bytes(int group, int N, int K) {
    return (size_t)((N + 15) / 16) * ((K + kCh - 1) / kCh) * linear_rec_bytes(group);
}

cudaError_t repack_linear(int group, const uint8_t* w, const void* scale, const uint8_t* zero, int N, int K, uint8_t* out,
                          cudaStream_t s) {
    const int Kc = (K + kCh - 1) / kCh;
    const size_t items = (size_t)((N + 15) / 16) * Kc * 64;
    const unsigned grid = (unsigned)std::min<size_t>((items + 255) / 256, 65535);
    const uint8_t* sc = static_cast<const uint8_t*>(scale);
    switch (group) {
        case 16: repack_linear_kernel<16><<<grid, 256, 0, s>>>(w, sc, zero, N, K, Kc, items, out); break;
        case 32: repack_linear_kernel<32><<<grid, 256, 0, s>>>(w, sc, zero, N, K, Kc, items, out); break;
        case 64: repack_linear_kernel<64><<<grid, 256, 0, s>>>(w, sc, zero, N, K, Kc, items, out); break;
        case 128: repack_linear_kernel<128><<<grid, 256, 0, s>>>(w, sc, zero, N, K, Kc, items, out); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaPeekAtLastError();
}

cudaError_t launch_linear_images(int group, const uint8_t* w, size_t w_bytes, const float* factors, int N, int K, int n0,
                                 int rows, bool rest, uint8_t* img, size_t img_bytes, cudaStream_t s) {
    const int Kc = (K + kCh - 1) / kCh, KS = (K + 63) / 64, Nt = (N + 15) / 16;
    const long recs = (long)(rows / 16) * Kc;
    const unsigned grid = (unsigned)std::min<long>((recs + 7) / 8, 1 << 20);
    switch (group) {
        case 16: linear_images_kernel<16><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, rest, img, img_bytes); break;
        case 32: linear_images_kernel<32><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, rest, img, img_bytes); break;
        case 64: linear_images_kernel<64><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, rest, img, img_bytes); break;
        case 128: linear_images_kernel<128><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, rest, img, img_bytes); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaPeekAtLastError();
}

cudaError_t launch_linear_factors(int group, const void* scale, int N, int K, float c, float* factors, int padded,
                                  cudaStream_t s) {
    linear_factors_kernel<<<(unsigned)std::min((padded + 7) / 8, 65535), 256, 0, s>>>(
        group == 16 ? nullptr : static_cast<const __half*>(scale), K / group, N, c, factors, padded);
    return cudaPeekAtLastError();
}

cudaError_t launch_linear(int group, const LinearArgs& a, int num_sms, cudaStream_t s) {
    switch (group) {
        case 16: return launch_g<16>(a, num_sms, s);
        case 32: return launch_g<32>(a, num_sms, s);
        case 64: return launch_g<64>(a, num_sms, s);
        case 128: return launch_g<128>(a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

QMLP_BOUNDS_UNIT(linear)

}  // namespace qmlp
