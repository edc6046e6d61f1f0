// linear.cu -- one projection with 4-bit weights and group scales:
//   y[m, n] = c sum_k x[m, k] W[n, k] + bias[n]
//   NVFP4: W = E2M1(code) E4M3(scale[n, k / 16]), c = 1 / global
//   INT4:  W = (code - zero[n, k / G]) scale[n, k / G], G = 32, 64 or 128, c = 1
// for a few tokens (here) or many (images for the tensor-core GEMM, below).
//
// Few tokens (at most 64 a launch): the weights are read once.
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
//  * A CTA takes 16 rows at a time, its eight warps an eighth of its k each; the
//    warps' sums are added in their order. A cluster of up to eight CTAs splits k
//    where x would not fit in shared memory or the rows are too few for the GPU;
//    its CTAs add their sums through distributed shared memory, in their order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kCh = kLinearChunk;   // k of a record
constexpr int kW = 8;               // warps of a CTA
constexpr int kD = 2;               // records a warp has in flight
constexpr int kXBytes = 48 * 1024;  // shared memory that a CTA should spend on x at most
constexpr int kSmemMax = 220 * 1024;

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

// A lane's part of a record: codes of rows g and g + 8, and their scales.
template <int G>
struct Frag {
    uint4 c[2];
    uint32_t s[2][G >= 64 ? 1 : 2];  // NVFP4: 8 E4M3; INT4: the groups' fp16 scales
    uint32_t z[2];                   // INT4: the groups' zeros, a byte each
};
template <int G>
QMLP_DEV void load_frag(Frag<G>& f, const uint8_t* rec, int lane) {
    using R = Rec<G>;
    const int g = lane >> 2;
    f.c[0] = ldg_stream_u4(reinterpret_cast<const uint4*>(rec) + lane);
    f.c[1] = ldg_stream_u4(reinterpret_cast<const uint4*>(rec + 512) + lane);
    const uint8_t* sc = rec + 1024;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
        if constexpr (G <= 32) {
            const uint2 v = ldg_stream_u2(reinterpret_cast<const uint2*>(sc) + row);
            f.s[h][0] = v.x;
            f.s[h][1] = v.y;
        } else if constexpr (G == 64) {
            f.s[h][0] = __ldg(reinterpret_cast<const unsigned int*>(sc) + row);
        } else {
            f.s[h][0] = __ldg(reinterpret_cast<const unsigned short*>(sc) + row);
        }
        if constexpr (G == 32) f.z[h] = __ldg(reinterpret_cast<const unsigned int*>(sc + R::kScales) + row);
        else if constexpr (G == 64) f.z[h] = __ldg(reinterpret_cast<const unsigned short*>(sc + R::kScales) + row);
        else if constexpr (G == 128) f.z[h] = __ldg(sc + R::kScales + row);
    }
}

QMLP_DEV uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
QMLP_DEV uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
QMLP_DEV uint32_t hadd2u(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Zero of group i (byte i of z) as {-(1024 + z)} twice: 0xE400 is -1024, whose last
// place is one.
QMLP_DEV uint32_t zero2(uint32_t z, int i) { return __byte_perm(z, 0xE4E4E4E4u, 0x4040u | (uint32_t)(i | i << 8)); }
// Eight codes (two steps of a row) less their zero: nibbles p and p + 4 of the word
// are pair p; 0x6400 | q is 1024 + q, 0x6400 | 16 q is 1024 + 16 q; both steps exact.
QMLP_DEV void int4x8(uint32_t w, uint32_t z1, uint32_t z16, uint32_t (&p)[4]) {
    const uint32_t v = w >> 8;
    p[0] = hadd2u((w & 0x000F000Fu) | 0x64006400u, z1);
    p[1] = hfma2u((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, z16);
    p[2] = hadd2u((v & 0x000F000Fu) | 0x64006400u, z1);
    p[3] = hfma2u((v & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, z16);
}

// One record times NT tiles of eight tokens. xb: this lane's x of the record, a
// uint4 a pair of steps and tile, `xs` apart (tiles: their own pointers).
template <int G, int NT>
QMLP_DEV void mma_record(const Frag<G>& f, const uint4* const (&xb)[NT], int xs, float (&acc)[NT][4]) {
    using R = Rec<G>;
    if constexpr (R::kNv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // two steps: groups 2i and 2i + 1 of both rows
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                e2m1x4_to_f16x2x4(word_of(f.c[h], i), a[h][0], a[h][1], a[h][2], a[h][3]);
                const uint32_t sp = e4m3x2_to_f16x2((f.s[h][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                const uint32_t lo = dup_lo16(sp), hi = dup_hi16(sp);
                a[h][0] = hmul2_u32(a[h][0], lo);
                a[h][1] = hmul2_u32(a[h][1], lo);
                a[h][2] = hmul2_u32(a[h][2], hi);
                a[h][3] = hmul2_u32(a[h][3], hi);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x = xb[n][i * xs];
                mma_f16_16816(acc[n], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                mma_f16_16816(acc[n], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < R::kPer; ++q) {
            uint32_t z1[2], z16[2];
            float s[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                z1[h] = zero2(f.z[h], q);
                z16[h] = hadd2u(z1[h], 0x63806380u);  // -(1024 + z) + 960 = -(64 + z)
                s[h] = __half2float(__ushort_as_half((unsigned short)(f.s[h][q >> 1] >> (16 * (q & 1)))));
            }
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
#pragma unroll
            for (int i = q * (4 / R::kPer); i < (q + 1) * (4 / R::kPer); ++i) {
                uint32_t a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) int4x8(word_of(f.c[h], i), z1[h], z16[h], a[h]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 x = xb[n][i * xs];
                    mma_f16_16816(d[n], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                    mma_f16_16816(d[n], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s[0], d[n][0], acc[n][0]);
                acc[n][1] = fmaf(s[0], d[n][1], acc[n][1]);
                acc[n][2] = fmaf(s[1], d[n][2], acc[n][2]);
                acc[n][3] = fmaf(s[1], d[n][3], acc[n][3]);
            }
        }
    }
}

QMLP_DEV void lin_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QMLP_DEV float peer_f32(const float* p, int rank) {
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}

QMLP_DEV int peer_s32(const int* p, int rank) {
    uint32_t ra;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

QMLP_DEV void store_out(const LinearArgs& a, int m, int n, float v) {
    const size_t at = (size_t)m * a.N + n;
    if (!QMLP_INB(at, (size_t)a.M * a.N, 92)) return;
    if (a.bias) v += __ldg(a.bias + n);
    if (a.odt == 0) static_cast<float*>(a.out)[at] = v;
    else if (a.odt == 1) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(a.out)[at] = __float2half_rn(v);
}

// Grid (splits, CTAs of a split), cluster (splits, 1). Shared memory: x, the
// warps' sums (two buffers), this CTA's sums of its tiles where k is split.
// Buffers of the warps' sums: with two, one barrier a tile is enough.
template <int NT>
constexpr int red_bufs() { return NT <= 2 ? 2 : 1; }
template <int NT>
constexpr int few_ctas() { return NT == 1 ? 3 : NT == 8 ? 1 : 2; }

template <int G, int NT>
__global__ void __launch_bounds__(kW * 32, few_ctas<NT>()) linear_few_kernel(const LinearArgs a) {
    using R = Rec<G>;
    constexpr int kC = 8 * NT;  // columns
    extern __shared__ __align__(16) uint4 xsm[];
    __shared__ int s_max[kC], s_sig[kC];
    const int S = gridDim.x, rank = blockIdx.x, M = a.M, K = a.K;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int Kc = (K + kCh - 1) / kCh, Nt = (a.N + 15) / 16;
    const int cps = (Kc + S - 1) / S;                     // records of k a CTA
    const int kc0 = rank * cps, nch = min(cps, Kc - kc0);  // this one's
    const int cpw = (cps + kW - 1) / kW;
    const int c0 = warp * cpw, cw = max(0, min(cpw, nch - c0));  // this warp's
    float* red = reinterpret_cast<float*>(xsm + (size_t)cps * 16 * M);  // [buffers][kW][16][kC]
    float* own = red + red_bufs<NT>() * kW * 16 * kC;                   // [tiles][16][kC]
    const int tiles = (Nt - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;

    // the first records are on their way before anything else
    const uint8_t* base = a.w + (size_t)(kc0 + c0) * R::kBytes;
    const size_t tile_bytes = (size_t)Kc * R::kBytes, hop = tile_bytes * gridDim.y;
    const uint8_t* next = base + (size_t)blockIdx.y * tile_bytes;  // record that is loaded next
    int nc = 0, nt = 0;                                            // its place in the slice, its tile
    auto fetch = [&](Frag<G>& f) {
        if (nt < tiles) {
            if (QMLP_INB(next - a.w + R::kBytes - 1, a.w_bytes, 91)) load_frag<G>(f, next, lane);
            next += R::kBytes;
            if (++nc == cw) {
                nc = 0;
                ++nt;
                next += hop - (size_t)cw * R::kBytes;
            }
        }
    };
    Frag<G> fr[kD];
    if (cw > 0)
#pragma unroll
        for (int d = 0; d < kD; ++d) fetch(fr[d]);

    // x of this CTA's k, in the order of the steps: slot ((c 4 + i) M + m) 4 + t has
    // k = 128 c + 32 i + 4 t.. (four) and 16 further (four) of token m. A thread
    // stays with one token: its largest value falls out of the copy, and the copy is
    // scaled in place once the row's exponent is known (M = 1, K = 5120: the kernel
    // took 10.3 us with a pass over x for the largest value before the copy)
    constexpr int kMp = NT == 1 ? 8 : 8 * NT;  // (M = 1: all threads on its row)
    const int mp = NT == 1 && M == 1 ? 1 : kMp;
    const int k0 = kc0 * kCh, xt = threadIdx.x & 3, xm = (threadIdx.x >> 2) % mp, hop_c = kW * 8 / mp;
    if (threadIdx.x < kC) s_max[threadIdx.x] = 0;
    __syncthreads();
    if (xm < M) {
        float mx = 0.0f;
        const uint16_t* row = static_cast<const uint16_t*>(a.x) + (size_t)xm * K;
#pragma unroll 4
        for (int ci = (threadIdx.x >> 2) / mp; ci < nch * 4; ci += hop_c) {
            const int k = k0 + 32 * ci + 4 * xt;
            uint2 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)  // K is a multiple of 16
                v[h] = k + 16 * h < K ? __ldg(reinterpret_cast<const uint2*>(row + k + 16 * h)) : make_uint2(0, 0);
            if (a.x_bf16)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(v[h].x << 16)), fabsf(__uint_as_float(v[h].x & 0xFFFF0000u))),
                                         fmaxf(fabsf(__uint_as_float(v[h].y << 16)), fabsf(__uint_as_float(v[h].y & 0xFFFF0000u)))));
            xsm[(ci * M + xm) * 4 + xt] = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
        }
        if (a.x_bf16) atomicMax(s_max + xm, __float_as_int(mx));
    }
    if (a.x_bf16) {
        if (S > 1) lin_cluster_sync();
        else __syncthreads();
        if (threadIdx.x < M) {
            int mx = 0;
            for (int r = 0; r < S; ++r) mx = max(mx, S > 1 ? peer_s32(s_max + threadIdx.x, r) : s_max[threadIdx.x]);
            s_sig[threadIdx.x] = prescale_exponent(__int_as_float(mx));
        }
        __syncthreads();
        if (xm < M) {
            const int sg = s_sig[xm];
            for (int ci = (threadIdx.x >> 2) / mp; ci < nch * 4; ci += hop_c) {
                uint4& slot = xsm[(ci * M + xm) * 4 + xt];
                const uint4 u = slot;
                uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 hv = __floats2half2_rn(scalbnf(__uint_as_float(v[j] << 16), sg),
                                                         scalbnf(__uint_as_float(v[j] & 0xFFFF0000u), sg));
                    v[j] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                slot = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    } else if (threadIdx.x < M) {
        s_sig[threadIdx.x] = 0;
    }
    __syncthreads();

    const uint4* xw[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xw[n] = xsm + (size_t)c0 * 16 * M + min(8 * n + g, M - 1) * 4 + t;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    // the warps' sums of a tile -> out, or this CTA's share of it
    int tile = 0;
    auto finish = [&] {
        float* rb = red + (red_bufs<NT>() > 1 ? (tile & 1) * kW * 16 * kC : 0);
        if (red_bufs<NT>() == 1) __syncthreads();  // the sums of the tile before are read
        float* mine = rb + warp * 16 * kC;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2*>(mine + g * kC + 8 * n + 2 * t) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2*>(mine + (g + 8) * kC + 8 * n + 2 * t) = make_float2(acc[n][2], acc[n][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
        }
        __syncthreads();
        const int row = threadIdx.x & 15, j = (int)blockIdx.y + tile * (int)gridDim.y;
        for (int m = threadIdx.x >> 4; m < M; m += kW * 2) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kW; ++w) v += rb[(w * 16 + row) * kC + m];
            if (S > 1) own[(tile * 16 + row) * kC + m] = v;
            else if (16 * j + row < a.N) store_out(a, m, 16 * j + row, scalbnf(v, -s_sig[m]) * a.factor);
        }
        ++tile;
    };
    if (cw > 0) {
        const int total = tiles * cw;
        int c = 0;
        for (int i = 0; i < total; i += kD) {
#pragma unroll
            for (int d = 0; d < kD; ++d) {
                if (i + d < total) {
                    const uint4* xb[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xb[n] = xw[n] + (size_t)c * 16 * M;
                    mma_record<G, NT>(fr[d], xb, 4 * M, acc);
                    fetch(fr[d]);
                    if (++c == cw) {
                        c = 0;
                        finish();
                    }
                }
            }
        }
    } else {
        while (tile < tiles) finish();
    }
    if (S > 1) {
        lin_cluster_sync();  // every CTA's shares are written
        const int per = (tiles * 16 * M + S - 1) / S;
        for (int i = rank * per + threadIdx.x; i < min(tiles * 16 * M, (rank + 1) * per); i += blockDim.x) {
            const int row = i & 15, m = (i >> 4) % M, tl = (i >> 4) / M;
            const int n = 16 * ((int)blockIdx.y + tl * (int)gridDim.y) + row;
            float v = 0.0f;
            for (int r = 0; r < S; ++r) v += peer_f32(own + (tl * 16 + row) * kC + m, r);
            if (n < a.N) store_out(a, m, n, scalbnf(v, -s_sig[m]) * a.factor);
        }
        lin_cluster_sync();  // none leaves while another reads its shares
    }
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
            const int r = g + 8 * h, groups = K / G;
            for (int q = 0; q < R::kPer; ++q) {
                const int gi = kc * R::kPer + q;
                const bool in = row < (size_t)N && gi < groups;
                const size_t at = row * groups + gi;
                if (R::kNv) {
                    dst[1024 + r * R::kPer + q] = in ? scale[at] : 0;
                } else {
                    reinterpret_cast<uint16_t*>(dst + 1024)[r * R::kPer + q] =
                        in ? reinterpret_cast<const uint16_t*>(scale)[at] : (uint16_t)0;
                    dst[1024 + R::kScales + r * R::kPer + q] = in ? zero[at] : 0;
                }
            }
        }
    }
}

// Records -> stage images: a warp a record (16 rows x 128 k), each lane the four k
// of its two rows that it has of a step, 8 bytes of an image row at a time.
template <int G>
__global__ void __launch_bounds__(256) linear_images_kernel(const uint8_t* __restrict__ w, size_t w_bytes,
                                                            const float* __restrict__ factors, int Nt, int Kc, int KS,
                                                            int tile0, long recs, uint8_t* __restrict__ img,
                                                            size_t img_bytes) {
    using R = Rec<G>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (long rec = (long)blockIdx.x * 8 + (threadIdx.x >> 5); rec < recs; rec += (long)gridDim.x * 8) {
        const int kc = (int)(rec % Kc), lt = (int)(rec / Kc), tile = tile0 + lt;  // 16 rows, from the images' first
        Frag<G> f;
        const bool in = tile < Nt;
        const size_t at = ((size_t)(in ? tile : 0) * Kc + kc) * R::kBytes;
        if (in && QMLP_INB(at + R::kBytes - 1, w_bytes, 93)) load_frag<G>(f, w + at, lane);
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
                        e2m1x4_to_f16x2x4(word_of(f.c[h], i), a[0], a[1], a[2], a[3]);
                        const uint32_t sp = e4m3x2_to_f16x2((f.s[h][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                        const uint32_t lo = dup_lo16(sp), hi = dup_hi16(sp);
                        a[0] = hmul2_u32(a[0], lo);
                        a[1] = hmul2_u32(a[1], lo);
                        a[2] = hmul2_u32(a[2], hi);
                        a[3] = hmul2_u32(a[3], hi);
                    } else {
                        const int q = i * R::kPer / 4;
                        const uint32_t z1 = zero2(f.z[h], q);
                        int4x8(word_of(f.c[h], i), z1, hadd2u(z1, 0x63806380u), a);
                        const float s =
                            rf * __half2float(__ushort_as_half((unsigned short)(f.s[h][q >> 1] >> (16 * (q & 1)))));
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&a[p]));
                            const __half2 o = __floats2half2_rn(v.x * s, v.y * s);
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

template <int G, int NT>
cudaError_t launch_few(const LinearArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kC = 8 * NT;
    const int Kc = (a.K + kCh - 1) / kCh, Nt = (a.N + 15) / 16;
    // k is split where x of one CTA would be too large, then as long as the GPU
    // has room for twice the CTAs and every warp keeps a record or more
    int S = 1;
    auto xbytes = [&](int sp) { return (size_t)((Kc + sp - 1) / sp) * 256 * a.M; };
    while (S < 8 && (xbytes(S) > kXBytes || ((long)Nt * S * 2 <= 2L * num_sms && Kc >= 2 * S * kW))) S *= 2;
    while (S > 1 && (S - 1) * ((Kc + S - 1) / S) >= Kc) S /= 2;  // every CTA has some of k
    if (xbytes(S) > kSmemMax - 64 * 1024) return cudaErrorInvalidValue;
    // as many CTAs as fit at once, each on an even share of the tiles
    const size_t fixed = xbytes(S) + red_bufs<NT>() * kW * 16 * kC * sizeof(float);
    const int fit = (int)std::max<size_t>(1, std::min<size_t>(few_ctas<NT>(), kSmemMax / (fixed + 2048)));
    int gy = std::max(1, std::min(Nt, num_sms * fit / S));
    int tiles = (Nt + gy - 1) / gy;
    // a split's sums of all its tiles wait in shared memory
    const int most = (int)((kSmemMax / fit - fixed) / (16 * kC * sizeof(float)));
    if (S > 1 && tiles > most) tiles = std::max(1, most);
    gy = (Nt + tiles - 1) / tiles;
    const size_t smem = fixed + (S > 1 ? (size_t)tiles * 16 * kC * sizeof(float) : 0);
    static bool attr = false;
    if (!attr) {
        const cudaError_t e = cudaFuncSetAttribute(linear_few_kernel<G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemMax);
        if (e != cudaSuccess) return e;
        attr = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S, (unsigned)gy);
    cfg.blockDim = dim3(kW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<G, NT>, a);
}

template <int G>
cudaError_t launch_g(LinearArgs a, int num_sms, cudaStream_t s) {
    // several launches of as many tokens each as one takes: 64, or what a cluster's
    // shared memory has room for
    const size_t ob = a.odt == 0 ? 4 : 2;
    const int M = a.M;
    int most = 64;
    while (most > 8 && (size_t)((a.K + 8 * kCh - 1) / (8 * kCh)) * 256 * most > kSmemMax - 64 * 1024) most /= 2;
    const int blocks = (M + most - 1) / most, step = ((M + blocks - 1) / blocks + 7) / 8 * 8;
    for (int m = 0; m < M; m += step) {
        LinearArgs b = a;
        b.M = std::min(step, M - m);
        b.x = static_cast<const uint8_t*>(a.x) + (size_t)m * a.K * 2;
        b.out = static_cast<uint8_t*>(a.out) + (size_t)m * a.N * ob;
        const cudaError_t e = b.M <= 8    ? launch_few<G, 1>(b, num_sms, s)
                              : b.M <= 16 ? launch_few<G, 2>(b, num_sms, s)
                              : b.M <= 32 ? launch_few<G, 4>(b, num_sms, s)
                                          : launch_few<G, 8>(b, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

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
                                 int rows, uint8_t* img, size_t img_bytes, cudaStream_t s) {
    const int Kc = (K + kCh - 1) / kCh, KS = (K + 63) / 64, Nt = (N + 15) / 16;
    const long recs = (long)(rows / 16) * Kc;
    const unsigned grid = (unsigned)std::min<long>((recs + 7) / 8, 1 << 20);
    switch (group) {
        case 16: linear_images_kernel<16><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, img, img_bytes); break;
        case 32: linear_images_kernel<32><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, img, img_bytes); break;
        case 64: linear_images_kernel<64><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, img, img_bytes); break;
        case 128: linear_images_kernel<128><<<grid, 256, 0, s>>>(w, w_bytes, factors, Nt, Kc, KS, n0 / 16, recs, img, img_bytes); break;
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
