// norm.cuh -- the norms before and after a block, fused with its gate, residual
// and residual scale; forward and backward.
//
// For every token (row), with z the block's output and r the residual stream:
//   n = z / rms(z) * (post_w + offset)      (no norm after the block: n = z)
//   h = r + scale * gate * n                (the residual stream behind the block)
//   y = h / rms(h) * (pre_w + offset)       (the next block's input)
//   rms(v) = sqrt(mean(v^2) + eps)
// gate: none, a value a channel, a token, or an element. Backward, from d y and
// the gradient d h of the stream behind (hh = h / rms(h), zh = z / rms(z)):
//   a  = dy (pre_w + offset);  dH = dh + (a - hh mean(a hh)) / rms(h);  d r = dH
//   dn = scale gate dH;  b = dn (post_w + offset);  d z = (b - zh mean(b zh)) / rms(z)
//   d pre_w = sum over tokens of dy hh;  d post_w = sum of dn zh
//   d gate = scale dH n, summed over what shares the gate's value
// h enters the norm as it is before its rounding to the stream's type, and the
// backward pass recomputes it from z and r with the two 1/rms that the forward
// kept: every value is rounded once, when it is stored. Sums are fp32.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kWarps = 8;  // rows (warps) of a CTA where a warp takes a row

template <typename T>
QMLP_DEV void open8(const uint4& a, float (&v)[8]) {
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
// V values of T as they lie in memory.
template <typename T, int V>
struct Packed {
    T v;
    QMLP_DEV void zero() { v = (T)0.0f; }
    QMLP_DEV void load(const T* p) { v = *p; }
    QMLP_DEV void open(float (&f)[V]) const { f[0] = (float)v; }
};
template <typename T>
struct Packed<T, 8> {
    uint4 v;
    QMLP_DEV void zero() { v = make_uint4(0, 0, 0, 0); }
    QMLP_DEV void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
    QMLP_DEV void open(float (&f)[8]) const { open8<T>(v, f); }
};
template <typename T, int V>
QMLP_DEV void ldv(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = (float)*p;
    } else if constexpr (sizeof(T) == 4) {
        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {  // a whole sector at once
            static_assert(V == 8);
            asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                         : "l"(p) : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i);
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        }
    } else {
        open8<T>(*reinterpret_cast<const uint4*>(p), v);
    }
}
QMLP_DEV void put(float* p, float v) { *p = v; }
QMLP_DEV void put(__half* p, float v) { *p = __float2half_rn(v); }
QMLP_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <typename T, int V>
QMLP_DEV void stv(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        put(p, v[0]);
    } else if constexpr (sizeof(T) == 4) {
        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
            asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                         "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// Weights: of T, or fp32.
template <typename T, int V>
QMLP_DEV void ldw(const void* p, bool f32, int i, float (&v)[V]) {
    if (f32) ldv<float, V>(static_cast<const float*>(p) + i, v);
    else ldv<T, V>(static_cast<const T*>(p) + i, v);
}

QMLP_DEV float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The sums of N values over a row's threads, in every thread. WARP: a warp has the row;
// else the CTA, through one of two buffers in turn (`turn` flips), so that one barrier a
// sum is enough.
template <bool WARP, int N>
QMLP_DEV void row_sum(float (&v)[N], float (*buf)[N][32], int& turn) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = warp_sum(v[j]);
    if (WARP) return;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < N; ++j) buf[turn][j][threadIdx.x >> 5] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float t = (threadIdx.x & 31) < nw ? buf[turn][j][threadIdx.x & 31] : 0.0f;
        v[j] = warp_sum(t);
    }
    turn ^= 1;
}

// Column of a thread's chunk i, and the row that a CTA's thread works on.
template <int V, bool WARP>
QMLP_DEV int column(int i) {
    return (WARP ? i * 32 + (int)(threadIdx.x & 31) : i * (int)blockDim.x + (int)threadIdx.x) * V;
}

// TIGHT: 32 registers a thread.
template <typename T, typename R, int V, int NC, bool WARP, bool TIGHT>
__global__ void __launch_bounds__(WARP ? kWarps * 32 : 1024, TIGHT ? 2 : 1) norm_forward_kernel(const NormArgs a) {
    __shared__ float buf[2][1][32];
    int turn = 0;
    const long m = WARP ? (long)blockIdx.x * kWarps + (threadIdx.x >> 5) : (long)blockIdx.x;
    if (m >= a.M) return;  // (WARP: no barrier follows)
    const int K = a.K;
    const size_t at = (size_t)m * K;
    const T* z = static_cast<const T*>(a.z) + at;
    const R* r = static_cast<const R*>(a.r) + at;
    float h[NC][V];
    Packed<T, V> zp[NC];  // (as it came: registers)
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = column<V, WARP>(i);
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] = 0.0f;
        zp[i].zero();
        if (c < K && QMLP_INB(at + c + V - 1, a.elems, 81)) {
            if (a.z) zp[i].load(z + c);
            if (a.r) ldv<R, V>(r + c, h[i]);
            if (a.gate_kind == kGateFull && a.post_w)  // (into L2 while the row is summed: 4096 x 4096 36.1 -> 34.5 us)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(a.gate) + at + c));
        }
    }
    float rz = 1.0f, rh = 1.0f;
    if (a.z) {
        if (a.post_w) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float v[V];
                zp[i].open(v);
#pragma unroll
                for (int e = 0; e < V; ++e) ss[0] = fmaf(v[e], v[e], ss[0]);
            }
            row_sum<WARP, 1>(ss, buf, turn);
            rz = rsqrtf(ss[0] * a.rK + a.eps);
        }
        const float gt = a.gate_kind == kGateToken ? (float)static_cast<const T*>(a.gate)[m] : 1.0f;
        const float s = a.scale * gt;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
            if (c < K) {
                float w[V], g[V], v[V];
                zp[i].open(v);
                if (a.post_w) ldw<T, V>(a.post_w, a.w_f32, c, w);
                if (a.gate_kind == kGateChannel) ldw<T, V>(a.gate, a.w_f32, c, g);
                if (a.gate_kind == kGateFull) ldv<T, V>(static_cast<const T*>(a.gate) + at + c, g);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float n = v[e];
                    if (a.post_w) n = n * rz * (w[e] + a.offset);
                    if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) n *= g[e];
                    h[i][e] = fmaf(s, n, h[i][e]);
                }
            }
        }
    }
    if (a.h) {
        R* ho = static_cast<R*>(a.h) + at;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
            if (c < K) stv<R, V>(ho + c, h[i]);
        }
    }
    if (a.pre_w) {
        ss[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) ss[0] = fmaf(h[i][e], h[i][e], ss[0]);
        row_sum<WARP, 1>(ss, buf, turn);
        rh = rsqrtf(ss[0] * a.rK + a.eps);
        T* y = static_cast<T*>(a.y) + at;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
            if (c < K) {
                float w[V];
                ldw<T, V>(a.pre_w, a.w_f32, c, w);
#pragma unroll
                for (int e = 0; e < V; ++e) w[e] = h[i][e] * rh * (w[e] + a.offset);
                stv<T, V>(y + c, w);
            }
        }
    }
    if (a.stats && (WARP ? threadIdx.x & 31 : threadIdx.x) == 0) a.stats[m] = make_float2(rz, rh);
}

template <typename T, typename R, int V, int NC, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarps * 32 : 1024) norm_backward_kernel(const NormArgs a) {
    __shared__ float buf1[2][1][32], buf2[2][2][32];
    extern __shared__ float cols[];  // WARP: [3][K], the CTA's sums over its rows
    int turn1 = 0, turn2 = 0;
    const int K = a.K;
    float acc[3][NC][V];  // d post_w, d pre_w, d gate (a value a channel)
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[j][i][e] = 0.0f;
    const long rows = WARP ? (long)gridDim.x * kWarps : (long)gridDim.x;
    for (long m = WARP ? (long)blockIdx.x * kWarps + (threadIdx.x >> 5) : (long)blockIdx.x; m < a.M; m += rows) {
        const size_t at = (size_t)m * K;
        const float2 st = a.stats[m];
        const float rz = a.post_w ? st.x : 1.0f, rh = st.y;
        const float gt = a.gate_kind == kGateToken ? (float)static_cast<const T*>(a.gate)[m] : 1.0f;
        float z[NC][V], h[NC][V], dh[NC][V], dy[NC][V];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
#pragma unroll
            for (int e = 0; e < V; ++e) z[i][e] = h[i][e] = dh[i][e] = dy[i][e] = 0.0f;
            if (c < K && QMLP_INB(at + c + V - 1, a.elems, 82)) {
                if (a.z) ldv<T, V>(static_cast<const T*>(a.z) + at + c, z[i]);
                if (a.r) ldv<R, V>(static_cast<const R*>(a.r) + at + c, h[i]);
                if (a.dh) ldv<R, V>(static_cast<const R*>(a.dh) + at + c, dh[i]);
                if (a.dy) ldv<T, V>(static_cast<const T*>(a.dy) + at + c, dy[i]);
            }
        }
        // n (kept in z's place where the norm after the block is there: zh), g
        float g[NC][V], c1[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
#pragma unroll
            for (int e = 0; e < V; ++e) g[i][e] = a.scale * gt;
            if (c < K) {
                float w[V];
                if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
                    if (a.gate_kind == kGateChannel) ldw<T, V>(a.gate, a.w_f32, c, w);
                    else ldv<T, V>(static_cast<const T*>(a.gate) + at + c, w);
#pragma unroll
                    for (int e = 0; e < V; ++e) g[i][e] = a.scale * w[e];
                }
                if (a.post_w) ldw<T, V>(a.post_w, a.w_f32, c, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    z[i][e] *= rz;
                    h[i][e] = fmaf(g[i][e], a.post_w ? z[i][e] * (w[e] + a.offset) : z[i][e], h[i][e]);
                }
                if (a.pre_w) {
                    ldw<T, V>(a.pre_w, a.w_f32, c, w);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        h[i][e] *= rh;  // hh
                        acc[1][i][e] = fmaf(dy[i][e], h[i][e], acc[1][i][e]);
                        dy[i][e] *= w[e] + a.offset;
                        c1[0] = fmaf(dy[i][e], h[i][e], c1[0]);
                    }
                }
            }
        }
        if (a.pre_w) {
            row_sum<WARP, 1>(c1, buf1, turn1);
            const float mean = c1[0] * a.rK;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) dh[i][e] = fmaf(rh, fmaf(-h[i][e], mean, dy[i][e]), dh[i][e]);
        }
        if (a.dr) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = column<V, WARP>(i);
                if (c < K) stv<R, V>(static_cast<R*>(a.dr) + at + c, dh[i]);
            }
        }
        if (!a.z) continue;
        float c2[2] = {0.0f, 0.0f};  // sum of b zh; of dH n for a token's gate
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
            if (c < K) {
                float w[V], dg[V];
                if (a.post_w) ldw<T, V>(a.post_w, a.w_f32, c, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float wo = a.post_w ? w[e] + a.offset : 1.0f;
                    dg[e] = a.scale * (dh[i][e] * (z[i][e] * wo));
                    acc[2][i][e] += dg[e];
                    c2[1] += dg[e];
                    const float dn = g[i][e] * dh[i][e];
                    acc[0][i][e] = fmaf(dn, z[i][e], acc[0][i][e]);
                    dh[i][e] = dn * wo;  // b
                    c2[0] = fmaf(dh[i][e], z[i][e], c2[0]);
                }
                if (a.gate_kind == kGateFull && a.dgate) stv<T, V>(static_cast<T*>(a.dgate) + at + c, dg);
            }
        }
        if (a.post_w || (a.gate_kind == kGateToken && a.dgate)) row_sum<WARP, 2>(c2, buf2, turn2);
        if (a.gate_kind == kGateToken && a.dgate && (WARP ? threadIdx.x & 31 : threadIdx.x) == 0)
            put(static_cast<T*>(a.dgate) + m, c2[1]);
        if (a.dz) {
            const float mean = c2[0] * a.rK;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = column<V, WARP>(i);
                if (c < K) {
                    if (a.post_w)
#pragma unroll
                        for (int e = 0; e < V; ++e) dh[i][e] = rz * fmaf(-z[i][e], mean, dh[i][e]);
                    stv<T, V>(static_cast<T*>(a.dz) + at + c, dh[i]);
                }
            }
        }
    }
    if (!a.part) return;
    // this CTA's sums over its rows, [3][K]
    float* part = a.part + (size_t)blockIdx.x * 3 * K;
    if (WARP) {
        for (int w = 0; w < kWarps; ++w) {  // warp after warp: a fixed order
            if ((int)(threadIdx.x >> 5) == w)
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int c = column<V, WARP>(i);
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (c < K) cols[j * K + c + e] = (w ? cols[j * K + c + e] : 0.0f) + acc[j][i][e];
                    }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 3 * K; i += blockDim.x)
            if (QMLP_INB((size_t)blockIdx.x * 3 * K + i, a.part_elems, 83)) part[i] = cols[i];
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = column<V, WARP>(i);
                if (c < K && QMLP_INB((size_t)blockIdx.x * 3 * K + j * K + c + V - 1, a.part_elems, 83))
#pragma unroll
                    for (int e = 0; e < V; ++e) part[(size_t)j * K + c + e] = acc[j][i][e];
            }
    }
}

// ---------------------------------------------------------------------------
// Rows in walks: a group of threads walks over rows, RP of them at a time, the next ones
// on their way into shared memory meanwhile (cp.async; a warp reads only what it has
// copied itself, so no barrier waits for the copies). Arrays are taken in aligned chunks
// of eight values whatever K is: a row that starts s values behind such a border has its
// first chunk s values early, and masks what belongs to its neighbours. A group's rows
// are a multiple of eight apart, so s is the same for all of them and a thread keeps its
// columns. With A = scale (post_w + offset) and a channel's gate in it, B = pre_w + offset
// (fp32, in shared memory), u = A (times the gate of an element) and t a token's gate:
//   q = zh u;  h = r + t q;  y = h / rms(h) B
//   dH = dh + dy B / rms - hh mean / rms, mean = sum(dy B hh) / K
// dH is linear in mean, so that one round of sums over the row does for both norms:
//   sum dH q = sum (dh + dy B / rms) q - mean / rms sum hh q;  d z = t u dH / rms(z) - zh t (sum dH q) / (K rms(z))
// and the columns' sums of dH zh give d post_w and a channel gate's gradient both.
// What bounds them is instructions and the sums' latency more than memory, hence the
// layout: a warp's pieces of 512 bytes lie one behind the other, every offset a constant.
// G: kAny, or z, the residual and both norms are there and no element has
// its own gate (kScalar) or every one has (kFull).
// ---------------------------------------------------------------------------
// (768: 4096 x 3333, whose rows take 448 threads, 42 us instead of 30; 1024: 31, and 8192 x
// 5120 69 instead of 66, by their fewer registers)
constexpr int kForwardThreads = 896;
constexpr int kAny = 0, kScalar = 1, kFull = 2;
// 16 bytes on their way, the first n of them from memory, zeros behind
QMLP_DEV void cp16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
QMLP_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QMLP_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
QMLP_DEV void cp_wait_but(int n) {  // all but the last n fetches
    if (n >= 3) cp_wait<3>();
    else if (n == 2) cp_wait<2>();
    else if (n == 1) cp_wait<1>();
    else cp_wait<0>();
}
// Sums of N values over a group, in every thread: lanes exchange halves of the values,
// so that N take little more than the steps of one.
template <int N>
QMLP_DEV void group_sum(float (&v)[N], float (*buf)[192], int& turn, int tg, int rg) {
    constexpr int NP = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : 8, L = 32 / NP;  // L lanes end with one value
    const int lane = threadIdx.x & 31;
    float t[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) t[j] = j < N ? v[j] : 0.0f;
#pragma unroll
    for (int c = NP / 2, o = 16; o > 0; o >>= 1, c >>= 1) {
        if (c > 0) {
#pragma unroll
            for (int j = 0; j < c; ++j) {
                const bool up = lane & o;
                const float keep = up ? t[j + c] : t[j], give = up ? t[j] : t[j + c];
                t[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        } else {
            t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
        }
    }
    if (tg > 32) {
        const int nw = tg >> 5;
        if (lane % L == 0) buf[turn][(threadIdx.x >> 5) * NP + lane / L] = t[0];
        named_bar_sync(1 + rg, tg);
        t[0] = 0.0f;
        for (int i = lane % L; i < nw; i += L) t[0] += buf[turn][(rg * nw + i) * NP + lane / L];
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
        turn ^= 1;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = NP == 1 ? t[0] : __shfl_sync(0xffffffffu, t[0], j * L);
}
QMLP_DEV uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
QMLP_DEV void sts16(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Two fp32 values in a register pair: one instruction for both (4096 x 4096 with an
// element's gate, backward: 61 us, one by one 63, 533 instructions a warp and row of 256
// values; 16384 x 1024 55 to 58 us).
typedef unsigned long long f2;
QMLP_DEV f2 pair(float a, float b) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
QMLP_DEV f2 both(float a) { return pair(a, a); }
QMLP_DEV float2 two(f2 v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
QMLP_DEV f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
QMLP_DEV f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
QMLP_DEV f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
QMLP_DEV float sum2(f2 v) {
    const float2 t = two(v);
    return t.x + t.y;
}
template <typename E>
QMLP_DEV void get8(uint32_t at, f2 (&v)[4]) {
    const uint4 a = lds16(at);
    if constexpr (sizeof(E) == 4) {
        const uint4 b = lds16(at + 512);
        v[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y)), v[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        v[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y)), v[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<E, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[i] = pair(f.x, f.y);
            } else {
                v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            }
        }
    }
}
QMLP_DEV void put8(uint32_t at, const float (&v)[8]) {
    sts16(at, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    sts16(at + 512, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
}

// A chunk's pieces of 16 bytes a thread: of the weights A and B, and of a row's arrays.
template <typename R, int G, bool BWD>
struct Layout {
    static constexpr int r = sizeof(R) / 2, gate = 1, dy = gate + (G != kScalar), res = dy + BWD, dh = res + r;
    static constexpr int row = dh + (BWD ? r : 0);
    static constexpr int weights(int nc) { return 4 * nc; }
    static constexpr int stage(int nc, int rp) { return row * nc * rp; }
};

// What a thread knows of its group's rows.
template <typename T, typename R, int NC, int RP, int G, bool BWD>
struct Walk {
    using L = Layout<R, G, BWD>;
    const NormArgs& a;
    int tg, rg, tid, K, shift;  // shift: values that a row starts behind a border of eight
    uint32_t w0, s0, sstage;    // weights; stages: this thread's places, a stage's bytes
    bool ok[NC], all[NC];       // the chunk has columns of the row; eight of them
    bool hz, hr, hd, full;
    QMLP_DEV Walk(const NormArgs& a_, uint8_t* dyn, int tg_) : a(a_), tg(tg_) {
        rg = threadIdx.x / tg;
        tid = threadIdx.x % tg;
        K = a.K;
        shift = (int)(((long)blockIdx.x * (blockDim.x / tg) + rg) * K % 8);
        const bool shared = K % 8 == 0;  // the groups' columns lie alike: one copy of the weights
        const uint32_t wn = shared ? tg : blockDim.x;
        const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        w0 = smem_u32(dyn) + (shared ? tid >> 5 : warp) * (L::weights(NC) * 512) + lane * 16;
        sstage = blockDim.x * (L::stage(NC, RP) * 16);
        s0 = smem_u32(dyn) + wn * (L::weights(NC) * 16) + warp * (L::stage(NC, RP) * 512) + lane * 16;
#pragma unroll
        for (int i = 0; i < NC; ++i) ok[i] = col(i) < K, all[i] = col(i) >= 0 && col(i) + 8 <= K;
        hz = G != kAny || a.z;
        hr = G != kAny || a.r;
        hd = BWD && a.dh;
        full = G == kFull || (G == kAny && a.gate_kind == kGateFull);
    }
    QMLP_DEV int col(int i) const { return (i * tg + tid) * 8 - shift; }  // first column of chunk i
    QMLP_DEV float weight1(const void* w, int c) const {
        return a.w_f32 ? static_cast<const float*>(w)[c] : (float)static_cast<const T*>(w)[c];
    }
    // A and B, zeros past the row's ends
    QMLP_DEV void fetch_weights() const {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!ok[i]) continue;
            float A[8], B[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col(i) + e;
                const bool in = c >= 0 && c < K;
                A[e] = in ? a.scale : 0.0f;
                if (in && a.post_w) A[e] *= weight1(a.post_w, c) + a.offset;
                if (in && a.gate_kind == kGateChannel) A[e] *= weight1(a.gate, c);
                B[e] = in && a.pre_w ? weight1(a.pre_w, c) + a.offset : 0.0f;
            }
            put8(w0 + (i * 4) * 512, A);
            put8(w0 + (i * 4 + 2) * 512, B);
        }
    }
    QMLP_DEV void getA(int i, f2 (&v)[4]) const { get8<float>(w0 + (i * 4) * 512, v); }
    QMLP_DEV void getB(int i, f2 (&v)[4]) const { get8<float>(w0 + (i * 4 + 2) * 512, v); }
    static constexpr uint32_t place(int p, int i, int piece) { return ((p * NC + i) * L::row + piece) * 512; }
    // The stream's chunk of a row at p: fp32 comes as the warp's 1024 bytes in a row (a
    // thread's two halves of its own 32 are half sectors both).
    QMLP_DEV void fetch_r(const void* p, size_t row, int i, uint32_t dst, bool in) const {
        const R* src = static_cast<const R*>(p) + row;
        if constexpr (sizeof(R) == 4) {
            const int lane = threadIdx.x & 31, c0 = col(i) - lane * 8 + lane * 4;
            dst += (lane & 1) * 512 - lane * 16 + (lane >> 1) * 16;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = c0 + 128 * j;
                const bool some = in && c < K;  // (else the second half of the row's last chunk)
                if (c - 4 * (lane & 1) < K) cp16(dst + 256 * j, some ? src + c : src, some ? min(16, (K - c) * 4) : 0);
            }
        } else if (ok[i]) {
            cp16(dst, in ? src + col(i) : src, in ? min(16, (K - col(i)) * 2) : 0);
        }
    }
    // rows m, m + hop, ...: RP of them into stage st; zeros behind a row's end and for rows
    // behind the last one
    QMLP_DEV void fetch_rows(long m, long hop, int st) const {
        const uint32_t s = s0 + sstage * (uint32_t)st;
#pragma unroll
        for (int p = 0; p < RP; ++p, m += hop) {
            const bool in = m < a.M;
            if (p == 0 && !in) break;
            const size_t row = in ? (size_t)m * K : 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint32_t d = s + place(p, i, 0);
                if (in && !QMLP_INB(row + K - 1, a.elems, BWD ? 86 : 85)) continue;
                if (hr) fetch_r(a.r, row, i, d + L::res * 512, in);
                if (hd) fetch_r(a.dh, row, i, d + L::dh * 512, in);
                if (!ok[i]) continue;
                const int n = in ? min(16, (K - col(i)) * 2) : 0;
                const size_t at = in ? row + col(i) : 0;
                if (hz) cp16(d, static_cast<const T*>(a.z) + at, n);
                if (full) cp16(d + L::gate * 512, static_cast<const T*>(a.gate) + at, n);
                if (BWD && (G != kAny || a.dy)) cp16(d + L::dy * 512, static_cast<const T*>(a.dy) + at, n);
            }
        }
        cp_commit();
    }
    // the stage's rows are there; what the first chunk holds of the row before becomes zeros
    QMLP_DEV uint32_t arrived(int st, int S) const {
        cp_wait_but(S - 1);
        __syncwarp();
        const uint32_t s = s0 + sstage * (uint32_t)st;
        if (tid == 0 && shift) {
#pragma unroll 1
            for (int p = 0; p < RP; ++p)
#pragma unroll 1
                for (int j = 0; j < L::row; ++j) {
                    const bool wide = sizeof(R) == 4 && (j >= L::res);
                    const uint32_t d = s + (p * NC * L::row + j) * 512;
                    const int n = wide ? min(max(shift - 4 * ((j - L::res) & 1), 0), 4) * 2 : shift;
#pragma unroll 1
                    for (int e = 0; e < n; ++e) asm volatile("st.shared.u16 [%0], %1;" ::"r"(d + 2 * e), "h"((short)0) : "memory");
                }
        }
        return s;
    }
    template <typename E>
    QMLP_DEV void get(uint32_t s, int p, int i, int piece, f2 (&v)[4]) const {
        get8<E>(s + place(p, i, piece), v);
    }
    template <typename E>
    QMLP_DEV void store(void* p, size_t row, int i, const f2 (&x)[4]) const {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = two(x[e]);
            v[2 * e] = t.x, v[2 * e + 1] = t.y;
        }
        E* dst = static_cast<E*>(p) + row + col(i);
        if (all[i]) {
            stv<E, 8>(dst, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col(i) + e >= 0 && col(i) + e < K) put(dst + e, v[e]);
        }
    }
};

template <typename T, typename R, int NC, int RP, int G>
__global__ void __launch_bounds__(kForwardThreads) norm_forward_rows_kernel(const NormArgs a, int tg, int S) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float buf[2][192];
    const Walk<T, R, NC, RP, G, false> k(a, dyn, tg);
    using L = typename decltype(k)::L;
    const bool post = G != kAny || a.post_w, pre = G != kAny || a.pre_w;
    const int groups = blockDim.x / tg;
    const long hop = (long)gridDim.x * groups, first = (long)blockIdx.x * groups + k.rg;
    for (int i = 0; i + 1 < S; ++i) k.fetch_rows(first + i * RP * hop, hop, i);
    k.fetch_weights();
    int st = 0, turn = 0;
    for (long m = first; m < a.M; m += RP * hop) {
        k.fetch_rows(m + (S - 1) * RP * hop, hop, st ? st - 1 : S - 1);
        float gt[RP];
        bool row[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p) {
            row[p] = p == 0 || m + p * hop < a.M;
            gt[p] = a.gate_kind == kGateToken && row[p] ? (float)static_cast<const T*>(a.gate)[m + p * hop] : 1.0f;
        }
        const uint32_t s = k.arrived(st, S);
        f2 h[RP][NC][4], sq[RP];
        float ss[RP], rz[RP], rh[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p) sq[p] = both(0.0f), rz[p] = rh[p] = 1.0f;
        if (post) {
#pragma unroll
            for (int p = 0; p < RP; ++p) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (k.ok[i]) {
                        f2 v[4];
                        k.template get<T>(s, p, i, 0, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) sq[p] = fma2(v[e], v[e], sq[p]);
                    }
                ss[p] = sum2(sq[p]);
            }
            group_sum<RP>(ss, buf, turn, tg, k.rg);
#pragma unroll
            for (int p = 0; p < RP; ++p) rz[p] = rsqrtf(ss[p] * a.rK + a.eps), sq[p] = both(0.0f);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!k.ok[i]) continue;
            f2 A[4];
            if (k.hz) k.getA(i, A);
#pragma unroll
            for (int p = 0; p < RP; ++p) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[p][i][e] = both(0.0f);
                if (k.hr) k.template get<R>(s, p, i, L::res, h[p][i]);
                if (k.hz) {
                    f2 v[4];
                    const f2 f = both(rz[p] * gt[p]);
                    k.template get<T>(s, p, i, 0, v);
                    if (k.full) {
                        f2 g[4];
                        k.template get<T>(s, p, i, L::gate, g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], g[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[p][i][e] = fma2(mul2(v[e], f), A[e], h[p][i][e]);
                }
                if (a.h && row[p]) k.template store<R>(a.h, (size_t)(m + p * hop) * a.K, i, h[p][i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) sq[p] = fma2(h[p][i][e], h[p][i][e], sq[p]);
            }
        }
        if (pre) {
#pragma unroll
            for (int p = 0; p < RP; ++p) ss[p] = sum2(sq[p]);
            group_sum<RP>(ss, buf, turn, tg, k.rg);
#pragma unroll
            for (int p = 0; p < RP; ++p) rh[p] = rsqrtf(ss[p] * a.rK + a.eps);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (!k.ok[i]) continue;
                f2 B[4];
                k.getB(i, B);
#pragma unroll
                for (int p = 0; p < RP; ++p) {
                    f2 v[4];
                    const f2 f = both(rh[p]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(h[p][i][e], f), B[e]);
                    if (row[p]) k.template store<T>(a.y, (size_t)(m + p * hop) * a.K, i, v);
                }
            }
        }
        if (a.stats && k.tid == 0)
#pragma unroll
            for (int p = 0; p < RP; ++p)
                if (row[p]) a.stats[m + p * hop] = make_float2(rz[p], rh[p]);
        st = st + 1 < S ? st + 1 : 0;
        __syncwarp();
    }
    cp_wait<0>();
}

template <typename T, typename R, int NC, int RP, int G>
__global__ void __launch_bounds__(NC == 1 && RP == 1 ? 640 : 512) norm_backward_rows_kernel(const NormArgs a, int tg, int S) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float buf[2][192];
    const Walk<T, R, NC, RP, G, true> k(a, dyn, tg);
    using L = typename decltype(k)::L;
    const bool post = G != kAny || a.post_w, pre = G != kAny || a.pre_w, token = a.gate_kind == kGateToken;
    const int groups = blockDim.x / tg, K = a.K;
    const long hop = (long)gridDim.x * groups, first = (long)blockIdx.x * groups + k.rg;
    pdl_launch_dependents();  // (the columns' kernel: it waits for this one's end)
    for (int i = 0; i + 1 < S; ++i) k.fetch_rows(first + i * RP * hop, hop, i);
    k.fetch_weights();
    f2 D[NC][4], P[NC][4];  // columns' sums of t dH zh (times an element's gate) and of dy hh
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) D[i][e] = P[i][e] = both(0.0f);
    int st = 0, turn = 0;
    for (long m = first; m < a.M; m += RP * hop) {
        k.fetch_rows(m + (S - 1) * RP * hop, hop, st ? st - 1 : S - 1);
        float gt[RP], rz[RP], rh[RP];
        bool row[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p) {
            row[p] = p == 0 || m + p * hop < a.M;
            const float2 f = row[p] ? __ldg(a.stats + m + p * hop) : make_float2(0.0f, 0.0f);
            rz[p] = post ? f.x : 1.0f, rh[p] = f.y;
            gt[p] = token && row[p] ? (float)static_cast<const T*>(a.gate)[m + p * hop] : 1.0f;
        }
        const uint32_t s = k.arrived(st, S);
        f2 x[RP][NC][4], y[RP][NC][4], c2[3 * RP];  // hh; dh + dy B / rms
        float c[3 * RP];
#pragma unroll
        for (int j = 0; j < 3 * RP; ++j) c2[j] = both(0.0f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!k.ok[i]) continue;
            f2 A[4], B[4];
            if (k.hz) k.getA(i, A);
            if (pre) k.getB(i, B);
#pragma unroll
            for (int p = 0; p < RP; ++p) {
                f2 q[4], v[4];
                if (k.hz) {
                    const f2 f = both(rz[p]);
                    k.template get<T>(s, p, i, 0, q);
                    if (k.full) {
                        k.template get<T>(s, p, i, L::gate, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) q[e] = mul2(q[e], v[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = mul2(mul2(q[e], f), A[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) y[p][i][e] = both(0.0f);
                if (k.hd) k.template get<R>(s, p, i, L::dh, y[p][i]);
                if (pre) {
                    f2 (&h)[4] = x[p][i];
                    const f2 g = both(gt[p]), f = both(rh[p]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = both(0.0f);
                    if (k.hr) k.template get<R>(s, p, i, L::res, h);
                    if (k.hz)
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = fma2(g, q[e], h[e]);
                    k.template get<T>(s, p, i, L::dy, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[e] = mul2(h[e], f);
                        P[i][e] = fma2(v[e], h[e], P[i][e]);
                        v[e] = mul2(v[e], B[e]);
                        c2[3 * p] = fma2(v[e], h[e], c2[3 * p]);
                        y[p][i][e] = fma2(v[e], f, y[p][i][e]);
                        if (k.hz) c2[3 * p + 2] = fma2(h[e], q[e], c2[3 * p + 2]);
                    }
                }
                if (k.hz)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c2[3 * p + 1] = fma2(y[p][i][e], q[e], c2[3 * p + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < 3 * RP; ++j) c[j] = sum2(c2[j]);
        group_sum<3 * RP>(c, buf, turn, tg, k.rg);
        float mr[RP], back[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p) {
            mr[p] = rh[p] * c[3 * p] * a.rK;                       // mean / rms
            const float dhq = c[3 * p + 1] - mr[p] * c[3 * p + 2];  // sum of dH q
            back[p] = post ? rz[p] * gt[p] * dhq * a.rK : 0.0f;
            if (token && a.dgate && k.tid == 0 && row[p]) put(static_cast<T*>(a.dgate) + m + p * hop, dhq);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!k.ok[i]) continue;
            f2 A[4];
            if (k.hz) k.getA(i, A);
#pragma unroll
            for (int p = 0; p < RP; ++p) {
                f2 (&d)[4] = y[p][i];
                const size_t at = (size_t)(m + p * hop) * K;
                if (pre) {
                    const f2 f = both(-mr[p]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = fma2(x[p][i][e], f, d[e]);
                }
                if (a.dr && row[p]) k.template store<R>(a.dr, at, i, d);
                if (!k.hz) continue;
                f2 z[4], t[4];
                k.template get<T>(s, p, i, 0, z);
                const f2 f = both(rz[p] * gt[p]), zb = both(-rz[p] * back[p]), r = both(rz[p]);
                if (k.full) {
                    if (a.dgate && row[p]) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[e] = mul2(d[e], mul2(mul2(z[e], r), A[e]));
                        k.template store<T>(a.dgate, at, i, t);
                    }
                    k.template get<T>(s, p, i, L::gate, t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = mul2(d[e], t[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    D[i][e] = fma2(d[e], mul2(z[e], f), D[i][e]);
                    t[e] = fma2(mul2(d[e], A[e]), f, mul2(z[e], zb));
                }
                if (a.dz && row[p]) k.template store<T>(a.dz, at, i, t);
            }
        }
        st = st + 1 < S ? st + 1 : 0;
        __syncwarp();
    }
    cp_wait<0>();
    if (!a.part) return;
    // this CTA's sums over its rows, group after group: [3][K]
    float* part = a.part + (size_t)blockIdx.x * 3 * K;
    float* sum = reinterpret_cast<float*>(dyn);
    const bool channel = a.gate_kind == kGateChannel;
    __syncthreads();  // every group is through with the rows' places
    for (int g = 0; g < groups; ++g) {
        if (k.rg == g)
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = k.col(i) + e;
                    if (c < 0 || c >= K) continue;
                    const float gate = channel ? k.weight1(a.gate, c) : 1.0f;
                    const float w = channel && a.post_w ? k.weight1(a.post_w, c) + a.offset : 1.0f;
                    const float2 d2 = two(D[i][e >> 1]), p2 = two(P[i][e >> 1]);
                    const float dv = e & 1 ? d2.y : d2.x, pv = e & 1 ? p2.y : p2.x;
                    sum[c] = (g ? sum[c] : 0.0f) + a.scale * gate * dv;
                    sum[K + c] = (g ? sum[K + c] : 0.0f) + pv;
                    if (channel) sum[2 * K + c] = (g ? sum[2 * K + c] : 0.0f) + a.scale * w * dv;
                }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < (channel ? 3 : 2) * K; i += blockDim.x)
        if (QMLP_INB((size_t)blockIdx.x * 3 * K + i, a.part_elems, 83)) part[i] = sum[i];
}

// The columns' sums over the CTAs' shares, in their order: 32 columns a CTA, sixteen
// warps each every sixteenth share.
constexpr int kColumnWarps = 16;
template <typename T>
__global__ void __launch_bounds__(kColumnWarps * 32) norm_columns_kernel(const NormArgs a, int shares) {
    __shared__ float sum[kColumnWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
    void* dst = j == 0 ? a.dpost : j == 1 ? a.dpre : a.gate_kind == kGateChannel ? a.dgate : nullptr;
    if (!dst) return;
    pdl_wait();  // the shares are written
    float s = 0.0f;
#pragma unroll 10
    for (int i = warp; i < shares; i += kColumnWarps) {
        const size_t at = ((size_t)i * 3 + j) * a.K + c;
        if (c < a.K && QMLP_INB(at, a.part_elems, 84)) s += a.part[at];
    }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.K) {
        for (int w = 1; w < kColumnWarps; ++w) s += sum[w][lane];
        if (a.w_f32) static_cast<float*>(dst)[c] = s;
        else put(static_cast<T*>(dst) + c, s);
    }
}
template <typename T>
cudaError_t launch_columns(const NormArgs& a, int shares, cudaStream_t s) {
    if (!a.part) return cudaSuccess;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.K + 31) / 32), 3);
    cfg.blockDim = dim3(kColumnWarps * 32);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_columns_kernel<T>, a, shares);
}

template <typename T, typename R, int V, int NC, bool WARP, bool TIGHT = false>
cudaError_t launch_forward(const NormArgs& a, int threads, cudaStream_t s) {
    const unsigned grid = (unsigned)(WARP ? (a.M + kWarps - 1) / kWarps : a.M);
    norm_forward_kernel<T, R, V, NC, WARP, TIGHT><<<grid, WARP ? kWarps * 32 : threads, 0, s>>>(a);
    return cudaPeekAtLastError();
}
template <typename T, typename R, int V, int NC, bool WARP>
cudaError_t launch_backward(const NormArgs& a, int threads, cudaStream_t s) {
    const int per = WARP ? kWarps : 1;
    const int grid = (int)std::min<long>((a.M + per - 1) / per, a.shares);
    norm_backward_kernel<T, R, V, NC, WARP>
        <<<grid, WARP ? kWarps * 32 : threads, WARP ? 3 * a.K * sizeof(float) : 0, s>>>(a);
    const cudaError_t e = cudaPeekAtLastError();
    return e != cudaSuccess ? e : launch_columns<T>(a, grid, s);
}

constexpr int kRowsSmem = 212 * 1024;  // of the kernels that walk over rows (beside the sums' buffer)
// Chunks of eight that a row of K values lies in at most.
int rows_chunks(int K) { return K % 8 ? (K + 14) / 8 : K / 8; }
// Threads of a group, groups of a CTA, CTAs, stages.
struct RowsPlan {
    int tg, groups, grid, S;
    size_t smem;
};
template <typename R, int NC, int RP, int G, bool BWD>
bool rows_plan(const NormArgs& a, RowsPlan& p) {
    using L = Layout<R, G, BWD>;
    const int K = a.K, most = !BWD ? kForwardThreads : NC == 1 && RP == 1 ? 640 : 512;
    p.tg = ((rows_chunks(K) + NC - 1) / NC + 31) / 32 * 32;
    if (p.tg > most) return false;
    auto smem = [&](int groups, int S) {
        const int n = p.tg * groups, wn = K % 8 == 0 ? p.tg : n;
        return std::max((size_t)16 * (wn * L::weights(NC) + (size_t)n * S * L::stage(NC, RP)), (size_t)(BWD ? 12 * K : 0));
    };
    p.groups = most / p.tg;
    while (p.groups > 1 && (smem(p.groups, 2) > kRowsSmem || a.M < (long)p.groups * RP * a.num_sms)) --p.groups;
    p.S = 4;
    while (p.S > 2 && smem(p.groups, p.S) > kRowsSmem) --p.S;
    p.smem = smem(p.groups, p.S);
    p.grid = (int)std::min<long>((a.M + p.groups - 1) / p.groups, a.num_sms);
    // a group's rows are a multiple of eight apart where K is no multiple of eight
    if (K % 8) p.grid = std::max(8, (p.grid + 7) / 8 * 8 <= a.num_sms ? (p.grid + 7) / 8 * 8 : p.grid / 8 * 8);
    return p.smem <= kRowsSmem;
}
template <typename T, typename R, int NC, int RP, int G, bool BWD>
bool rows_try(const NormArgs& a, cudaStream_t s, cudaError_t& e) {
    RowsPlan p;
    if (!rows_plan<R, NC, RP, G, BWD>(a, p)) return false;
    static unsigned long done = 0;
    if constexpr (!BWD) {
        auto* kernel = norm_forward_rows_kernel<T, R, NC, RP, G>;
        if ((e = smem_once(kernel, kRowsSmem, done)) != cudaSuccess) return true;
        kernel<<<p.grid, p.tg * p.groups, p.smem, s>>>(a, p.tg, p.S);
        e = cudaPeekAtLastError();
    } else {
        auto* kernel = norm_backward_rows_kernel<T, R, NC, RP, G>;
        if ((e = smem_once(kernel, kRowsSmem, done)) != cudaSuccess) return true;
        kernel<<<p.grid, p.tg * p.groups, p.smem, s>>>(a, p.tg, p.S);
        if ((e = cudaPeekAtLastError()) == cudaSuccess) e = launch_columns<T>(a, p.grid, s);
    }
    return true;
}
// The first form that fits: two rows at a time (16384 x 1024, backward 58 us, one 64; 4096
// x 4096 with an element's gate 63 and 81), one, sixteen values a thread.
template <typename T, typename R, int G, bool BWD>
bool rows_g(const NormArgs& a, cudaStream_t s, cudaError_t& e) {
    if constexpr (G != kAny) {
        if (a.M >= 2L * a.num_sms && rows_try<T, R, 1, 2, G, BWD>(a, s, e)) return true;
        if (rows_try<T, R, 1, 1, G, BWD>(a, s, e)) return true;
    }
    return rows_try<T, R, 2, 1, G, BWD>(a, s, e);
}
template <typename T, typename R, bool BWD>
bool launch_rows(const NormArgs& a, cudaStream_t s, cudaError_t& e) {
    if (!(a.z && a.r && a.post_w && a.pre_w)) return rows_g<T, R, kAny, BWD>(a, s, e);
    return a.gate_kind == kGateFull ? rows_g<T, R, kFull, BWD>(a, s, e) : rows_g<T, R, kScalar, BWD>(a, s, e);
}

// Backward, the kernels that walk over rows wherever they fit. Forward a row a CTA (up to
// 256 columns: a warp), which hides a row's latencies behind other rows'. From four rows an
// SM on it may take 32 registers, so that an SM is full of threads (8192 x 5120 with an fp32
// stream 84 us, 95 with the 42 it would like, 102 walking; 8192 x 4096 64 to 81; with fewer
// rows the spilled ones show, 512 x 5120 8.1 to 8.8). Walking is ahead for very many long
// rows of a 16-bit stream (8192 x 5120 66 us to 70; 8192 x 2048 28 both, 4096 x 4096 32 to 29.5),
// a warp a row is behind from 512 columns on (16384 x 512 17.5 us to 15.2, 2048 x 1024 8.8 to
// 5.8). Rows of no multiple of eight values have the walks, or a value at a time (301 x
// 2571 7.5 to 9.8 us, backward 16 to 25; 4096 x 3333 30 to 48 and 61 to 198).
template <typename T, typename R>
cudaError_t launch_tr(const NormArgs& a, bool backward, cudaStream_t s) {
    const int K = a.K;
    auto up = [](int n) { return (n + 31) / 32 * 32; };
    cudaError_t e = cudaSuccess;
    if (backward) {
        if (a.vec && launch_rows<T, R, true>(a, s, e)) return e;
        if (a.vec && K % 8 == 0) return launch_backward<T, R, 8, 2, false>(a, up((K / 8 + 1) / 2), s);
        if (K <= 256) return launch_backward<T, R, 1, 8, true>(a, 0, s);
        if (K <= 8192) return launch_backward<T, R, 1, 8, false>(a, up((K + 7) / 8), s);
        return launch_backward<T, R, 1, 16, false>(a, up((K + 15) / 16), s);
    }
    const bool walk = K % 8 || (sizeof(R) == 2 && K > 4096 && a.M >= 32L * a.num_sms);
    if (a.vec && walk && launch_rows<T, R, false>(a, s, e)) return e;
    if (a.vec && K % 8 == 0) {
        if (K <= 256) return launch_forward<T, R, 8, 1, true>(a, 0, s);
        if (K <= 8192)
            return a.M >= 4L * a.num_sms ? launch_forward<T, R, 8, 1, false, true>(a, up(K / 8), s)
                                         : launch_forward<T, R, 8, 1, false>(a, up(K / 8), s);
        return launch_forward<T, R, 8, 2, false>(a, up((K / 8 + 1) / 2), s);
    }
    if (K <= 256) return launch_forward<T, R, 1, 8, true>(a, 0, s);
    if (K <= 8192) return launch_forward<T, R, 1, 8, false>(a, up((K + 7) / 8), s);
    return launch_forward<T, R, 1, 16, false>(a, up((K + 15) / 16), s);
}

}  // namespace
}  // namespace qmlp
