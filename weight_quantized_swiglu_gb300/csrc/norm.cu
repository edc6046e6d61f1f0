// norm.cu -- the norms before and after a block, fused with its gate, residual
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
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kWarps = 8;  // rows (warps) of a CTA where a warp takes a row

template <typename T, int V>
QMLP_DEV void ldv(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = (float)*p;
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i);
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        }
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
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
QMLP_DEV void put(float* p, float v) { *p = v; }
QMLP_DEV void put(__half* p, float v) { *p = __float2half_rn(v); }
QMLP_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <typename T, int V>
QMLP_DEV void stv(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        put(p, v[0]);
    } else if constexpr (sizeof(T) == 4) {
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
// The sums of N values over a row's threads, in every thread. ROWS > 1: a warp a
// row; else the CTA, through one of two buffers in turn (`turn` flips), so that
// one barrier a sum is enough.
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

template <typename T, typename R, int V, int NC, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarps * 32 : 1024) norm_forward_kernel(const NormArgs a) {
    __shared__ float buf[2][1][32];
    int turn = 0;
    const long m = WARP ? (long)blockIdx.x * kWarps + (threadIdx.x >> 5) : (long)blockIdx.x;
    if (m >= a.M) return;  // (WARP: no barrier follows)
    const int K = a.K;
    const size_t at = (size_t)m * K;
    const T* z = static_cast<const T*>(a.z) + at;
    const R* r = static_cast<const R*>(a.r) + at;
    float h[NC][V], zv[NC][V];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = column<V, WARP>(i);
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] = zv[i][e] = 0.0f;
        if (c < K && QMLP_INB(at + c + V - 1, a.elems, 81)) {
            if (a.z) ldv<T, V>(z + c, zv[i]);
            if (a.r) ldv<R, V>(r + c, h[i]);
        }
    }
    float rz = 1.0f, rh = 1.0f;
    if (a.z) {
        if (a.post_w) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) ss[0] = fmaf(zv[i][e], zv[i][e], ss[0]);
            row_sum<WARP, 1>(ss, buf, turn);
            rz = rsqrtf(ss[0] * a.rK + a.eps);
        }
        const float gt = a.gate_kind == kGateToken ? (float)static_cast<const T*>(a.gate)[m] : 1.0f;
        const float s = a.scale * gt;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column<V, WARP>(i);
            if (c < K) {
                float w[V], g[V];
                if (a.post_w) ldw<T, V>(a.post_w, a.w_f32, c, w);
                if (a.gate_kind == kGateChannel) ldw<T, V>(a.gate, a.w_f32, c, g);
                if (a.gate_kind == kGateFull) ldv<T, V>(static_cast<const T*>(a.gate) + at + c, g);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float n = zv[i][e];
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

// The columns' sums over the CTAs' shares, in their order: 32 columns a CTA, eight
// warps each every eighth share.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormArgs a, int shares) {
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
    void* dst = j == 0 ? a.dpost : j == 1 ? a.dpre : a.gate_kind == kGateChannel ? a.dgate : nullptr;
    if (!dst) return;
    float s = 0.0f;
    if (c < a.K)
        for (int i = warp; i < shares; i += 8) {
            const size_t at = ((size_t)i * 3 + j) * a.K + c;
            if (QMLP_INB(at, a.part_elems, 84)) s += a.part[at];
        }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.K) {
        for (int w = 1; w < 8; ++w) s += sum[w][lane];
        if (a.w_f32) static_cast<float*>(dst)[c] = s;
        else put(static_cast<T*>(dst) + c, s);
    }
}

template <typename T, typename R, int V, int NC, bool WARP>
cudaError_t launch_v(const NormArgs& a, bool backward, int threads, cudaStream_t s) {
    if (!backward) {
        const unsigned grid = (unsigned)(WARP ? (a.M + kWarps - 1) / kWarps : a.M);
        norm_forward_kernel<T, R, V, NC, WARP><<<grid, WARP ? kWarps * 32 : threads, 0, s>>>(a);
        return cudaPeekAtLastError();
    }
    const int per = WARP ? kWarps : 1;
    const int grid = (int)std::min<long>((a.M + per - 1) / per, a.shares);
    norm_backward_kernel<T, R, V, NC, WARP>
        <<<grid, WARP ? kWarps * 32 : threads, WARP ? 3 * a.K * sizeof(float) : 0, s>>>(a);
    cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess || !a.part) return e;
    norm_columns_kernel<T><<<dim3((unsigned)((a.K + 31) / 32), 3), 256, 0, s>>>(a, grid);
    return cudaPeekAtLastError();
}

template <typename T, typename R>
cudaError_t launch_tr(const NormArgs& a, bool backward, cudaStream_t s) {
    const int K = a.K;
    auto up = [](int n) { return (n + 31) / 32 * 32; };
    if (a.vec) {
        const int chunks = K / 8;
        if (K <= 512) return launch_v<T, R, 8, 2, true>(a, backward, 0, s);
        if (K <= 1024) return launch_v<T, R, 8, 4, true>(a, backward, 0, s);
        if (chunks <= 1024) return launch_v<T, R, 8, 1, false>(a, backward, up(chunks), s);
        return launch_v<T, R, 8, 2, false>(a, backward, up((chunks + 1) / 2), s);
    }
    if (K <= 256) return launch_v<T, R, 1, 8, true>(a, backward, 0, s);
    if (K <= 8192) return launch_v<T, R, 1, 8, false>(a, backward, up((K + 7) / 8), s);
    return launch_v<T, R, 1, 16, false>(a, backward, up((K + 15) / 16), s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, bool t_f16, bool r_f32, bool backward, cudaStream_t s) {
    if (t_f16)
        return r_f32 ? launch_tr<__half, float>(a, backward, s) : launch_tr<__half, __half>(a, backward, s);
    return r_f32 ? launch_tr<__nv_bfloat16, float>(a, backward, s)
                 : launch_tr<__nv_bfloat16, __nv_bfloat16>(a, backward, s);
}

QMLP_BOUNDS_UNIT(norm)

}  // namespace qmlp
