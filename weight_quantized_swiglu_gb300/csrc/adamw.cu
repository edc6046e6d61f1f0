// adamw.cu -- one AdamW step over many tensors in one launch.
//
// For every element of every tensor, with the constants of the step computed
// once on the host (in fp64, then fp32):
//   g = gscale grad
//   m = m b1 + g (1 - b1)
//   v = v b2 + g g (1 - b2)
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / ( sqrt(v) / sqrt(1 - b2^t) + eps )
// All of it in fp32, each operation of a state rounded once and none contracted,
// so that a state does not depend on how the compiler fuses a product and a sum;
// the update's root and quotient are the fast ones (a few units of the last
// place of a term of the size of lr). p is
// the fp32 master where there is one (then param = bf16(p) is written beside
// it), else the parameter itself.
//
// 8-bit states: 256 consecutive elements of a tensor are a block with one fp32
// scale. m is held as e4m3 codes times max|m| / 448; v as the codes of its
// square root r times max(r) / 448, which halves the range that the codes have
// to span (r: 2^-9 .. 448 of the scale, v: its square, 35 powers of two). r > 0
// never rounds to the code zero: the quotient m / r of the next step would
// otherwise divide what is left of m by eps. Both are rounded after the step's
// own update has used them unrounded, so a parameter sees each state rounded
// once (the choice: 4 bytes less a state and step in each direction, for a
// relative error of 2^-4 of each state).
//
// One warp takes a block of 256 elements, eight consecutive ones a lane, so a
// block's maximum is one warp reduction. A CTA takes a chunk of 8 blocks; its
// addresses come from one 64-byte entry of a table that is written when the
// handle is made. Bound by memory: fp32 28 B an element (bf16 parameter, fp32
// master, bf16 gradient and 8-bit states: 16 B).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // elements a lane
static_assert(kAdamWBlock == 32 * kPer && kAdamWChunk == kThreads * kPer, "a warp a block, a CTA a chunk");

template <bool VEC>
QMLP_DEV void load8(const float* p, int n, float (&v)[kPer]) {
    if (VEC) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
}
template <bool VEC>
QMLP_DEV void load8(const __nv_bfloat16* p, int n, float (&v)[kPer]) {
    if (VEC) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
}
template <bool VEC>
QMLP_DEV void store8(float* p, int n, const float (&v)[kPer]) {
    if (VEC) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <bool VEC>
QMLP_DEV void store8(__nv_bfloat16* p, int n, const float (&v)[kPer]) {
    if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}

// Eight e4m3 codes times their block's scale.
template <bool VEC>
QMLP_DEV void load8_codes(const uint8_t* p, int n, float s, float (&v)[kPer]) {
    uint32_t w[2] = {0, 0};
    if (VEC) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x, w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[2];
        e4m3x4_to_f16x2x2(w[i], h[0], h[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[4 * i + 2 * j] = __fmul_rn(f.x, s);
            v[4 * i + 2 * j + 1] = __fmul_rn(f.y, s);
        }
    }
}
// Two floats -> two e4m3 codes, nearest (ties to even), a first.
QMLP_DEV uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
QMLP_DEV float sqrt_fast(float v) {  // within 2^-23
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The block's codes of w: w / s, s = max|w| / 448 over the warp (zero: codes
// zero). ROOT: w = sqrt(v), of which the correctly rounded one counts (its
// maximum is the root of v's), and what is above zero keeps at least the
// smallest code.
//
// The quotients are products with the reciprocal, and the roots fast ones: five
// units of the last place off at most. So both ends of that error (2^-20 to each
// side) are made codes, and only where they differ, or a root came to the code
// zero, are root and quotient taken again, correctly rounded. A lane asks that
// once for its eight elements. (69M elements, 384 tensors: 229 us with every
// root and quotient rounded, 203 with the quotients' bits compared to the middles
// of the codes, 190 with the two codes.)
template <bool VEC, bool ROOT>
QMLP_DEV void store8_codes(uint8_t* p, float* scale, int n, const float (&v)[kPer], const float (&w)[kPer]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(v[i]));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // bits order as the floats do
    if (ROOT) top = __fsqrt_rn(top);
    const float s = __fmul_rn(top, 1.0f / 448.0f), rs = __frcp_rn(s);
    const float lo = __fmul_rn(rs, 1.0f - 9.5367431640625e-7f), hi = __fmul_rn(rs, 1.0f + 9.5367431640625e-7f);
    uint32_t c[2], d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        c[i] = e4m3x2(__fmul_rn(w[4 * i], lo), __fmul_rn(w[4 * i + 1], lo)) |
               e4m3x2(__fmul_rn(w[4 * i + 2], lo), __fmul_rn(w[4 * i + 3], lo)) << 16;
        d[i] = e4m3x2(__fmul_rn(w[4 * i], hi), __fmul_rn(w[4 * i + 1], hi)) |
               e4m3x2(__fmul_rn(w[4 * i + 2], hi), __fmul_rn(w[4 * i + 3], hi)) << 16;
    }
    // (under 2^-126 the reciprocal may be infinite: momenta that decay without gradients come there)
    bool again = !(s >= 1.17549435e-38f) || c[0] != d[0] || c[1] != d[1];
    if (ROOT)  // a byte that is zero
        again |= (((c[0] - 0x01010101u) & ~c[0]) | ((c[1] - 0x01010101u) & ~c[1])) & 0x80808080u;
    if (again) {
        float q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float x = ROOT ? __fsqrt_rn(v[i]) : v[i];
            // no scale: zeros (and values under 448 of the smallest subnormal), or a NaN, which stays one
            q[i] = s > 0.0f ? __fdiv_rn(x, s) : x;
            if (ROOT && s > 0.0f && q[i] > 0.0f) q[i] = fmaxf(q[i], 0.001953125f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = e4m3x2(q[4 * i], q[4 * i + 1]) | e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
    }
    if ((threadIdx.x & 31) == 0) *scale = s;
    if (VEC) {
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < n) p[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
    }
}

template <typename P, typename G, bool S8, bool MASTER, bool VEC>
QMLP_DEV void step8(const AdamWChunk& c, const AdamWStep& k, int at, int n) {
    float p[kPer], g[kPer], m[kPer], v[kPer];
    P* param = static_cast<P*>(c.param) + at;
    float* master = MASTER ? c.master + at : nullptr;
    if (MASTER) load8<VEC>(master, n, p);
    else load8<VEC>(param, n, p);
    load8<VEC>(static_cast<const G*>(c.grad) + at, n, g);
    const int blk = at / kAdamWBlock;
    if (S8) {
        load8_codes<VEC>(static_cast<const uint8_t*>(c.m) + at, n, c.m_scale[blk], m);
        load8_codes<VEC>(static_cast<const uint8_t*>(c.v) + at, n, c.v_scale[blk], v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = __fmul_rn(v[i], v[i]);
        __syncwarp();  // every lane has read the block's scales before lane 0 writes the new ones
    } else {
        load8<VEC>(static_cast<const float*>(c.m) + at, n, m);
        load8<VEC>(static_cast<const float*>(c.v) + at, n, v);
    }
    float r[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float gs = __fmul_rn(g[i], k.gscale);
        m[i] = __fadd_rn(__fmul_rn(m[i], k.b1), __fmul_rn(gs, k.omb1));
        v[i] = __fadd_rn(__fmul_rn(v[i], k.b2), __fmul_rn(__fmul_rn(gs, gs), k.omb2));
        r[i] = sqrt_fast(v[i]);
        const float d = __fadd_rn(__fmul_rn(r[i], k.rbc2), k.eps);
        p[i] = __fsub_rn(__fmul_rn(p[i], k.decay), __fmul_rn(__fdividef(m[i], d), k.step));
    }
    if (MASTER) store8<VEC>(master, n, p);
    store8<VEC>(param, n, p);
    if (S8) {
        store8_codes<VEC, false>(static_cast<uint8_t*>(c.m) + at, c.m_scale + blk, n, m, m);
        store8_codes<VEC, true>(static_cast<uint8_t*>(c.v) + at, c.v_scale + blk, n, v, r);
    } else {
        store8<VEC>(static_cast<float*>(c.m) + at, n, m);
        store8<VEC>(static_cast<float*>(c.v) + at, n, v);
    }
}

// `bytes` (a multiple of 16) from p on their way to L2; only from a 16-byte
// boundary, as the copy wants it (8-bit states may start on 8).
QMLP_DEV void to_l2(const void* p, uint32_t bytes) {
    if (bytes && !(reinterpret_cast<uintptr_t>(p) & 15))
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

constexpr int kResident = 5;  // CTAs an SM

// Five CTAs an SM (8-bit states, with the middles compared: 212 us with four, 202
// with five, 209 with six; the next chunk's words prefetched into registers: 243
// and more). 8-bit states: a chunk is half the bytes of fp32's behind the same
// two latencies, the table's entry and then the data, so one thread sends the
// data of the chunk `ahead`, half of the GPU's resident CTAs on, to L2. (69M
// elements, 384 tensors: 186 us without; 188 with half a CTA an SM ahead, 179 with
// one and a half, 175 with two and a half, 174 with three, 177 with five, 178 with
// ten. fp32 states, 150M elements: 591 without and with two and a half, 610 with
// five, 781 with ten: they do without.)
template <typename P, typename G, bool S8, bool MASTER>
__global__ void __launch_bounds__(kThreads, kResident)
    adamw_kernel(const AdamWChunk* __restrict__ chunks, const AdamWStep k, const unsigned ahead) {
    const AdamWChunk c = chunks[blockIdx.x];
    if (S8 && threadIdx.x == 0 && blockIdx.x + ahead < gridDim.x) {
        const AdamWChunk& f = chunks[blockIdx.x + ahead];
        if (f.vec && QMLP_INB(f.n - 1, kAdamWChunk, 71)) {
            const uint32_t n = (uint32_t)f.n & ~15u;  // whole 16 bytes of every type
            if (MASTER) to_l2(f.master, n * 4);
            else to_l2(f.param, n * (uint32_t)sizeof(P));
            to_l2(f.grad, n * (uint32_t)sizeof(G));
            to_l2(f.m, n);
            to_l2(f.v, n);
        }
    }
    if (!QMLP_INB(c.n - 1, kAdamWChunk, 71)) return;
    const int at = threadIdx.x * kPer;  // within the chunk
    if ((at & ~(kAdamWBlock - 1)) >= c.n) return;  // the whole warp's block is past the end
    const int n = min(max(c.n - at, 0), kPer);     // elements of this lane
    // whole blocks of aligned tensors take the wide loads; the choice is the warp's
    if (c.vec && (at | (kAdamWBlock - 1)) < c.n) step8<P, G, S8, MASTER, true>(c, k, at, n);
    else step8<P, G, S8, MASTER, false>(c, k, at, n);
}

template <typename P, typename G, bool MASTER>
cudaError_t launch_s(const AdamWChunk* chunks, long count, bool s8, const AdamWStep& k, unsigned ahead,
                     cudaStream_t s) {
    if (s8) adamw_kernel<P, G, true, MASTER><<<(unsigned)count, kThreads, 0, s>>>(chunks, k, ahead);
    else adamw_kernel<P, G, false, MASTER><<<(unsigned)count, kThreads, 0, s>>>(chunks, k, ahead);
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamWChunk* chunks, long count, bool param_bf16, bool master, bool grad_bf16, bool s8,
                         const AdamWStep& k, int num_sms, cudaStream_t s) {
    const unsigned ahead = (unsigned)(kResident * std::max(num_sms, 1) / 2);
    if (count < 1 || count > 0x7fffffffL) return cudaErrorInvalidValue;
    using B = __nv_bfloat16;
    if (!param_bf16)
        return grad_bf16 ? launch_s<float, B, false>(chunks, count, s8, k, ahead, s)
                         : launch_s<float, float, false>(chunks, count, s8, k, ahead, s);
    if (master)
        return grad_bf16 ? launch_s<B, B, true>(chunks, count, s8, k, ahead, s)
                         : launch_s<B, float, true>(chunks, count, s8, k, ahead, s);
    return grad_bf16 ? launch_s<B, B, false>(chunks, count, s8, k, ahead, s)
                     : launch_s<B, float, false>(chunks, count, s8, k, ahead, s);
}

QMLP_BOUNDS_UNIT(adamw)

}  // namespace qmlp
