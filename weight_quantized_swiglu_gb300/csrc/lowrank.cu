// lowrank.cu -- the products of low-rank adapters: z A^T (wide in, r out),
// v B^T (r in, wide out) and z^T v (over the tokens), r <= 64.
//
// Notation: an adapter of a projection W [N, D] is A [r, D], B [N, r] and a
// factor c; it adds c B (A z) to W z. All inputs are bf16 and every sum is
// fp32. v = c A z is kept in three bf16 words, each the rounding of what the
// ones before it leave, so that the second product sees v as fp32 holds it, at
// the price of two more MMAs of a product that is bound by memory. (With two
// words, 2^-17 of v: the block's output differed from the 64-bit one, both in
// bf16, by 5e-4 where the adapters' terms are as large as the block's; 2e-4
// with three, as without adapters.)
//
// Ranks are padded to Rp = 16, 32 or 64 with zeros (the packed copies of a
// handle), tokens are taken in tiles of 64 of one adapter: for calls of many
// requests a plan kernel groups the tokens by adapter (perm, tiles); with one
// adapter a tile is 64 consecutive tokens. Every row of a tile is summed on
// its own and in an order that depends on the sizes alone, so a token's result
// does not depend on the tokens beside it.
//
// Bound by memory: z (or the wide output) passes once; the MMAs (mma.sync
// m16n8k16) are below the tensor cores' rate at these ranks, but for the wide
// products at rank 64, whose three words are 47 GFLOP for 3001 tokens of the
// 27B-class block. Measured there (K 5120, I 17408):
//   c A x, 8192 tokens, 32 columns: 25 us (84 MB); c dG B, 2 x 16 columns: 102 us
//   (570 MB, 5.6 TB/s)
//   B v as an fp32 array, 8192 tokens, rank 16: 240 us (1.14 GB, 4.8 TB/s); 3001
//   tokens, rank 64: 128 us (the MMAs) -- hence the further GEMM steps, for which
//   the image and the plan kernels below make the operands
//   all six gradients, 8192 tokens, rank 16: 193 us (1.02 GB, 5.3 TB/s)
#include "lowrank.cuh"

namespace qmlp {
namespace {

constexpr int kT = kLrTile;    // tokens of a tile
constexpr int kThr = 128;      // 4 warps, 16 tokens each
constexpr int kStep = 64;      // contraction length of a step
constexpr int kPlanTable = 128;  // groups that the plan counts warp by warp
constexpr int kLrMaxEnts = 256;  // 256-token tiles of the plan: 65536 tokens

QMLP_DEV void cp16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
QMLP_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QMLP_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

QMLP_DEV void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
QMLP_DEV void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
QMLP_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row `row` in a tile of rows of CPR chunks
// (CPR 2, 4, 8 or 16), swizzled so that eight rows at one c, or eight chunks
// of a row, fall into different banks.
template <int CPR>
QMLP_DEV uint32_t sw(int row, int c) {
    const int x = CPR >= 8 ? row & 7 : CPR == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
    return (uint32_t)((row * CPR + (c ^ x)) * 16);
}

// The B fragments (two n8 tiles, one k16) of columns n0..n0+15, contraction
// k0..k0+15 of a tile in shared memory: rows of k (TRANS: [k][n]) or of n.
template <bool TRANS, int CPR>
QMLP_DEV void load_b(uint32_t base, int n0, int k0, int lane, uint32_t (&b)[4]) {
    const int q = lane >> 3, r = lane & 7;
    if (TRANS) ldsm4t(b, base + sw<CPR>(k0 + (q & 1) * 8 + r, (n0 >> 3) + (q >> 1)));
    else ldsm4(b, base + sw<CPR>(n0 + (q >> 1) * 8 + r, (k0 >> 3) + (q & 1)));
}

// v as NW bf16 words, the largest first.
template <int NW>
QMLP_DEV void split_bf16(float v, __nv_bfloat16 (&w)[NW]) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        w[i] = __float2bfloat16_rn(v);
        v -= __bfloat162float(w[i]);
    }
}

// The tile of this CTA: slot, first position, tokens. False: no such tile.
QMLP_DEV bool tile_of(const LrTokens& t, int i, int& slot, int& pos0, int& n, int& entry0) {
    entry0 = 0;
    if (!t.tiles) {
        slot = 0;
        pos0 = i * kT;
        n = min(kT, t.M - pos0);
        return n > 0;
    }
    if (i >= *t.n_tiles) return false;
    const int4 e = t.tiles[i];
    if (!QMLP_INB(e.x + 1, t.slots + 1, 61) || !QMLP_INB(e.z - 1, kT, 61) || !QMLP_INB(e.y, t.M - e.z + 1, 61))
        return false;
    slot = e.x;
    pos0 = e.y;
    n = e.z;
    entry0 = e.w;
    return true;
}

// The token at a position (index checks: `bad` for one that does not exist).
QMLP_DEV int token_at(const LrTokens& t, int pos, int bad) {
    const int tok = t.perm ? t.perm[pos] : pos;
    return QMLP_INB(tok, t.M, 62) ? tok : bad;
}

// The CTAs of a cluster (along y) hold partial sums of one tile in their shared
// memory; each adds a share of it over all of them, in rank order.
QMLP_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QMLP_DEV float4 sum_cluster(uint32_t addr, int n) {  // n <= 8
    float4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        v[r] = make_float4(0, 0, 0, 0);
        if (r < n) {
            uint32_t ra;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(r));
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                         : "r"(ra)
                         : "memory");
        }
    }
#pragma unroll
    for (int r = 1; r < 8; ++r) {
        v[0].x += v[r].x;
        v[0].y += v[r].y;
        v[0].z += v[r].z;
        v[0].w += v[r].w;
    }
    return v[0];
}

// ---------------------------------------------------------------------------
// v = c z W^T of a tile, NC columns. W: [NC][D], or with TRANS [D][NC]. The
// contraction is split over the CTAs of a cluster (gridDim.y), which add their
// partials through distributed shared memory.
// ---------------------------------------------------------------------------
template <int NC, bool TRANS, bool TWO>
struct ShrinkSmem {
    static constexpr int X = kT * kStep * 2, W = NC * kStep * 2;
    static constexpr int Stage = X + W * (TWO ? 2 : 1);
    static constexpr int Stages = 4;
    static constexpr int Bytes = Stage * Stages;
};

template <int NC, bool TRANS, bool TWO>
__global__ void __launch_bounds__(kThr) shrink_kernel(const LrShrink a) {
    using S = ShrinkSmem<NC, TRANS, TWO>;
    extern __shared__ __align__(128) uint8_t smem[];
    // (in this order: a GEMM launched early reads without a wait of its own what
    // the launches before this one wrote, see GemmLaunch::early)
    pdl_wait();
    pdl_launch_dependents();
    int slot, pos0, n, entry0;
    if (!tile_of(a.tok, blockIdx.x, slot, pos0, n, entry0) || slot < 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int z = blockIdx.z;
    const __nv_bfloat16* x = a.x + (size_t)z * a.x_z;
    const ptrdiff_t lo = a.x_lo ? a.x_lo - a.x : 0;
    const __nv_bfloat16* w = a.w + (size_t)slot * a.w_slot + (size_t)z * a.w_z;
    const __nv_bfloat16* w2 = TWO ? a.w_lo + (size_t)z * a.w_z : nullptr;
    // a second word of x is the same contraction once more
    const int one = (a.D + kStep - 1) / kStep, steps = a.x_lo ? 2 * one : one;
    const int s0 = (int)((long)steps * blockIdx.y / gridDim.y), s1 = (int)((long)steps * (blockIdx.y + 1) / gridDim.y);
    const uint32_t base = smem_u32(smem);

    // this thread's chunks of a step: x rows (tid >> 3) + 16 i, chunk tid & 7
    const __nv_bfloat16* xr[4];
    bool xl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 16 * i;
        xl[i] = r < n;
        const int tok = xl[i] ? token_at(a.tok, pos0 + r, 0) : 0;
        xr[i] = x + (size_t)tok * a.ldx;
    }
    auto load = [&](int step, int stage) {
        const uint32_t sx = base + stage * S::Stage, swt = sx + S::X;
        const int d0 = (step < one ? step : step - one) * kStep;
        const ptrdiff_t word = step < one ? 0 : lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 16 * i, c = tid & 7, d = d0 + c * 8;
            const bool live = xl[i] && d < a.D;
            cp16(sx + sw<8>(r, c), live ? xr[i] + word + d : x, live);
        }
        constexpr int kW = NC * kStep / 8;  // chunks of the W tile
#pragma unroll
        for (int i = 0; i < kW / kThr; ++i) {
            const int k = tid + i * kThr;
            if (TRANS) {
                const int r = k / (NC / 8), c = k % (NC / 8);
                const bool live = d0 + r < a.D;
                const size_t off = live ? (size_t)(d0 + r) * NC + c * 8 : 0;
                cp16(swt + sw<NC / 8>(r, c), w + off, live);
                if (TWO) cp16(swt + S::W + sw<NC / 8>(r, c), w2 + off, live);
            } else {
                const int r = k >> 3, c = k & 7, d = d0 + c * 8;
                bool live = d < a.D;
                const __nv_bfloat16* src = w + (size_t)r * a.D;
                if (!a.w) {
                    const int part = r >= a.R, j = r - part * a.R;
                    src = a.wa[part] + (size_t)j * a.D;
                    live = live && a.wa[part] && j < a.r;
                }
                cp16(swt + sw<8>(r, c), live ? src + d : x, live);
            }
        }
        cp_commit();
    };

    float acc[NC / 8][4];
#pragma unroll
    for (int j = 0; j < NC / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
    for (int p = 0; p < S::Stages - 1; ++p) {
        if (s0 + p < s1) load(s0 + p, p);
        else cp_commit();
    }
    const int q = lane >> 3, r8 = lane & 7;
    for (int st = s0; st < s1; ++st) {
        cp_wait<S::Stages - 2>();
        __syncthreads();
        const int nx = st + S::Stages - 1;
        if (nx < s1) load(nx, (nx - s0) % S::Stages);
        else cp_commit();
        const uint32_t sx = base + ((st - s0) % S::Stages) * S::Stage, swt = sx + S::X;
        if (warp * 16 < n) {
#pragma unroll
            for (int k = 0; k < kStep; k += 16) {
                uint32_t af[4];
                ldsm4(af, sx + sw<8>(warp * 16 + (q & 1) * 8 + r8, (k >> 3) + (q >> 1)));
#pragma unroll
                for (int j = 0; j < NC / 16; ++j) {
                    uint32_t b[4];
                    load_b<TRANS, TRANS ? NC / 8 : 8>(swt, j * 16, k, lane, b);
                    mma_bf16(acc[2 * j], af, b[0], b[1]);
                    mma_bf16(acc[2 * j + 1], af, b[2], b[3]);
                    if (TWO) {
                        load_b<TRANS, TRANS ? NC / 8 : 8>(swt + S::W, j * 16, k, lane, b);
                        mma_bf16(acc[2 * j], af, b[0], b[1]);
                        mma_bf16(acc[2 * j + 1], af, b[2], b[3]);
                    }
                }
            }
        }
    }

    // fragment (j, e): row 16 warp + g + 8 (e >> 1), column 8 j + 2 t + (e & 1)
    const int g = lane >> 2, t = lane & 3, ns = gridDim.y;
    constexpr int kPitch = NC + 4;  // floats of a row of the partial tile
    static_assert(kT * kPitch * 4 <= S::Bytes, "the tile takes the stages' place");
    __syncthreads();
    float* tile = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int j = 0; j < NC / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(tile + (warp * 16 + g + 8 * h) * kPitch + j * 8 + 2 * t) =
                make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    if (ns > 1) cluster_sync();
    else __syncthreads();
    const float c = a.scale ? a.scale[slot] : a.scale_all;
    // this CTA's share of the rows, four columns a thread and round
    const int rows = kT / ns, r0 = blockIdx.y * rows;
    for (int i = tid; i < rows * (NC / 4); i += kThr) {
        const int row = r0 + i / (NC / 4), col = (i % (NC / 4)) * 4;
        if (row >= n) break;
        const uint32_t at = base + (row * kPitch + col) * 4;
        const float4 s = ns > 1 ? sum_cluster(at, ns) : *reinterpret_cast<const float4*>(tile + row * kPitch + col);
        const float f = c * (z * NC + col < a.half ? a.mul0 : a.mul1);
        const float val[4] = {s.x * f, s.y * f, s.z * f, s.w * f};
        __nv_bfloat16 w[4][kLrWords];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            split_bf16(val[e], w[e]);
            if (a.again) w[e][2] = w[e][0];
        }
        const int pos = pos0 + row;
        const ptrdiff_t line0 = (ptrdiff_t)(a.entries ? (entry0 + (pos >> 8)) * 256 + (pos & 255) : pos) * a.ldv;
        if (!QMLP_INB(line0, (ptrdiff_t)a.v_elems - a.ldv + 1, 63)) continue;
        __nv_bfloat16* line = a.v + line0;
        __nv_bfloat16* o = line + z * NC + col;
#pragma unroll
        for (int k = 0; k < kLrWords; ++k)
            if (k < a.words) {
                const __nv_bfloat162 p[2] = {__halves2bfloat162(w[0][k], w[1][k]), __halves2bfloat162(w[2][k], w[3][k])};
                *reinterpret_cast<uint2*>(o + k * a.v_word) = *reinterpret_cast<const uint2*>(p);
            }
        // the columns past the words of a row that a GEMM reads whole
        for (int p = col + z * NC; p < a.pad; p += NC * gridDim.z)
            *reinterpret_cast<uint2*>(line + a.ldv - a.pad + p) = make_uint2(0, 0);
    }
    if (ns > 1) cluster_sync();  // no CTA leaves while another reads its tile
}

// ---------------------------------------------------------------------------
// y = v W^T of a tile (RC columns of v): W [N][RC], or with TRANS [RC][N].
// A CTA takes kNB columns of y in pieces of 64; the fragments of v stay in
// registers. Epilogue: fp32 y, or bf16(factor[n] raw + y).
// ---------------------------------------------------------------------------
constexpr int kNB = 256;
template <int RC>
constexpr int expand_smem() { return 3 * 64 * RC * 2; }

template <int RC, bool TRANS, int NW>
__global__ void __launch_bounds__(kThr) expand_kernel(const LrExpand a) {
    constexpr int kPiece = 64 * RC * 2;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    int slot, pos0, n, entry0;
    if (!tile_of(a.tok, blockIdx.x, slot, pos0, n, entry0)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int z = blockIdx.z;
    const int n0 = blockIdx.y * kNB, n1 = min(a.N, n0 + kNB);
    const int pieces = (n1 - n0 + 63) / 64;
    const __nv_bfloat16* w = a.w + (size_t)max(slot, 0) * a.w_slot + (size_t)z * a.w_z;
    const uint32_t base = smem_u32(smem);
    const int row0 = warp * 16 + g;
    int tok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row0 + 8 * h;
        tok[h] = r < n ? token_at(a.tok, pos0 + r, -1) : -1;
    }
    auto load = [&](int p, int stage) {
        constexpr int kC = 64 * RC / 8;
        const int nb = n0 + p * 64;
#pragma unroll
        for (int i = 0; i < kC / kThr; ++i) {
            const int k = tid + i * kThr;
            if (TRANS) {
                const int r = k >> 3, c = k & 7;
                const bool live = nb + c * 8 < a.N;
                cp16(base + stage * kPiece + sw<8>(r, c), w + (live ? (size_t)r * a.N + nb + c * 8 : 0), live);
            } else {
                const int r = k / (RC / 8), c = k % (RC / 8);
                const bool live = nb + r < a.N;
                cp16(base + stage * kPiece + sw<RC / 8>(r, c), w + (live ? (size_t)(nb + r) * RC + c * 8 : 0), live);
            }
        }
        cp_commit();
    };
    uint32_t af[RC / 16][NW][4];
    if (slot >= 0) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (p < pieces) load(p, p);
            else cp_commit();
        }
#pragma unroll
        for (int k = 0; k < RC / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = row0 + 8 * (e & 1);
                const __nv_bfloat16* o = a.v + (size_t)(pos0 + r) * a.ldv + z * RC + k * 16 + 2 * t + 8 * (e >> 1);
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    af[k][i][e] = r < n ? *reinterpret_cast<const uint32_t*>(o + i * a.v_word) : 0u;
            }
    }
    for (int p = 0; p < pieces; ++p) {
        float acc[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
        if (slot >= 0) {
            cp_wait<1>();
            __syncthreads();
            if (p + 2 < pieces) load(p + 2, (p + 2) % 3);
            else cp_commit();
            if (warp * 16 < n) {
                const uint32_t sb = base + (p % 3) * kPiece;
#pragma unroll
                for (int k = 0; k < RC / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t b[4];
                        load_b<TRANS, TRANS ? 8 : RC / 8>(sb, j * 16, k * 16, lane, b);
#pragma unroll
                        for (int i = 0; i < NW; ++i) {
                            mma_bf16(acc[2 * j], af[k][i], b[0], b[1]);
                            mma_bf16(acc[2 * j + 1], af[k][i], b[2], b[3]);
                        }
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = n0 + p * 64 + j * 8 + 2 * t;
            if (col >= a.N) continue;  // N is even
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (tok[h] < 0) continue;
                const float v0 = acc[j][2 * h], v1 = acc[j][2 * h + 1];
                if (a.out) {
                    const float2 r = *reinterpret_cast<const float2*>(a.raw + (size_t)tok[h] * a.N + col);
                    const float f0 = a.factor ? a.factor[col] : a.factor_all, f1 = a.factor ? a.factor[col + 1] : a.factor_all;
                    *reinterpret_cast<__nv_bfloat162*>(a.out + (size_t)tok[h] * a.N + col) =
                        __floats2bfloat162_rn(r.x * f0 + v0, r.y * f1 + v1);
                } else {
                    const size_t at = (size_t)tok[h] * a.ldy + (size_t)z * a.N + col;
                    if (QMLP_INB(at + 1, a.y_elems, 64)) *reinterpret_cast<float2*>(a.y + at) = make_float2(v0, v1);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// z^T v over the tokens (the words of z in turn): a CTA takes 128 columns of z
// (32 a warp) and the NC of v; the tokens are split over the CTAs of a cluster;
// one launch takes all gradients of an adapter, tile after tile. v in two words (2^-17): the gradients are bf16.
// ---------------------------------------------------------------------------
constexpr int kGD = 128;
template <int NC>
struct GradSmem {
    static constexpr int X = 64 * kGD * 2, V = 64 * NC * 2;
    static constexpr int Stage = X + 2 * V;
    static constexpr int Stages = 3;
    static constexpr int Bytes = Stage * Stages;
};

template <int NC>
__global__ void __launch_bounds__(kThr) tokgrad_kernel(const __grid_constant__ LrTokGrads jobs) {
    using S = GradSmem<NC>;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    int tile = blockIdx.x, job = 0;
    while (tile >= jobs.tiles[job]) tile -= jobs.tiles[job++];
    const LrTokGrad& a = jobs.job[job];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int d0 = tile * kGD;
    const int one = (a.M + 63) / 64, steps = a.x_lo ? 2 * one : one;
    const int s0 = (int)((long)steps * blockIdx.y / gridDim.y), s1 = (int)((long)steps * (blockIdx.y + 1) / gridDim.y);
    const __nv_bfloat16* x = a.x + d0;
    const ptrdiff_t lo = a.x_lo ? a.x_lo - a.x : 0;
    const __nv_bfloat16* v = a.v;
    const uint32_t base = smem_u32(smem);
    auto load = [&](int step, int stage) {
        const uint32_t sx = base + stage * S::Stage, sv = sx + S::X;
        const int m0 = (step < one ? step : step - one) * 64;
        const ptrdiff_t word = step < one ? 0 : lo;
#pragma unroll
        for (int i = 0; i < 64 * (kGD / 8) / kThr; ++i) {
            const int k = tid + i * kThr, r = k >> 4, c = k & 15;
            const bool live = m0 + r < a.M && d0 + c * 8 < a.D;
            cp16(sx + sw<16>(r, c), live ? x + word + (size_t)(m0 + r) * a.ldx + c * 8 : a.x, live);
        }
#pragma unroll
        for (int i = 0; i < 64 * (NC / 8) / kThr; ++i) {
            const int k = tid + i * kThr, r = k / (NC / 8), c = k % (NC / 8);
            const bool live = m0 + r < a.M;
            const __nv_bfloat16* p = live ? v + (size_t)(m0 + r) * a.ldv + c * 8 : a.v;
            cp16(sv + sw<NC / 8>(r, c), p, live);
            cp16(sv + S::V + sw<NC / 8>(r, c), p + (live ? a.v_word : 0), live);
        }
        cp_commit();
    };
    float acc[2][NC / 8][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NC / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[h][j][e] = 0.0f;
#pragma unroll
    for (int p = 0; p < S::Stages - 1; ++p) {
        if (s0 + p < s1) load(s0 + p, p);
        else cp_commit();
    }
    const int q = lane >> 3, r8 = lane & 7;
    for (int st = s0; st < s1; ++st) {
        cp_wait<S::Stages - 2>();
        __syncthreads();
        const int nx = st + S::Stages - 1;
        if (nx < s1) load(nx, (nx - s0) % S::Stages);
        else cp_commit();
        const uint32_t sx = base + ((st - s0) % S::Stages) * S::Stage, sv = sx + S::X;
#pragma unroll
        for (int k = 0; k < 64; k += 16) {
            uint32_t af[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)  // the transposed tile: rows are columns of z, the contraction tokens
                ldsm4t(af[h], sx + sw<16>(k + (q >> 1) * 8 + r8, (warp * 32 + h * 16) / 8 + (q & 1)));
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int j = 0; j < NC / 16; ++j) {
                    uint32_t b[4];
                    load_b<true, NC / 8>(sv + w * S::V, j * 16, k, lane, b);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma_bf16(acc[h][2 * j], af[h], b[0], b[1]);
                        mma_bf16(acc[h][2 * j + 1], af[h], b[2], b[3]);
                    }
                }
        }
    }
    const int g = lane >> 2, t = lane & 3, ns = gridDim.y;
    constexpr int kPitch = NC + 4;
    static_assert(kGD * kPitch * 4 <= S::Bytes, "the tile takes the stages' place");
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);  // [column of z][column of v]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NC / 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2*>(sums + (warp * 32 + h * 16 + g + 8 * e) * kPitch + j * 8 + 2 * t) =
                    make_float2(acc[h][j][2 * e], acc[h][j][2 * e + 1]);
    if (ns > 1) cluster_sync();
    else __syncthreads();
    const int rows = kGD / ns, r0 = blockIdx.y * rows;
    for (int i = tid; i < rows * (NC / 4); i += kThr) {
        // B's gradient lies along v's columns, A's along z's
        const int row = r0 + (a.rows_d ? i / (NC / 4) : i % rows);
        const int col = (a.rows_d ? i % (NC / 4) : i / rows) * 4;
        const int d = d0 + row;
        if (d >= a.D) continue;
        const uint32_t at = base + (row * kPitch + col) * 4;
        const float4 s4 = ns > 1 ? sum_cluster(at, ns) : *reinterpret_cast<const float4*>(sums + row * kPitch + col);
        const float s[4] = {s4.x, s4.y, s4.z, s4.w};
        if (a.rows_d) {
            const float f = a.div ? a.div[d] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.r && QMLP_INB((size_t)d * a.r + col + e, (size_t)a.D * a.r, 68))
                    a.out[(size_t)d * a.r + col + e] = __float2bfloat16_rn(a.div ? s[e] / f : s[e] * a.mul);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.r && QMLP_INB((size_t)(col + e) * a.D + d, (size_t)a.D * a.r, 68))
                    a.out[(size_t)(col + e) * a.D + d] = __float2bfloat16_rn(s[e] * a.mul);
        }
    }
    if (ns > 1) cluster_sync();
}

// ---------------------------------------------------------------------------
// Few tokens (M <= kLrFew): each names its slot itself; no plan.
// ---------------------------------------------------------------------------
QMLP_DEV float dot8(const uint4& a, const uint4& b, float s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
        s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
    }
    return s;
}

// v[m, j] = c A[slot(m)][j] . x[m]: a CTA a (row j, token m). The next launch may
// start at once or, `late`, once everything before this one has completed: for
// kernels that read what came before without a wait of their own (gemv_split.cu,
// GemmLaunch::early).
__global__ void __launch_bounds__(kThr) shrink_few_kernel(const LrFew a) {
    const int j = blockIdx.x, m = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!a.late) pdl_launch_dependents();
    pdl_wait();
    if (a.late) pdl_launch_dependents();
    const int slot = a.ids[m];
    const bool has = slot >= 0 && slot < a.slots && a.rank[slot] > j % a.Rp;
    float s = 0.0f;
    if (has) {
        const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)m * a.D);
        const uint4* w = reinterpret_cast<const uint4*>(a.w + (size_t)slot * a.w_slot + (size_t)j * a.D);
#pragma unroll 4
        for (int i = threadIdx.x; i < a.D / 8; i += kThr) s = dot8(__ldg(x + i), __ldg(w + i), s);
    }
    __shared__ float red[kThr / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0 && QMLP_INB((size_t)m * a.ncol + j, a.v_elems, 65))
        a.v[(size_t)m * a.ncol + j] = has ? (red[0] + red[1] + red[2] + red[3]) * a.scale[slot] : 0.0f;
}

// y[m, n] = sum_j v[m, j] B[slot(m)][n][j]: a thread an n, kFewTok tokens in turn
// (so few CTAs that all are resident at once: the GEMM after them then starts
// beside them).
constexpr int kFewTok = 8;
__global__ void __launch_bounds__(kThr) expand_few_kernel(const LrFew a) {
    pdl_launch_dependents();
    const int n = blockIdx.x * kThr + threadIdx.x, z = blockIdx.z, m0 = blockIdx.y * kFewTok;
    pdl_wait();
    if (n >= a.D) return;
    const float f = a.factor ? a.factor[n] : a.factor_all;
#pragma unroll 2
    for (int m = m0; m < min(a.M, m0 + kFewTok); ++m) {
        const int slot = a.ids[m];
        const int nr = slot >= 0 && slot < a.slots ? (a.rank[slot] + 7) / 8 : 0;
        const uint4* b = reinterpret_cast<const uint4*>(a.w + (size_t)(nr ? slot : 0) * a.w_slot + ((size_t)z * a.D + n) * a.Rp);
        const float* v = a.v + (size_t)m * a.ncol + z * a.Rp;
        float s = 0.0f;
#pragma unroll 2
        for (int i = 0; i < nr; ++i) {
            const uint4 q = __ldg(b + i);
            const uint32_t y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s = fmaf(v[i * 8 + 2 * e], __uint_as_float(y[e] << 16), s);
                s = fmaf(v[i * 8 + 2 * e + 1], __uint_as_float(y[e] & 0xFFFF0000u), s);
            }
        }
        if (a.out) a.out[(size_t)m * a.D + n] = __float2bfloat16_rn(a.raw[(size_t)m * a.D + n] * f + s);
        else if (QMLP_INB((size_t)m * a.ldy + (size_t)z * a.D + n, a.y_elems, 65))
            a.y[(size_t)m * a.ldy + (size_t)z * a.D + n] = s;
    }
}

// ---------------------------------------------------------------------------
// act = bf16(SiLU(fg raw_g + y_g) * (fu raw_u + y_u)), y = [M][2I] the adapters'
// terms: shapes whose gate/up kernels cannot add them themselves.
__global__ void __launch_bounds__(256) swiglu_raw_kernel(const LrSwiGLU a) {
    pdl_launch_dependents();
    pdl_wait();
    const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long)a.M * a.I) return;
    const int m = (int)(i / a.I), n = (int)(i % a.I);
    const float g = a.raw_g[i] * (a.fg ? a.fg[n] : a.fg_all) + a.y[(size_t)m * 2 * a.I + n];
    const float u = a.raw_u[i] * (a.fu ? a.fu[n] : a.fu_all) + a.y[(size_t)m * 2 * a.I + a.I + n];
    a.act[i] = __float2bfloat16_rn(silu_f32(g) * u);
}

// Tokens grouped by slot: perm holds the tokens slot by slot (those without an
// adapter last), tiles the {slot or -1, first position, tokens} of at most 64.
// One CTA (3001 tokens, 7 slots: 8 us, 14 to 16 with the GEMM's lists); the order of a
// slot's tokens is left to the atomics where no result depends on it.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) plan_kernel(const int* __restrict__ ids, int M, int slots,
                                                    const int* __restrict__ rank, int* perm, int4* tiles,
                                                    int* n_tiles, int2* ents, int* ent_slot,
                                                    const int* __restrict__ odd, int* odd_rows, int max_tiles,
                                                    int max_ents) {
    __shared__ int cnt[kLrMaxSlots + 1], pos[kLrMaxSlots + 1];
    __shared__ int wsum[3][32];
    __shared__ int first[kLrMaxEnts], last[kLrMaxEnts];
    __shared__ int wcnt[32 * kPlanTable];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= slots; i += 1024) cnt[i] = 0;
    __syncthreads();
    auto group = [&](int m) {
        const int s = ids[m];
        return s >= 0 && s < slots && rank[s] > 0 ? s : slots;
    };
    // one atomic a warp and group: the lanes of a group find each other first
    auto claim = [&](int* at, int gr) {
        const unsigned mask = __match_any_sync(0xffffffffu, gr);
        const int lead = __ffs(mask) - 1;
        int b = 0;
        if (lane == lead && gr >= 0) b = atomicAdd(&at[gr], __popc(mask));
        return __shfl_sync(0xffffffffu, b, lead) + __popc(mask & ((1u << lane) - 1u));
    };
    for (int m = tid; m < (M + 31) / 32 * 32; m += 1024) claim(cnt, m < M ? group(m) : -1);
    __syncthreads();
    const int big = (M + 255) / 256;
    if (ents)
        for (int t = tid; t < big; t += 1024) first[t] = 0, last[t] = -1;
    const int with = M - cnt[slots];  // tokens with an adapter: positions 0 .. with - 1
    __syncthreads();
    // exclusive sums over the groups of tokens, tiles and entries, 1024 groups a
    // round. A group's entries: one for each 256 positions that it reaches into,
    // which its first position has to be known for: a second scan
    int tok0 = 0, til0 = 0, ent0 = 0;
    for (int b = 0; b <= slots; b += 1024) {
        const int i = b + tid;
        const int c = i <= slots ? cnt[i] : 0, tl = (c + kT - 1) / kT;
        int sc = c, st = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sc, o), v = __shfl_up_sync(0xffffffffu, st, o);
            if (lane >= o) sc += u, st += v;
        }
        if (lane == 31) wsum[0][warp] = sc, wsum[1][warp] = st;
        __syncthreads();
        int bc = tok0, bt = til0, ac = 0, at = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) bc += wsum[0][w], bt += wsum[1][w];
            ac += wsum[0][w], at += wsum[1][w];
        }
        const int p0 = bc + sc - c;
        const int ne = ents && c && i < slots ? ((p0 + c - 1) >> 8) - (p0 >> 8) + 1 : 0;
        int se = ne;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, se, o);
            if (lane >= o) se += v;
        }
        if (lane == 31) wsum[2][warp] = se;
        __syncthreads();
        int be = ent0, ae = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) be += wsum[2][w];
            ae += wsum[2][w];
        }
        if (i <= slots) {
            pos[i] = p0;
            const int e0 = be + se - ne;  // its first entry
            for (int k = 0; k < tl && QMLP_INB(bt + st - tl + k, max_tiles, 66); ++k)
                tiles[bt + st - tl + k] =
                    make_int4(i < slots ? i : -1, p0 + k * kT, min(kT, c - k * kT), e0 - (p0 >> 8));
            for (int k = 0; k < ne && QMLP_INB(e0 + k, max_ents, 66) && QMLP_INB((p0 >> 8) + k, big, 66); ++k) {
                // positions are filled from 0 on: a tile's entries lie together,
                // from the group at its first position to that at its last
                const int t = (p0 >> 8) + k, lo = t * 256, hi = min(lo + 256, with) - 1;
                ent_slot[e0 + k] = i;
                if (p0 <= lo) first[t] = e0 + k;
                if (p0 + c - 1 >= hi) last[t] = e0 + k;
            }
        }
        ent0 += ae;
        tok0 += ac;
        til0 += at;
        __syncthreads();
    }
    if (!ents) {
        for (int m = tid; m < (M + 31) / 32 * 32; m += 1024) {
            const int at = claim(pos, m < M ? group(m) : -1);
            if (m < M && QMLP_INB(at, M, 66)) perm[at] = m;
        }
        if (tid == 0) *n_tiles = til0;
        return;
    }
    // With GEMM lists the order within a group is the tokens': the position
    // decides which tile, and so which order of sums. For few groups the warps'
    // counts of 1024 tokens are scanned together, for many the warps claim in turn
    // (3001 tokens, 7 slots: 30 us in turn)
    const bool table = slots < kPlanTable;
    auto place = [&](int at, int m, int gr) {
        if (!QMLP_INB(at, M, 66)) return;
        perm[at] = m;
        odd_rows[at] = gr < slots ? odd[gr] : 0;
    };
    for (int b = 0; b < M; b += 1024) {
        const int m = b + tid, gr = m < M ? group(m) : -1;
        if (table) {
            for (int i = tid; i < 32 * kPlanTable; i += 1024) wcnt[i] = 0;
            __syncthreads();
            const unsigned mask = __match_any_sync(0xffffffffu, gr);
            if (gr >= 0 && lane == __ffs(mask) - 1) wcnt[warp * kPlanTable + gr] = __popc(mask);
            __syncthreads();
            if (tid <= slots) {
                int at = pos[tid];
                for (int w = 0; w < 32; ++w) {
                    const int n = wcnt[w * kPlanTable + tid];
                    wcnt[w * kPlanTable + tid] = at;
                    at += n;
                }
                pos[tid] = at;
            }
            __syncthreads();
            if (m < M) place(wcnt[warp * kPlanTable + gr] + __popc(mask & ((1u << lane) - 1u)), m, gr);
            __syncthreads();
        } else {
            for (int w = 0; w < 32 && b + w * 32 < M; ++w) {
                if (w == warp) {
                    const int at = claim(pos, gr);
                    if (m < M) place(at, m, gr);
                }
                __syncthreads();
            }
        }
    }
    if (tid == 0) *n_tiles = til0;
    for (int t = tid; t < big; t += 1024) ents[t] = make_int2(first[t], last[t] - first[t] + 1);
}

__global__ void __launch_bounds__(256) gather_kernel(const uint4* __restrict__ x, const int* __restrict__ perm, int n16,
                                                     uint4* rows) {
    pdl_launch_dependents();
    pdl_wait();
    const int tok = perm[blockIdx.x];
    const uint4* src = x + (size_t)(QMLP_INB(tok, gridDim.x, 62) ? tok : 0) * n16;
    uint4* dst = rows + (size_t)blockIdx.x * n16;
    for (int i = threadIdx.x; i < n16; i += 256) dst[i] = src[i];
}

// One adapter into a slot's padded rows: A [r, D] -> [Rp][D], B [N, r] ->
// [N][Rp] (B / div[n] where div is given, in two bf16 words), zero past r or
// where the projection is not adapted.
__global__ void __launch_bounds__(256) pack_kernel(const LrPack a) {
    pdl_launch_dependents();
    pdl_wait();
    const int p = a.first + blockIdx.y;  // 0..2: A of gate, up, down; 3..5: B
    const LrPackPart& q = a.part[p];
    const uint32_t total = (uint32_t)q.rows * q.cols;  // at most 64 x 65536
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
        const int row = (int)(i / (uint32_t)q.cols), col = (int)(i % (uint32_t)q.cols);
        // A: rows are the rank; B: columns are
        const bool in = q.src && (p < 3 ? row : col) < a.r;
        __nv_bfloat16 v = __float2bfloat16_rn(0.0f);
        if (in) v = q.src[p < 3 ? (size_t)row * q.cols + col : (size_t)row * a.r + col];
        q.dst[i] = v;
        if (q.dst_h) {
            __nv_bfloat16 d[2];
            split_bf16(__bfloat162float(v) / (q.div ? q.div[row] : q.div_all), d);
            q.dst_h[i] = d[0];
            q.dst_l[i] = d[1];
        }
    }
    if (blockIdx.y == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        *a.rank_out = a.r;
        *a.scale_out = a.scale;
        if (a.odd_out) *a.odd_out = 0;
    }
}

// B's value as a step image holds it: over its row's factor (T = 3) or as it is.
QMLP_DEV float step_value(__nv_bfloat16 b, float div, int T) {
    const float v = __bfloat162float(b);
    return T == 3 ? __fdividef(v, div) : v;
}
// Not finite, in bf16.
QMLP_DEV bool odd_value(float v) {
    return (__bfloat16_as_ushort(__float2bfloat16_rn(v)) & 0x7F80u) == 0x7F80u;
}

// (4.5 MB of images of rank 16: 9 us.)
// Stage images of an adapter's side of a GEMM's further steps: 256 rows of 64
// columns each, 128-byte swizzled (16-byte chunk l of row n at l ^ (n & 7)). A
// column is (word, part, j): with T = 2 words (the activations' v = h + l) both
// hold the value; with T = 3 the value over the row's factor does not fit one
// bf16 word: h and l times its first word, h times its second.
__global__ void __launch_bounds__(256) image_kernel(const LrImage a) {
    pdl_launch_dependents();
    pdl_wait();
    const int sh = a.R == 16 ? 4 : a.R == 32 ? 5 : 6, two = a.parts - 1;
    const int img = blockIdx.x >> 3, e = img % a.ext, nt = img / a.ext;  // a CTA 32 rows of an image
    const int i = (blockIdx.x & 7) * 256 + threadIdx.x;
    const int p = i & 7, row = i >> 3, l = p ^ (row & 7);
    const int side = a.interleaved ? row >> 7 : 0;
    const int n = a.interleaved ? nt * 128 + (row & 127) : nt * 256 + row;
    const float div = a.T == 3 && n < a.N ? a.div[side][n] : 1.0f;
    // the eight columns of a chunk lie in one word and part (R is 16 or more)
    const int c = e * 64 + l * 8, wp = c >> sh, j0 = c & (a.R - 1);
    const int w = wp >> two, part = wp & two;
    const bool in = w < a.T && n < a.N && a.src[part] && (!a.interleaved || part == side);
    const __nv_bfloat16* src = in ? a.src[part] + (size_t)n * a.sn + (size_t)j0 * a.sj : nullptr;
    __align__(16) __nv_bfloat16 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = in && j0 + k < a.r ? src[(size_t)k * a.sj] : __float2bfloat16_rn(0.0f);
    bool left = false;
    if (a.T == 3 || a.odd) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float v = step_value(o[k], div, a.T);
            if (a.odd && odd_value(v)) {
                left = true;
                v = 0.0f;
            }
            if (w == 2) v -= __bfloat162float(__float2bfloat16_rn(v));
            o[k] = __float2bfloat16_rn(v);
        }
    }
    if (left) *a.odd = 1;
    if (QMLP_INB(((size_t)img * 2048 + i) * 16 + 15, a.img_bytes, 67))
        *reinterpret_cast<uint4*>(a.img + ((size_t)img * 2048 + i) * 16) = *reinterpret_cast<const uint4*>(o);
}

// The further steps of a 256-token tile multiply all its rows by the images of
// every slot in it, the rows of other slots being zeros. A value of one request's
// B that is not finite (Inf or NaN, or past bf16 over its row's factor) would make
// those zeros NaN, so the images hold a zero in its place, and its terms, B v
// value by value, come to its own tokens' rows alone: through y, which the GEMM's
// epilogue adds where the plan has marked the row. Calls without such values pay
// for an empty launch before each GEMM (3001 FP8 tokens: 5 and 2 us of 1200).
__global__ void __launch_bounds__(kThr) odd_kernel(const LrOdd a) {
    pdl_wait();
    pdl_launch_dependents();
    int slot, pos0, n, entry0;
    if (!tile_of(a.tok, blockIdx.x, slot, pos0, n, entry0) || slot < 0 || !a.odd[slot]) return;
    const int z = blockIdx.z;
    for (int c = blockIdx.y * kThr + threadIdx.x; c < a.N; c += gridDim.y * kThr) {
        const __nv_bfloat16* b = a.w + (size_t)slot * a.w_slot + ((size_t)z * a.N + c) * a.R;
        const float div = a.T == 3 ? a.div[z][c] : 1.0f;
        uint64_t left = 0;
        for (int j = 0; j < a.R; ++j) left |= (uint64_t)odd_value(step_value(b[j], div, a.T)) << j;
        for (int r = 0; r < n; ++r) {
            const int pos = pos0 + r;
            const ptrdiff_t line = (ptrdiff_t)((entry0 + (pos >> 8)) * 256 + (pos & 255)) * a.ldv;
            if (!QMLP_INB(line, (ptrdiff_t)a.v_elems - a.ldv + 1, 63)) continue;
            const __nv_bfloat16* v = a.v + line + z * a.R;
            float s = 0.0f;
            for (uint64_t m = left; m; m &= m - 1) {
                const int j = __ffsll((long long)m) - 1;
                s = fmaf(__bfloat162float(b[j]), __bfloat162float(v[j]) + __bfloat162float(v[a.nc + j]), s);
            }
            const size_t at = (size_t)pos * a.ldy + (size_t)z * a.N + c;
            if (QMLP_INB(at, a.y_elems, 64)) a.y[at] = s * a.mul[z];
        }
    }
}

template <typename K, typename A>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, int smem, const A& a, cudaStream_t s, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = (unsigned)cluster;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int NC, bool TRANS, bool TWO>
cudaError_t shrink_t(const LrShrink& a, int tiles, int splits, int zs, cudaStream_t s) {
    static bool attr = false;
    using S = ShrinkSmem<NC, TRANS, TWO>;
    if (!attr) {
        const cudaError_t e = cudaFuncSetAttribute(shrink_kernel<NC, TRANS, TWO>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, S::Bytes);
        if (e != cudaSuccess) return e;
        attr = true;
    }
    return launch_pdl(shrink_kernel<NC, TRANS, TWO>, dim3(tiles, splits, zs), kThr, S::Bytes, a, s, splits);
}
template <bool TRANS, bool TWO>
cudaError_t shrink_n(const LrShrink& a, int nc, int tiles, int splits, int zs, cudaStream_t s) {
    switch (nc) {
        case 16: return shrink_t<16, TRANS, TWO>(a, tiles, splits, zs, s);
        case 32: return shrink_t<32, TRANS, TWO>(a, tiles, splits, zs, s);
        case 64: return shrink_t<64, TRANS, TWO>(a, tiles, splits, zs, s);
        case 128:
            if constexpr (!TRANS) return shrink_t<128, false, false>(a, tiles, splits, zs, s);
    }
    return cudaErrorInvalidValue;
}
template <int RC, bool TRANS, int NW>
cudaError_t expand_t(const LrExpand& a, int tiles, int zs, cudaStream_t s) {
    static bool attr = false;
    if (!attr) {
        const cudaError_t e = cudaFuncSetAttribute(expand_kernel<RC, TRANS, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   expand_smem<RC>());
        if (e != cudaSuccess) return e;
        attr = true;
    }
    return launch_pdl(expand_kernel<RC, TRANS, NW>, dim3(tiles, (a.N + kNB - 1) / kNB, zs), kThr, expand_smem<RC>(), a, s);
}

}  // namespace

int lr_max_tiles(int M, int slots) { return M / kT + std::min(slots + 1, M) + 1; }

// CTAs of a cluster that share a contraction of `steps`: a power of two up to
// 8, while the grid stays under four CTAs an SM and each has two steps.
static int lr_splits(int tiles, int steps, int num_sms) {
    int n = 1;
    while (n < 8 && 2 * n * tiles <= 4 * num_sms && steps >= 4 * n) n *= 2;
    return n;
}

cudaError_t launch_lr_shrink(const LrShrink& a, int nc, bool trans, int tiles, int zs, int num_sms, cudaStream_t s) {
    const int splits = lr_splits(tiles * zs, (a.D + kStep - 1) / kStep, num_sms);
    if (!trans) return shrink_n<false, false>(a, nc, tiles, splits, zs, s);
    return a.w_lo ? shrink_n<true, true>(a, nc, tiles, splits, zs, s) : shrink_n<true, false>(a, nc, tiles, splits, zs, s);
}

cudaError_t launch_lr_expand(const LrExpand& a, int rc, bool trans, int tiles, int zs, cudaStream_t s) {
    switch (rc) {
        case 16: return trans ? expand_t<16, true, 2>(a, tiles, zs, s) : expand_t<16, false, 3>(a, tiles, zs, s);
        case 32: return trans ? expand_t<32, true, 2>(a, tiles, zs, s) : expand_t<32, false, 3>(a, tiles, zs, s);
        case 64: return trans ? expand_t<64, true, 2>(a, tiles, zs, s) : expand_t<64, false, 3>(a, tiles, zs, s);
        case 128:
            if (trans) return expand_t<128, true, 2>(a, tiles, zs, s);
    }
    return cudaErrorInvalidValue;
}

template <int NC>
static cudaError_t tokgrad_t(const LrTokGrads& a, dim3 grid, cudaStream_t s) {
    static bool attr = false;
    if (!attr) {
        const cudaError_t e = cudaFuncSetAttribute(tokgrad_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   GradSmem<NC>::Bytes);
        if (e != cudaSuccess) return e;
        attr = true;
    }
    return launch_pdl(tokgrad_kernel<NC>, grid, kThr, GradSmem<NC>::Bytes, a, s, (int)grid.y);
}
cudaError_t launch_lr_tokgrad(LrTokGrads& a, int nc, int num_sms, cudaStream_t s) {
    int tiles = 0;
    for (int i = 0; i < a.count; ++i) tiles += a.tiles[i] = (a.job[i].D + kGD - 1) / kGD;
    if (!tiles) return cudaSuccess;
    const dim3 grid(tiles, lr_splits(tiles, (a.job[0].M + 63) / 64, 2 * num_sms), 1);
    switch (nc) {
        case 16: return tokgrad_t<16>(a, grid, s);
        case 32: return tokgrad_t<32>(a, grid, s);
        case 64: return tokgrad_t<64>(a, grid, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_lr_shrink_few(const LrFew& a, int M, cudaStream_t s) {
    return launch_pdl(shrink_few_kernel, dim3(a.ncol, M), kThr, 0, a, s);
}
cudaError_t launch_lr_expand_few(const LrFew& a, int M, int zs, cudaStream_t s) {
    LrFew b = a;
    b.M = M;
    return launch_pdl(expand_few_kernel, dim3((a.D + kThr - 1) / kThr, (M + kFewTok - 1) / kFewTok, zs), kThr, 0, b, s);
}

cudaError_t launch_lr_swiglu_raw(const LrSwiGLU& a, cudaStream_t s) {
    const long n = (long)a.M * a.I;
    return launch_pdl(swiglu_raw_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, a, s);
}

cudaError_t launch_lr_plan(const int* ids, int M, int slots, const int* rank, int* perm, int4* tiles, int* n_tiles,
                           int2* ents, int* ent_slot, const int* odd, int* odd_rows, cudaStream_t s) {
    if (slots < 1 || slots > kLrMaxSlots || (ents && M > 256 * kLrMaxEnts)) return cudaErrorInvalidValue;
    plan_kernel<<<1, 1024, 0, s>>>(ids, M, slots, rank, perm, tiles, n_tiles, ents, ent_slot, odd, odd_rows,
                                   lr_max_tiles(M, slots), lr_max_entries(M, slots));
    return cudaPeekAtLastError();
}

cudaError_t launch_lr_gather(const void* x, const int* perm, int M, int K, void* rows, cudaStream_t s) {
    gather_kernel<<<M, 256, 0, s>>>(static_cast<const uint4*>(x), perm, K / 8, static_cast<uint4*>(rows));
    return cudaPeekAtLastError();
}

cudaError_t launch_lr_image(const LrImage& a, cudaStream_t s) {
    return launch_pdl(image_kernel, dim3((unsigned)(a.tiles * a.ext * 8)), 256, 0, a, s);
}

cudaError_t launch_lr_odd(const LrOdd& a, int tiles, int parts, cudaStream_t s) {
    return launch_pdl(odd_kernel, dim3((unsigned)tiles, 4, (unsigned)parts), kThr, 0, a, s);
}

cudaError_t launch_lr_pack(const LrPack& a, cudaStream_t s) {
    pack_kernel<<<dim3(256, a.count), 256, 0, s>>>(a);
    return cudaPeekAtLastError();
}

QMLP_BOUNDS_UNIT(lowrank)

}  // namespace qmlp
