// lowrank.cuh -- launch arguments of the low-rank products (lowrank.cu).
#pragma once
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace qmlp {

constexpr int kLrTile = 64;       // tokens of a tile
constexpr int kLrMaxRank = 64;
constexpr int kLrWords = 3;       // bf16 words of a value of v
constexpr int kLrMaxSlots = 1024;
// Tokens that the kernels without a plan take (61 tokens of 16 adapters of rank
// 8 on a 4096 x 11008 block: 125 us with the plan's, 106 us with these).
constexpr int kLrFew = 64;

// Which tokens a tile holds: tiles null: one adapter, 64 consecutive tokens.
struct LrTokens {
    const int4* tiles = nullptr;  // {slot or -1, first position, tokens, entry of position p minus p / 256}
    const int* n_tiles = nullptr;
    const int* perm = nullptr;    // position -> token
    int M = 0;
    int slots = 1;                // index checks: slots that a tile may name
};

struct LrShrink {
    LrTokens tok;
    const __nv_bfloat16* x = nullptr;  // [M][ldx], D columns from z * x_z on
    const __nv_bfloat16* x_lo = nullptr;  // optional second word of x
    size_t ldx = 0, x_z = 0;
    int D = 0;
    const __nv_bfloat16* w = nullptr;     // slot and part strides in elements
    const __nv_bfloat16* w_lo = nullptr;  // second word of w, or null
    size_t w_slot = 0, w_z = 0;
    // or, not transposed, an adapter's own A's: row j of part p at wa[p] + j D, r
    // rows (the columns from r to R of a part are zero)
    const __nv_bfloat16* wa[2] = {nullptr, nullptr};
    int r = 0, R = 0;
    const float* scale = nullptr;  // per slot, or
    float scale_all = 1.0f;
    __nv_bfloat16* v = nullptr;    // [position][ldv], columns z * NC on, word i at i * v_word elements
    size_t v_word = 0;
    int ldv = 0;
    int words = kLrWords;
    bool entries = false;          // rows by GEMM entry: 256 entry(p) + p % 256 for position p
    bool again = false;            // the third word is the first once more
    int pad = 0;                   // columns at a row's end to fill with zeros
    size_t v_elems = 0;            // index checks: values that v holds
    float mul0 = 1.0f, mul1 = 1.0f;  // factors of the columns before and from `half` on
    int half = 1 << 30;
};

struct LrExpand {
    LrTokens tok;
    const __nv_bfloat16* v = nullptr;
    size_t v_word = 0;
    int ldv = 0;
    const __nv_bfloat16* w = nullptr;
    size_t w_slot = 0, w_z = 0;
    int N = 0;
    float* y = nullptr;  // fp32 [M][ldy], columns z * N on
    size_t ldy = 0, y_elems = 0;  // y_elems: index checks
    // or out = bf16(factor raw + y)
    __nv_bfloat16* out = nullptr;
    const float* raw = nullptr;     // fp32 [M][N]
    const float* factor = nullptr;  // per column, or factor_all
    float factor_all = 1.0f;
};

struct LrFew {
    const int* ids = nullptr;  // [M]
    const int* rank = nullptr;
    const float* scale = nullptr;
    int slots = 0, Rp = 0;
    int M = 0;  // expand: set by the launch
    bool late = false;
    const __nv_bfloat16* x = nullptr;  // shrink: [M][D]
    const __nv_bfloat16* w = nullptr;
    size_t w_slot = 0;
    int D = 0;           // shrink: contraction; expand: columns of a part
    int ncol = 0;        // columns of v
    float* v = nullptr;  // [M][ncol]
    float* y = nullptr;  // expand: as LrExpand
    size_t ldy = 0, v_elems = 0, y_elems = 0;
    __nv_bfloat16* out = nullptr;
    const float* raw = nullptr;
    const float* factor = nullptr;
    float factor_all = 1.0f;
};

// out = z^T v over the tokens of one adapter, in bf16: with rows_d, [D][r]
// (a B's gradient), else [r][D] (an A's).
struct LrTokGrad {
    const __nv_bfloat16* x = nullptr;  // [M][ldx], D columns
    const __nv_bfloat16* x_lo = nullptr;  // optional second word of x
    size_t ldx = 0;
    int D = 0, M = 0;
    const __nv_bfloat16* v = nullptr;  // [M][ldv], words v_word columns apart
    size_t v_word = 0;
    int ldv = 0;
    bool rows_d = false;
    int r = 0;
    __nv_bfloat16* out = nullptr;
    const float* div = nullptr;  // rows_d: the row's divisor; else mul
    float mul = 1.0f;
};
struct LrTokGrads {
    LrTokGrad job[6];
    int count = 0;
    int tiles[6] = {0, 0, 0, 0, 0, 0};  // set by the launch
};

struct LrSwiGLU {
    const float* raw_g = nullptr;  // [M][I]
    const float* raw_u = nullptr;
    const float* y = nullptr;      // [M][2I]
    const float* fg = nullptr;     // factors per column, or fg_all / fu_all
    const float* fu = nullptr;
    float fg_all = 1.0f, fu_all = 1.0f;
    __nv_bfloat16* act = nullptr;
    int M = 0, I = 0;
};

struct LrPackPart {
    const __nv_bfloat16* src = nullptr;
    __nv_bfloat16* dst = nullptr;
    int rows = 0, cols = 0;  // of dst
    __nv_bfloat16* dst_h = nullptr;  // B / div in two words, or null
    __nv_bfloat16* dst_l = nullptr;
    const float* div = nullptr;
    float div_all = 1.0f;
};
struct LrPack {
    LrPackPart part[6];
    int first = 0, count = 6;  // the parts to pack
    int r = 0;
    float scale = 0.0f;
    int* rank_out = nullptr;
    float* scale_out = nullptr;
    int* odd_out = nullptr;  // optional: set to 0
};

struct LrImage {
    const __nv_bfloat16* src[2] = {nullptr, nullptr};  // value of row n, column j: src[part][n sn + j sj]
    size_t sn = 0, sj = 0;
    int r = 0, R = 0, parts = 1, T = 2;
    const float* div[2] = {nullptr, nullptr};  // T = 3: the rows' factors
    int N = 0;            // rows of a part
    int interleaved = 0;  // tiles of 128 rows of part 0 and the same of part 1, each with its own columns
    int tiles = 0, ext = 0;
    uint8_t* img = nullptr;
    size_t img_bytes = 0; // index checks
    int* odd = nullptr;   // optional: values that are not finite are left out (zeros), and 1 goes there
};
cudaError_t launch_lr_image(const LrImage& a, cudaStream_t s);

// y = the terms of the values that a slot's images leave out, for the tokens of
// the slots that have such values (see odd_kernel).
struct LrOdd {
    LrTokens tok;
    const int* odd = nullptr;          // per slot
    const __nv_bfloat16* v = nullptr;  // by GEMM entry, two words nc columns apart
    int ldv = 0, nc = 0;
    const __nv_bfloat16* w = nullptr;  // padded B's: [slot][part][N][R]
    size_t w_slot = 0;
    int N = 0, R = 0, T = 2;
    const float* div[2] = {nullptr, nullptr};  // T = 3: the rows' factors
    float mul[2] = {1.0f, 1.0f};               // what v's columns lack, by part
    float* y = nullptr;                        // fp32 [position][ldy], columns part * N on
    size_t ldy = 0, v_elems = 0, y_elems = 0;
};
cudaError_t launch_lr_odd(const LrOdd& a, int tiles, int parts, cudaStream_t s);

int lr_max_tiles(int M, int slots);
cudaError_t launch_lr_tokgrad(LrTokGrads& a, int nc, int num_sms, cudaStream_t s);
cudaError_t launch_lr_shrink(const LrShrink& a, int nc, bool trans, int tiles, int zs, int num_sms, cudaStream_t s);
cudaError_t launch_lr_expand(const LrExpand& a, int rc, bool trans, int tiles, int zs, cudaStream_t s);
cudaError_t launch_lr_shrink_few(const LrFew& a, int M, cudaStream_t s);
cudaError_t launch_lr_expand_few(const LrFew& a, int M, int zs, cudaStream_t s);
cudaError_t launch_lr_swiglu_raw(const LrSwiGLU& a, cudaStream_t s);
// With ents: the GEMM's lists too, the entries {first, count} of each 256-token
// tile and the entries' slots (at most lr_max_entries of them), and odd_rows, the
// value of odd at each position's slot (0: no slot).
cudaError_t launch_lr_plan(const int* ids, int M, int slots, const int* rank, int* perm, int4* tiles, int* n_tiles,
                           int2* ents, int* ent_slot, const int* odd, int* odd_rows, cudaStream_t s);
inline int lr_max_entries(int M, int slots) { return (M + 255) / 256 + std::min(slots, M); }
// rows[p] = x[perm[p]] of K bf16 values (a multiple of 8).
cudaError_t launch_lr_gather(const void* x, const int* perm, int M, int K, void* rows, cudaStream_t s);
cudaError_t launch_lr_pack(const LrPack& a, cudaStream_t s);

}  // namespace qmlp
