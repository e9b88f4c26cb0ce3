// Per-channel INT8 weights, the schedules of the products with them, and their launch
// arguments.
//
// Device layout of a per-channel INT8 weight [N, K].  Tiles of 16 output channels by one
// chunk of 64 inputs, 1024 bytes each; the chunks of one tile follow each other.  Inside a
// tile lane l of a wavefront owns the 16 bytes at 16 l: channel l mod 16, inputs
// 16 (l div 16) .. +15 of the chunk, two's complement -- the operand slice that the lane
// feeds to v_mfma_i32_16x16x64_i8, so one 1 KiB load is one operand.  Channels past N and
// inputs past K are zero, which is what makes activations read past a row's end harmless.
// A gated weight (up and gate, N channels each) alternates tiles: tile 2 j holds 16 up
// channels, tile 2 j + 1 the gate channels they are multiplied with, so the wavefront that
// holds the sums of one holds those of the other.  Scales are float32 in tile order.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ql_common.hpp"

namespace ql {

constexpr int I8_CHUNK = 64;
constexpr int64_t I8_K_MAX = 131071;   // 128 * 128 * K < 2^31: the int32 sums cannot wrap
// A launch may have fewer than 2^32 threads in a dimension.  Elementwise passes walk their data
// with a grid of at most 2^30; products refuse the shapes whose tiles no schedule can launch.
constexpr int64_t LAUNCH_THREADS_MAX = (int64_t(1) << 32) - 1;
inline dim3 elementwise_grid(int64_t n) {
    const int64_t blocks = ceil_div(n, 256), most = int64_t(1) << 22;
    return dim3(unsigned(blocks < most ? blocks : most));
}

struct I8Layout {
    int64_t N = 0, K = 0;
    bool gated = false;
    int64_t ntiles = 0;      // 16-channel tiles (gated: up and gate tiles)
    int64_t kchunks = 0;
    size_t w_bytes = 0, s_bytes = 0;
};

inline I8Layout make_i8_layout(int64_t N, int64_t K, bool gated) {
    I8Layout L;
    L.N = N;
    L.K = K;
    L.gated = gated;
    L.ntiles = ceil_div(N, TILE_N) * (gated ? 2 : 1);
    L.kchunks = ceil_div(K, I8_CHUNK);
    L.w_bytes = size_t(L.ntiles) * size_t(L.kchunks) * TILE_BYTES;
    L.s_bytes = round256(size_t(L.ntiles) * TILE_N * 4);
    return L;
}

// Schedules of the forward products.
//   kind 0 (few rows): one workgroup per NT column tiles over the whole input dimension,
//          its WK wavefronts taking the chunks in turn; MT row tiles of 16
//   kind 1 (tiles): WN wavefronts (WM is 1), each MT x NT tiles of 16 x 16, WK times on
//          alternate stages of two chunks; activations staged through LDS, S stages
//   kind 2 (large tiles): WM x WN wavefronts, both operands staged through LDS, S stages of
//          two chunks, each workgroup walking several tiles
struct I8Cfg { int kind, MT, NT, WK, WM, WN, S; };

struct I8Plan {
    int cfg = 0;
    int mtiles = 1, nblocks = 1;
    int ks = 1, cps = 0;         // splits of the input dimension, chunks per split
    int64_t threads = 0;         // of the product's grid along x
    size_t ws_bytes = 0;         // int32 partial sums of a split [ks][M][16 ntiles]
};

struct I8Args {
    const int8_t *x;        // codes [M, K]
    const float *xs;        // token scales [M]
    const uint8_t *w;       // packed tiles
    const float *s;         // channel scales in tile order
    const uint16_t *bias;   // bf16 [N] (gated: [2N] = [up | gate]) or null
    void *out;              // [M, N] bf16 or float32
    uint16_t *raw;          // gated: bf16 [M, 2N] = [up | gate] or null
    int32_t *part;          // partial sums or null
    int M, N, K, ntiles, kchunks;
    int mtiles, nblocks, ks, cps;
    int act, out_f32;
    int pieces;             // rows of out and raw lie on 16-byte boundaries
};

I8Plan make_i8_plan(const I8Layout &L, int64_t M);

// Launch arguments of the pass that forms the operand of a backward product.
struct I8BackOperand {
    const uint16_t *dy;     // bf16 [M, N]: dy, or dh
    const uint16_t *raw;    // gated: bf16 [M, 2N] = [up | gate]
    const float *s;         // channel scales in tile order
    uint16_t *draw;         // gated: bf16 [M, 2N]
    uint16_t *operand;      // fp16 [M, Np] (gated [M, 2Np])
    int32_t *ex;            // [splits][M]
    int64_t M, N, Np;
    int64_t groups;         // of eight channels in a split
    int act;
};

// Launch arguments of the backward products  dx = operand . q.
struct I8BackArgs {
    const uint16_t *dy;     // the operand: scaled gradients, fp16, rows of ldy elements in packed
                            // row order, ldy a multiple of 8, zero past the last channel
    const int32_t *ex;      // [ks][M]: split s of row m is the scaled gradients times 2^ex[s][m]
    const uint8_t *w;
    uint16_t *dx;           // bf16 [M, K]
    float *part;            // float32 partial sums [ks][M][K] or null
    int64_t ldy;
    int M, K, ntiles, kchunks;
    int mtiles, nblocks, ks, nps;   // nps: 32-row steps of the contraction per split
};

struct I8BackPlan {
    int cfg = 0, mtiles = 1, nblocks = 1;
    int ks = 1, nps = 0;
    int64_t threads = 0;                      // of the product's grid along x
    int64_t Np = 0;                           // N rounded up to eight (gated: to a tile)
    size_t operand_bytes = 0, ex_bytes = 0, ws_bytes = 0;   // the operand, its exponents, partial sums
};

I8BackPlan make_i8_back_plan(const I8Layout &L, int64_t M);

hipError_t launch_i8_pack(const I8Layout &L, const int8_t *codes, const float *scales, const int8_t *gate_codes,
                          const float *gate_scales, void *pw, void *ps, hipStream_t st);
hipError_t launch_i8_unpack(const I8Layout &L, const void *pw, const void *ps, int8_t *codes, float *scales,
                            int8_t *gate_codes, float *gate_scales, hipStream_t st);
hipError_t launch_i8_forward(const I8Layout &L, const I8Plan &p, const I8Args &a, hipStream_t st);
hipError_t launch_i8_backward(const I8Layout &L, const I8BackPlan &p, const uint16_t *dy, const uint16_t *raw, int act,
                              int64_t M, const void *pw, const void *ps, uint16_t *dx, uint16_t *draw, void *ws,
                              hipStream_t st);

}  // namespace ql
