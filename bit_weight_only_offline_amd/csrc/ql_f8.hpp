// Block-scaled e4m3 weights and activations: layout, schedules and launch arguments.
//
// Activations are e4m3 codes (OCP: 448 the largest value, no infinities) [M, K] row-major with one
// float32 scale for each block of 128 inputs of a row; weights e4m3 codes [N, K] with one
// float32 scale for each block of 128 channels by 128 inputs, scales in row-major order.
//
// Device layout of a weight.  Tiles of 16 channels by one block of 128 inputs, 2048 bytes each;
// the blocks of one tile follow each other.  A tile is two halves of 64 inputs; in a half lane l
// of a wavefront owns the 16 bytes at 16 l: channel l mod 16, inputs 16 (l div 16) .. +15 of the
// half.  The two halves of a lane, one after the other, are its operand slice of
// v_mfma_f32_16x16x128_f8f6f4: which 32 inputs of the block a lane group holds does not matter as
// long as the activations' operand holds the same.  Channels past N and inputs past K are zero.
// Experts follow each other.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ql_common.hpp"
#include "ql_i8.hpp"

namespace ql {

constexpr int F8_BLOCK = 128;
constexpr int F8_TILE_BYTES = TILE_N * F8_BLOCK;
constexpr float F8_MAX = 448.0f;

struct F8Layout {
    int64_t E = 1, N = 0, K = 0;
    int64_t ntiles = 0, kblocks = 0, nblocks = 0;   // 16-channel tiles, blocks of inputs and of channels
    size_t w_bytes = 0;                             // of one expert
};

inline F8Layout make_f8_layout(int64_t E, int64_t N, int64_t K) {
    F8Layout L;
    L.E = E;
    L.N = N;
    L.K = K;
    L.ntiles = ceil_div(N, TILE_N);
    L.kblocks = ceil_div(K, F8_BLOCK);
    L.nblocks = ceil_div(N, F8_BLOCK);
    L.w_bytes = size_t(L.ntiles) * size_t(L.kblocks) * F8_TILE_BYTES;
    return L;
}

// Rows of a product.  Plain: `rows` rows of one weight.  Grouped: expert e owns the next counts[e]
// of them, counts on the device.  The workgroups of a grouped product find their rows from the
// counts themselves (find_rows), so that no other launch has to come before.
struct F8Rows {
    const int32_t *counts;   // [E], or null: plain
    int E, rows;
};

// The most row blocks of `block` rows that `rows` rows of E experts can take.
inline int64_t most_row_blocks(int64_t rows, int64_t E, bool grouped, int64_t block) {
    if (!grouped) return ceil_div(rows, block);
    const int64_t part = rows / block + (E < rows ? E : rows);   // each expert ends with at most one short block
    return part < rows ? part : rows;
}

struct F8Plan {
    int cfg = 0;
    int64_t mtiles = 1, nblocks = 1;   // workgroups along the rows (grouped: at most) and the channels
    int ks = 1, bps = 0;               // splits of the input dimension, blocks per split
    int64_t threads = 0;               // of the grid along x
    size_t ws_bytes = 0;               // float32 partial sums of a split [ks][M][16 ntiles]
};

struct F8Args {
    F8Rows r;
    const uint8_t *x;       // codes [M, K]
    const float *xs;        // [M, kblocks]
    const uint8_t *w;       // packed tiles
    const float *ws;        // [E, ceil(N / 128), kblocks]
    const uint16_t *bias;   // bf16 [E, N] or null
    void *out;              // [M, N] bf16 or float32
    float *part;            // partial sums or null
    uint64_t w_stride;      // of an expert, bytes
    int N, K, ntiles, kblocks, nbs;   // nbs: blocks of channels
    int mtiles, nblocks, ks, bps;
    int out_f32;
};

F8Plan make_f8_plan(const F8Layout &L, int64_t M, bool grouped, bool f32);
hipError_t launch_f8_forward(const F8Layout &L, const F8Plan &p, const F8Args &a, hipStream_t st);

// Backward products  dx = sum over channel blocks of scale (dy . codes).
struct F8BackPlan {
    int cfg = 0;
    int64_t mtiles = 1, nblocks = 1;
    int ks = 1, bps = 0;                 // splits of the channels, blocks of 128 per split
    int64_t threads = 0;
    int64_t ldy = 0;                     // channels of a row of the operand
    size_t operand_bytes = 0, ws_bytes = 0;   // a copy of dy in rows of ldy, and all of the workspace
};

struct F8BackArgs {
    F8Rows r;
    const uint16_t *dy;     // bf16 rows of ldy elements
    const uint8_t *w;
    const float *ws;
    uint16_t *dx;           // bf16 [M, K]
    float *part;            // float32 partial sums [ks][M][K] or null
    uint64_t w_stride;
    int64_t ldy;
    int N, K, ntiles, kblocks, nbs;
    int mtiles, nblocks, ks, bps;
};

F8BackPlan make_f8_back_plan(const F8Layout &L, int64_t M, bool grouped);
hipError_t launch_f8_backward(const F8Layout &L, const F8BackPlan &p, const F8BackArgs &a, void *workspace, hipStream_t st);

// Quantisation.
struct F8Quant {
    const void *x;          // [R, K], or [R, 2K] = [up | gate]
    uint8_t *codes;         // [R, K]
    float *scales;          // [R, ceil(K / 128)]
    int64_t R;
    int K;
    int f32, swiglu;
};
hipError_t launch_f8_quantize(const F8Quant &a, hipStream_t st);
hipError_t launch_f8_quantize_backward(const uint16_t *dh, const uint16_t *raw, uint16_t *draw, int64_t R, int K,
                                       hipStream_t st);
hipError_t launch_f8_dequantize(const uint8_t *codes, const float *scales, void *out, int64_t R, int K, bool f32,
                                hipStream_t st);
hipError_t launch_f8_quantize_weight(const F8Layout &L, const void *w, bool f32, uint8_t *codes, float *scales,
                                     hipStream_t st);
hipError_t launch_f8_pack(const F8Layout &L, const uint8_t *codes, uint8_t *packed, hipStream_t st);
hipError_t launch_f8_unpack(const F8Layout &L, const uint8_t *packed, uint8_t *codes, hipStream_t st);

}  // namespace ql
