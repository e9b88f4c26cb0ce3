// Forward products of block-scaled e4m3 activations and weights on the 8-bit matrix cores, plain or
// over experts.
//
//   y[m, n] = sum over blocks b of (sum over k in b of x[m, k] w[n, k]) xs[m, b] ws[n / 128, b] + bias[n]
//
// A block of 128 inputs is the contraction of one v_mfma_f32_16x16x128_f8f6f4, so a block's sum is one
// instruction from zero, and joining it to the running float32 sum under its scale four fused
// multiply-adds a lane; the two kinds of units work side by side.  The weight is the A
// operand and the activations the B operand: a lane ends up with four consecutive channels of one token,
// so the activation scale is one value a lane and 16 x 16 tile and the weight's one a wavefront, whose
// channels lie in one block of 128.
//
// What that instruction rounds.  It aligns the products of eight inputs (a lane's bytes 8 i .. 8 i + 7) to
// the largest of them and drops what lies below 2^-13 of it, then adds the groups in float32 (measured with
// one large and one small product, place by place).  For normal values its sums are 1.5e-5 off, relative to their size:
// a hundredth of what rounding to bf16 (1.7e-3) does, so products with a bf16 result take it.  Results in float32
// are to be as exact as their type: there the codes, exact in bf16, go through v_mfma_f32_16x16x32_bf16, which sums
// in float32 throughout (1e-7), at half the rate.  So do products of few rows, whose time is
// the weight's way from memory whatever the instruction.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ql_f8_device.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_launch.hpp"
#include "ql_lds_limit.hpp"

namespace ql {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;   // a buffer offset that reads as zero

struct Operand {
    u32x4 lo, hi;                                // inputs 16 g .. of the block's first and second half
};

// One block's sums of 16 channels x 16 tokens.
__device__ inline f32x4 block_product(const Operand &w, const Operand &x) {
    const i32x8 a{int(w.lo[0]), int(w.lo[1]), int(w.lo[2]), int(w.lo[3]), int(w.hi[0]), int(w.hi[1]), int(w.hi[2]), int(w.hi[3])};
    const i32x8 b{int(x.lo[0]), int(x.lo[1]), int(x.lo[2]), int(x.lo[3]), int(x.hi[0]), int(x.hi[1]), int(x.hi[2]), int(x.hi[3])};
    // e4m3 both, no scales of the instruction's own
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
// The codes as bf16: the operand slices of four v_mfma_f32_16x16x32_bf16, eight inputs each.
struct Wide {
    u32x4 part[4];
};
__device__ inline Wide widen(const Operand &o) {
    Wide w;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = (p < 2 ? o.lo : o.hi)[2 * (p & 1) + h];
            w.part[p][2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
            w.part[p][2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
        }
    return w;
}
__device__ inline f32x4 block_product(const Wide &w, const Wide &x) {
    f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < 4; ++p)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.part[p]), __builtin_bit_cast(bf16x8, x.part[p]), s, 0, 0, 0);
    return s;
}
__device__ inline void join(f32x4 &acc, const f32x4 &sum, float scale) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(sum[r], scale, acc[r]);
}

// Channels n .. n + 3 of token m.
__device__ inline void emit(const F8Args &a, int expert, int m, int n, const f32x4 &sum) {
    const int count = a.N - n;
    if (count <= 0) return;
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        v[r] = sum[r] + (a.bias && r < count ? bf16_bits_to_f32(a.bias[int64_t(expert) * a.N + n + r]) : 0.0f);
    const int64_t i = int64_t(m) * a.N + n;
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, v, count);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, v, count);
}

// ---- few rows: the weight streams through registers ----------------------------------
// One workgroup owns NT column tiles over the whole input dimension.  Its WK wavefronts take the
// blocks in turn (block i goes to wavefront i mod WK), so together they read one contiguous run per
// tile; the next block is in flight while one is multiplied (two to four were slower: their registers leave room for
// fewer wavefronts; 32 rows of 8 experts of 28672 x 4096: 149 us, 6.3 TB/s, 177 with two).  The wavefronts' sums
// meet in LDS and are added in a fixed order.
template <int NT, int WK>
__global__ void __launch_bounds__(64 * WK) f8_rows_kernel(F8Args a) {
    extern __shared__ __attribute__((aligned(16))) f32x4 red[];      // [WK][NT][64]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    RowBlock rb;
    int blocks;
    if (!find_rows(a.r, 16, blockIdx.y, lane, rb, blocks)) return;
    const int nt0 = blockIdx.x * NT, nt_here = min(NT, a.ntiles - nt0);

    const __amdgpu_buffer_rsrc_t wr = make_uniform_rsrc(
        a.w + uint64_t(rb.expert) * a.w_stride + int64_t(nt0) * a.kblocks * F8_TILE_BYTES,
        uint32_t(nt_here) * uint32_t(a.kblocks) * F8_TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_uniform_rsrc(a.x + int64_t(rb.first) * a.K, uint32_t(rb.count) * uint32_t(a.K));
    const __amdgpu_buffer_rsrc_t sr = make_uniform_rsrc(a.xs + int64_t(rb.first) * a.kblocks, uint32_t(rb.count) * uint32_t(a.kblocks) * 4u);
    const __amdgpu_buffer_rsrc_t vr = make_uniform_rsrc(
        a.ws + (int64_t(rb.expert) * a.nbs + nt0 * TILE_N / F8_BLOCK) * a.kblocks, uint32_t(a.kblocks) * 4u);

    uint32_t w_off[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        w_off[j] = j < nt_here ? uint32_t(j) * uint32_t(a.kblocks) * F8_TILE_BYTES + 16u * lane : OUT_OF_RANGE;
    const uint32_t x_off = c < rb.count ? uint32_t(c) * uint32_t(a.K) + 16u * g : OUT_OF_RANGE;
    const uint32_t s_off = c < rb.count ? uint32_t(c) * uint32_t(a.kblocks) * 4u : OUT_OF_RANGE;

    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Block {
        Operand w[NT], x;
        uint32_t xs, ws;
    };
    auto load = [&](int it, Block &b) {
        const int kb = it * WK + wv;
        const uint32_t past = kb < a.kblocks ? 0u : OUT_OF_RANGE;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            b.w[j].lo = ld128(wr, (w_off[j] + uint32_t(kb) * F8_TILE_BYTES) | past);
            b.w[j].hi = ld128(wr, (w_off[j] + uint32_t(kb) * F8_TILE_BYTES + 1024u) | past);
        }
        // the next row's codes behind the last input might be NaN: they are not read
        const int k = kb * F8_BLOCK + 16 * g;
        b.x.lo = ld128(xr, k < a.K ? x_off + uint32_t(kb) * F8_BLOCK : OUT_OF_RANGE);
        b.x.hi = ld128(xr, k + 64 < a.K ? x_off + uint32_t(kb) * F8_BLOCK + 64u : OUT_OF_RANGE);
        b.xs = ld32(sr, (s_off + uint32_t(kb) * 4u) | past);
        b.ws = ld32(vr, uint32_t(kb) * 4u | past);
    };
    auto multiply = [&](const Block &b) {
        const float f = __uint_as_float(b.xs) * __uint_as_float(b.ws);
        const Wide x = widen(b.x);
#pragma unroll
        for (int j = 0; j < NT; ++j) join(acc[j], block_product(widen(b.w[j]), x), f);
    };
    const int its = (a.kblocks + WK - 1) / WK;
    Block b0, b1;
    load(0, b0);
    for (int it = 0; it < its; it += 2) {
        if (it + 1 < its) load(it + 1, b1);
        multiply(b0);
        if (it + 1 < its) {
            if (it + 2 < its) load(it + 2, b0);
            multiply(b1);
        }
    }

#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wv * NT + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int e = tid; e < NT * 64; e += 64 * WK) {
        const int l = e & 63, j = e >> 6;
        if ((l & 15) >= rb.count || j >= nt_here) continue;
        f32x4 t = red[j * 64 + l];
#pragma unroll
        for (int w = 1; w < WK; ++w) t += red[(w * NT + j) * 64 + l];
        emit(a, rb.expert, rb.first + (l & 15), (nt0 + j) * TILE_N + 4 * (l >> 4), t);
    }
}

// ---- tiles: activations through LDS, the weight straight to registers ------------------
// WN wavefronts, each all 16 MT tokens x its own NT column tiles, WK times on alternate stages (their
// sums meet in LDS at the end).  No two wavefronts of a group read the same weight tile: packed in operand
// order it goes from memory to the registers it is multiplied from, S stages ahead, and LDS holds and
// serves the activations and their scales.
//
// A stage is a block of 128 inputs: 128-byte runs of the rows, whose 16-byte pieces are swizzled so
// that sixteen rows' pieces spread over all banks.  Operands are read P tiles ahead.  One barrier a stage, P
// tiles before its end: by then every wavefront has read all of the stage's operands and the next stage has
// arrived, so the rows of the stage S on go to this one's place.
//
// 2048 x 4096 x 14336 takes 112 to 129 us by the card, 2.0 PFLOP/s (a library's product with one scale for each tensor
// 130).  Nothing bounds it alone: its loads by themselves take 100 us (48 KiB a stage and compute unit through the caches),
// its matrix instructions 56 to 70; without the joins it takes 111, without the operand reads 103.
//
// Scales come in panels of 32 blocks, 128 bytes of a row (and of the weight's rows of scales), swizzled in the
// same way, the next panel while one is in use.  Taken block by block instead, 64 lanes a load fetched 64 cache
// lines for four bytes of each.
template <int MT>
constexpr int ahead() { return MT >= 8 ? 3 : (MT >= 4 ? 2 : 1); }
template <int MT>
constexpr int x_bytes() { return 16 * MT * F8_BLOCK; }
constexpr int PANEL_BLOCKS = 32;
template <int MT>
constexpr int panel_bytes() { return (16 * MT + 8) * PANEL_BLOCKS * 4; }   // the tokens' rows, and eight of the weight's
template <int NT>
constexpr int out_stride() { return NT * 32 + 16; }
template <int WN, int WK, int MT, int NT, int S>
constexpr int tile_lds() {
    const int ring = S * WK * x_bytes<MT>() + 2 * panel_bytes<MT>(), rows = (WK - 1) * WN * MT * NT * 1024 + WN * 16 * out_stride<NT>();
    return ring > rows ? ring : rows;
}

// Outputs of a wavefront's MT x NT tiles.  A lane holds four channels of a token, eight bytes of
// bf16; sixteen tokens of the wavefront's columns go through LDS (its own part, `mine`), so that the
// stores are whole 16-byte pieces of contiguous runs, which memory takes at any address; element by
// element only where a row ends.
template <int MT, int NT>
__device__ inline void store_tiles(const F8Args &a, const RowBlock &rb, int ct0, const f32x4 (&acc)[NT][MT], uint8_t *mine,
                                   int lane) {
    constexpr int PIECES = 2 * NT, STRIDE = out_stride<NT>(), ROWS = 64 / PIECES < 16 ? 64 / PIECES : 16;
    const int g = lane >> 4, c = lane & 15;
    const int p_row = lane / PIECES, n_mine = ct0 * TILE_N + 8 * (lane % PIECES);
    const int last = rb.first + rb.count;
    f32x4 b[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = (ct0 + j) * TILE_N + 4 * g + r;
            b[j][r] = a.bias && n < a.N ? bf16_bits_to_f32(a.bias[int64_t(rb.expert) * a.N + n]) : 0.0f;
        }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int mi = rb.first + i * 16;
        if (mi >= last) break;
        float v[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[j][r] = acc[j][i][r] + b[j][r];
        if (a.out_f32) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = (ct0 + j) * TILE_N + 4 * g;
                if (mi + c < last && n < a.N) store4_f32(static_cast<float *>(a.out), int64_t(mi + c) * a.N + n, v[j], a.N - n);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<u32x2 *>(mine + c * STRIDE + j * 32 + g * 8) = u32x2{pack_bf16(v[j][0], v[j][1]), pack_bf16(v[j][2], v[j][3])};
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += ROWS) {
            const int row = r0 + p_row, m = mi + row;
            const uint8_t *const from = mine + (row & 15) * STRIDE + (lane % PIECES) * 16;
            const u32x4 piece = *reinterpret_cast<const u32x4 *>(from);
            if (p_row < ROWS && m < last && n_mine < a.N) {
                uint16_t *const to = static_cast<uint16_t *>(a.out) + int64_t(m) * a.N + n_mine;
                if (n_mine + 8 > a.N) {
#pragma unroll 1
                    for (int e = 0; n_mine + e < a.N; ++e) to[e] = reinterpret_cast<const uint16_t *>(from)[e];
                } else {
                    *reinterpret_cast<u32x4_any *>(to) = piece;
                }
            }
        }
    }
}

// EXACT: through the bf16 matrix cores.
template <int WN, int WK, int MT, int NT, int S, bool SPLIT, bool EXACT>
__device__ inline void tile_product(const F8Args &a, const RowBlock &rb, const int nt0, uint8_t *const lds) {
    constexpr int MP = 16 * MT, NTT = NT * WN;
    constexpr int XL = MP / 8 / WN;                        // 1 KiB loads of a block's rows a wavefront
    constexpr int PER_STAGE = XL + 2 * NT;
    constexpr int P = ahead<MT>(), XB = MT >= 4 ? 4 : 2;   // operands read ahead, and buffers for them
    static_assert(XL * WN * 8 == MP && XL >= 1, "loads divide evenly");
    static_assert((S * MT) % XB == 0 && P < XB && P < MT, "buffers come round");
    static_assert(F8_BLOCK % (16 * NT) == 0 && NTT * TILE_N <= 8 * F8_BLOCK, "one weight scale a wavefront and block, eight rows of them");
    static_assert(PANEL_BLOCKS % WK == 0 && PANEL_BLOCKS / WK > 2 * S, "a panel lasts longer than a load takes");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wv / WN, wn = wv % WN;
    const int g = lane >> 4, c = lane & 15;
    const int nt_here = min(NTT, a.ntiles - nt0);

    const int kb0 = SPLIT ? int(blockIdx.y) * a.bps : 0;
    const int nkb = SPLIT ? min(a.kblocks - kb0, a.bps) : a.kblocks;
    const int nst = (nkb + WK - 1) / WK;

    const __amdgpu_buffer_rsrc_t wr = make_uniform_rsrc(
        a.w + uint64_t(rb.expert) * a.w_stride + int64_t(nt0) * a.kblocks * F8_TILE_BYTES,
        uint32_t(nt_here) * uint32_t(a.kblocks) * F8_TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_uniform_rsrc(a.x + int64_t(rb.first) * a.K, uint32_t(rb.count) * uint32_t(a.K));
    const __amdgpu_buffer_rsrc_t sr = make_uniform_rsrc(a.xs + int64_t(rb.first) * a.kblocks, uint32_t(rb.count) * uint32_t(a.kblocks) * 4u);
    const int nb0 = nt0 * TILE_N / F8_BLOCK, nb_here = min((NTT * TILE_N + F8_BLOCK - 1) / F8_BLOCK, a.nbs - nb0);
    const __amdgpu_buffer_rsrc_t vr =
        make_uniform_rsrc(a.ws + (int64_t(rb.expert) * a.nbs + nb0) * a.kblocks, uint32_t(nb_here) * uint32_t(a.kblocks) * 4u);

    const int k_first = kb0 + wk;                          // the wavefront's first block
    // A wavefront's first rows of a block; the others lie a fixed distance on, those past the last past the range.
    static_assert(WN % 2 == 0, "a wavefront's rows have one swizzle");
    const int x_row = wn * 8 + (lane >> 3), x_piece = (lane & 7) ^ ((x_row >> 1) & 7);
    const uint32_t x_off = uint32_t(x_row) * uint32_t(a.K) + uint32_t(k_first) * F8_BLOCK + 16u * uint32_t(x_piece);
    const uint32_t x_far = uint32_t(WN * 8) * uint32_t(a.K);
    const int x_left = a.K - k_first * F8_BLOCK - 16 * x_piece;   // inputs from the piece to the row's end
    uint32_t w_off[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int tile = wn * NT + j;
        w_off[j] = tile < nt_here ? (uint32_t(tile) * uint32_t(a.kblocks) + uint32_t(k_first)) * F8_TILE_BYTES + 16u * lane : OUT_OF_RANGE;
    }
    constexpr int STAGE = x_bytes<MT>();
    uint8_t *const ring = lds + wk * (S * STAGE);
    auto past = [&](int st) { return st * WK + wk < nkb ? 0u : OUT_OF_RANGE; };
    auto load_x = [&](int st, int u) {
        const int on = st * WK;                            // blocks after the first
#pragma unroll
        for (int q = 0; q < XL; ++q)
            ld128_lds(xr, on * F8_BLOCK < x_left ? (x_off + uint32_t(q) * x_far + uint32_t(on) * F8_BLOCK) | past(st) : OUT_OF_RANGE,
                      ring + u * STAGE + (wn + WN * q) * 1024);
    };
    uint8_t *const panels = lds + WK * S * STAGE;
    constexpr int PANEL = panel_bytes<MT>();
    // a wavefront's loads of a panel: eight rows each, the last of all the weight's
    constexpr int PL = (MP / 8 + WN * WK) / (WN * WK);
    uint32_t p_off[PL];
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        const int unit = wv + q * WN * WK, row = 8 * unit + (lane >> 3), mine = unit < MP / 8 ? row : row - MP;
        p_off[q] = mine < (unit < MP / 8 ? rb.count : nb_here)
                       ? (uint32_t(mine) * uint32_t(a.kblocks) + uint32_t(kb0 + 4 * ((lane & 7) ^ (row & 7)))) * 4u
                       : OUT_OF_RANGE;
    }
    auto load_panel = [&](int at) {                        // blocks 32 at .. of this split
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const int unit = wv + q * WN * WK;
            uint8_t *const to = panels + (at & 1) * PANEL + unit * 1024;
            if (unit < MP / 8) ld128_lds(sr, p_off[q] + uint32_t(at) * (PANEL_BLOCKS * 4), to);
            else if (unit == MP / 8) ld128_lds(vr, p_off[q] + uint32_t(at) * (PANEL_BLOCKS * 4), to);
        }
    };
    Operand w[S][NT], x[XB];
    auto load_w = [&](int st, int u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t off = w_off[j] + uint32_t(st * WK) * F8_TILE_BYTES;
            w[u][j].lo = ld128(wr, off | past(st));
            w[u][j].hi = ld128(wr, (off + 1024u) | past(st));
        }
    };
    const uint8_t *const x_at[2] = {ring + c * 128 + ((g ^ (c >> 1)) * 16), ring + c * 128 + (((4 + g) ^ (c >> 1)) * 16)};
    // token tile q of the stage st in place u, those past its last from the next stage, with their scales
    float f[XB], v;                                        // the tokens' scales, the weight's of a block
    const int v_row = (nt0 + wn * NT) * TILE_N / F8_BLOCK - nb0;
    auto scale_at = [&](int st, int row) {                 // of rows with the same low bits as `row`
        const int block = st * WK + wk, word = block & (PANEL_BLOCKS - 1);
        return panels + (block / PANEL_BLOCKS & 1) * PANEL + (((word >> 2) ^ (row & 7)) * 16) + (word & 3) * 4;
    };
    auto read_x = [&](int st, int u, int q) {
        const int at = (q < MT ? u : (u + 1) % S) * STAGE + q % MT * 2048, to = (u * MT + q) % XB;
        x[to].lo = *reinterpret_cast<const u32x4 *>(x_at[0] + at);
        x[to].hi = *reinterpret_cast<const u32x4 *>(x_at[1] + at);
        f[to] = *reinterpret_cast<const float *>(scale_at(q < MT ? st : st + 1, c) + c * 128 + q % MT * 2048);
    };
    auto read_v = [&](int st) { v = *reinterpret_cast<const float *>(scale_at(st, v_row) + (MP + v_row) * 128); };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    load_panel(0);
    load_panel(1);
#pragma unroll
    for (int u = 0; u < S; ++u) {
        load_x(u, u);
        __builtin_amdgcn_sched_barrier(0);                 // the waits count loads in this order
        load_w(u, u);
        __builtin_amdgcn_sched_barrier(0);
    }
    wait_vmcnt<(S - 1) * PER_STAGE>();
    ring_barrier();
#pragma unroll
    for (int i = 0; i < P; ++i) read_x(0, 0, i);
    read_v(0);

    // Stage st in place u.  A tile's sums are joined while the next tile's instructions run.
    auto stage = [&](int st, int u, bool more) {
        f32x4 sum[2][NT];
        const float w_scale = v;
        float s[2];
        Wide wide[EXACT ? NT : 1];
        if constexpr (EXACT)
#pragma unroll
            for (int j = 0; j < NT; ++j) wide[j] = widen(w[u][j]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (i == MT - P) {
                // the next stage has arrived, those after it may be under way
                if (more) wait_vmcnt<(S - 2) * PER_STAGE>();
                ring_barrier();
                if (more) load_x(st + S, u);
                __builtin_amdgcn_sched_barrier(0);
                read_v(st + 1);
            }
            s[i & 1] = f[(u * MT + i) % XB] * w_scale;
            // past the last block: weights that read as zero, but whatever scales lie there
            if (WK > 1 && past(st)) s[i & 1] = 0.0f;
            if constexpr (EXACT) {
                const Wide xw = widen(x[(u * MT + i) % XB]);
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[i & 1][j] = block_product(wide[j], xw);
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[i & 1][j] = block_product(w[u][j], x[(u * MT + i) % XB]);
            }
            read_x(st, u, i + P);
            __builtin_amdgcn_sched_barrier(0);             // joined first, the last sums would be waited for
            if (i > 0)
#pragma unroll
                for (int j = 0; j < NT; ++j) join(acc[j][i - 1], sum[(i - 1) & 1][j], s[(i - 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (more) load_w(st + S, u);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NT; ++j) join(acc[j][MT - 1], sum[(MT - 1) & 1][j], s[(MT - 1) & 1]);
    };
    int st = 0, panel = 2;
    for (; st + S <= nst; st += S) {
        // Every wavefront has read the scales of stage st - 1: the panel before its own is free.  The next is read C - S
        // stages on at the earliest, and the waits, which count its loads as a stage's, have seen to them by then.
        constexpr int C = PANEL_BLOCKS / WK;
        if (st > (panel - 1) * C) load_panel(panel++);
#pragma unroll
        for (int u = 0; u < S; ++u) stage(st + u, u, true);
    }
    // what is left has been loaded
    wait_vmcnt<0>();
#pragma unroll
    for (int u = 0; u < S - 1; ++u)
        if (st + u < nst) stage(st + u, u, false);
    ring_barrier();                                        // the ring is free for what follows
    if constexpr (WK > 1) {
        // the later groups hand their sums to the first: 1 KiB a tile, 16 bytes a lane
        f32x4 *const at = reinterpret_cast<f32x4 *>(lds) + wn * (MT * NT) * 64 + lane;
        constexpr int GROUP = WN * MT * NT * 64;
        if (wk > 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) at[(wk - 1) * GROUP + (j * MT + i) * 64] = acc[j][i];
        }
        ring_barrier();
        if (wk > 0) return;                                // no barrier follows
#pragma unroll
        for (int k = 0; k < WK - 1; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] += at[k * GROUP + (j * MT + i) * 64];
    }
    const int ct0 = nt0 + wn * NT;
    if constexpr (SPLIT) {
        const int64_t width = int64_t(a.ntiles) * TILE_N;
        float *const part = a.part + int64_t(blockIdx.y) * a.r.rows * width;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (16 * i + c >= rb.count) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (wn * NT + j < nt_here)
                    *reinterpret_cast<f32x4 *>(part + int64_t(rb.first + 16 * i + c) * width + (ct0 + j) * TILE_N + 4 * g) = acc[j][i];
        }
    } else {
        constexpr int SUMS = (WK - 1) * WN * MT * NT * 1024;   // sums of the other groups may still be read
        store_tiles<MT, NT>(a, rb, ct0, acc, lds + SUMS + wn * 16 * out_stride<NT>(), lane);
    }
}

// Which tile a workgroup takes.  Block b runs on XCD b mod 8: each XCD takes one contiguous run of the tile order, and
// the tiles are ordered in bands of eight row blocks, so that the workgroups an XCD runs together share rows and columns
// in its L2.  A grouped product has at most a.mtiles row blocks; the counts say how many.
struct Tiles {
    int mtiles, first, run, at;                            // row blocks; this XCD's run; the workgroup's place on it
    __device__ Tiles(const F8Args &a, int rows, int lane) {
        mtiles = a.mtiles;
        RowBlock none;
        if (a.r.counts) find_rows(a.r, rows, -1, lane, none, mtiles);
        const int tiles = mtiles * a.nblocks, xcd = blockIdx.x & 7, q8 = tiles >> 3, r8 = tiles & 7;
        first = xcd * q8 + min(xcd, r8);
        run = q8 + (xcd < r8 ? 1 : 0);
        at = blockIdx.x >> 3;
    }
    // rows of the run's tile `place`; its block of columns
    __device__ int open(const F8Args &a, int rows, int place, int lane, RowBlock &rb) {
        const int lin = first + place, band = lin / (8 * a.nblocks), in_band = lin - band * 8 * a.nblocks;
        const int band_rows = min(8, mtiles - 8 * band);
        find_rows(a.r, rows, 8 * band + in_band % band_rows, lane, rb, mtiles);
        return in_band / band_rows;
    }
};

template <int WN, int WK, int MT, int NT, int S, bool SPLIT, bool EXACT>
__global__ void __launch_bounds__(64 * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) f8_tile_kernel(F8Args a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    Tiles t(a, 16 * MT, lane);
    if (t.at >= t.run) return;
    RowBlock rb;
    const int column = t.open(a, 16 * MT, t.at, lane, rb);
    tile_product<WN, WK, MT, NT, S, SPLIT, EXACT>(a, rb, column * NT * WN, lds);
}

// Stages of the ring of eight wavefronts of MT x NT tiles.
template <int MT, int NT>
constexpr int large_ring() { return MT == 16 ? 2 : (MT == 8 ? (NT == 2 ? 3 : 4) : (NT == 2 ? 4 : 6)); }

// 128 x 256 and 256 x 256 (TALL), which reads three quarters of the operand bytes and loses more to the ends of rounds and
// experts: 8192 x 4096 x 14336 435 -> 406 us (2.4 PFLOP/s), 8192 x 14336 x 4096 475 -> 426, but 3000 x 4096 x 14336 174 -> 188.
// Its blocks of at most half the rows take the tile of half the rows (1 to 3% of ragged grouped products).  A workgroup fills a compute unit, so an XCD's 32 take the tiles of its run in rounds, and
// a last round of few tiles would leave most of them idle for as long as a whole one takes: its tiles are cut in two (half the
// rows) where they are at most 16, in four (half the columns too) where they are at most 8.  2176 x 4096 x 14336: 186 -> 143
// us, 2900: 192 -> 170, 4500: 291 -> 263; 8192 ragged rows over 8 experts 564 -> 525.
constexpr int XCD_UNITS = 32;
__host__ __device__ constexpr int last_parts(int tiles) { return tiles <= XCD_UNITS / 4 ? 4 : (tiles <= XCD_UNITS / 2 ? 2 : 1); }
constexpr int LAST_MORE = 3 * XCD_UNITS / 4;               // workgroups that cutting adds to an XCD's, at most
template <bool TALL, bool EXACT>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) f8_large_kernel(F8Args a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int MT = TALL ? 16 : 8, HALF = 8 * MT;
    const int lane = threadIdx.x & 63;
    Tiles t(a, 2 * HALF, lane);
    const int last = t.run % XCD_UNITS, whole = t.run - last, parts = last_parts(last);
    if (t.at >= whole + last * parts) return;
    const int part = t.at < whole ? 0 : (t.at - whole) % parts, place = t.at < whole ? t.at : whole + (t.at - whole) / parts;
    RowBlock rb;
    const int column = t.open(a, 2 * HALF, place, lane, rb);
    if (t.at < whole || parts == 1) {
        if (TALL && rb.count <= HALF) tile_product<8, 1, MT / 2, 2, large_ring<MT / 2, 2>(), false, EXACT>(a, rb, column * 16, lds);
        else tile_product<8, 1, MT, 2, large_ring<MT, 2>(), false, EXACT>(a, rb, column * 16, lds);
        return;
    }
    const int down = HALF * (part & 1), right = 8 * (part >> 1);
    rb.first += down;
    rb.count = min(HALF, rb.count - down);
    if (rb.count <= 0 || column * 16 + right >= a.ntiles) return;
    if (parts == 2) tile_product<8, 1, MT / 2, 2, large_ring<MT / 2, 2>(), false, EXACT>(a, rb, column * 16, lds);
    else tile_product<8, 1, MT / 2, 1, large_ring<MT / 2, 1>(), false, EXACT>(a, rb, column * 16 + right, lds);
}
template <int MT>
constexpr int large_lds() {
    const int a = tile_lds<8, 1, MT, 2, large_ring<MT, 2>()>(), b = tile_lds<8, 1, MT / 2, 2, large_ring<MT / 2, 2>()>(),
              c = tile_lds<8, 1, MT / 2, 1, large_ring<MT / 2, 1>()>();
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

// Adds the splits' sums in their order and finishes: a thread takes four channels of one token at a time.
__global__ void __launch_bounds__(256) f8_join_kernel(F8Args a) {
    const int per_row = a.ntiles * 4;
    const int64_t width = int64_t(a.ntiles) * TILE_N, all = int64_t(a.r.rows) * width;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < int64_t(a.r.rows) * per_row; e += int64_t(gridDim.x) * 256) {
        const int m = int(e / per_row), n = int(e % per_row) * 4;
        const float *const p = a.part + int64_t(m) * width + n;
        f32x4 s = *reinterpret_cast<const f32x4 *>(p);
        for (int k = 1; k < a.ks; ++k) s += *reinterpret_cast<const f32x4 *>(p + k * all);
        emit(a, 0, m, n, s);
    }
}

// Schedules.  kind 0 (few rows): NT column tiles a workgroup, WK wavefronts on alternate blocks; kind
// 1 (tiles): WN wavefronts of MT x NT tiles, WK times on alternate blocks, a ring of S stages.
struct F8Cfg { int kind, MT, NT, WK, WN, S; };
constexpr F8Cfg CFGS[] = {
    {0, 1, 1, 8, 1, 0}, {0, 1, 2, 8, 1, 0},
    {1, 8, 2, 1, 8, 3},      // 128 x 256, with a kernel of its own
    {1, 4, 2, 1, 8, 4},      // 64 x 256
    {1, 4, 2, 1, 4, 4},      // 64 x 128
    {1, 4, 1, 2, 4, 4},      // 64 x 64, two groups
    {1, 2, 2, 1, 4, 6},      // 32 x 128
    {1, 2, 1, 2, 4, 6},      // 32 x 64, two groups
    {1, 16, 2, 1, 8, 2},     // 256 x 256, with the same kernel as 2
};
constexpr int NUM_CFGS = 9, FIRST_TILE = 2, TALL_TILE = 8;
// Microseconds that a compute unit takes for one block of a workgroup's tile, and for the tile besides (start, first
// loads, stores); and what a round of 256 workgroups after the first takes of either, less where several share a unit,
// more where the operands of more workgroups pass through the caches.  For results in bf16 and, through the bf16 cores,
// in float32.  Fitted to 60 sizes each, 20 to 8192 x 4096 x 14336, 14336 x 4096, 4096 x 4096, 5001 x 4128 and 2048 x
// 2048, every schedule in one to eight splits, and in bf16 the tiles of 256 columns again to 64 of 200 to 32768 rows.
// The rates of float32 and of the small tiles were fitted before scales came in panels and last rounds were cut.
//
// How the choice compares with the fastest of all schedules, at 60 sizes of the same layers, 20 to 4096 rows: the median is
// the fastest itself.  To bf16 it loses more than 6% at two, 48 x 4096 x 14336 (17.9 against 16.3 us) and 64 x 14336 x 4096
// (13.7 against 12.7); to float32 at two, 33 x 4096 x 4096 (11.4 against 9.5) and 333 x 4096 x 14336 (61.5 against 55.5).
// Grouped products have no sizes in the fit, and the model has no term for the bytes of the experts' weights: 512 equal
// rows over 8 experts of 4096 x 14336 take 110 us, 64 x 128 tiles would 85 (to float32 123 and 91), 8192 rows to float32 960
// against 846 with 128 x 256; 8192 rows to bf16, and 64 experts of 4096 x 7168, take the fastest.
struct F8Rate { float block, tile, tile_more, block_more; };   // zeros: not compared
constexpr F8Rate RATES[2][NUM_CFGS] = {
    {{0.0f, 0.0f, 0.0f, 0.0f}, {0.105f, 5.1f, 0.18f, 1.11f}, {0.87f, 6.6f, 0.8f, 1.15f}, {0.433f, 5.7f, 1.1f, 1.45f},
     {0.296f, 5.6f, 0.12f, 1.05f}, {0.20f, 5.0f, 0.36f, 1.04f}, {0.20f, 5.0f, 0.0f, 1.09f}, {0.104f, 5.15f, 0.1f, 1.2f},
     {1.77f, 7.2f, 1.0f, 0.97f}},
    {{0.0f, 0.0f, 0.0f, 0.0f}, {0.086f, 6.3f, 0.01f, 1.49f}, {1.195f, 18.1f, 0.84f, 1.2f}, {0.629f, 12.6f, 0.24f, 1.73f},
     {0.421f, 7.3f, 0.63f, 0.79f}, {0.337f, 5.6f, 0.53f, 1.04f}, {0.312f, 6.5f, 0.17f, 0.93f}, {0.169f, 6.2f, 0.14f, 1.05f},
     {0.0f, 0.0f, 0.0f, 0.0f}},
};
constexpr float JOIN_US[2] = {4.0f, 3.1f}, JOIN_BYTES_PER_US[2] = {7.8e6f, 2.0e7f};

template <int I>
hipError_t launch_rows(const F8Args &a, hipStream_t st) {
    constexpr F8Cfg t = CFGS[I];
    constexpr size_t lds = size_t(t.WK) * t.NT * 1024;
    hipLaunchKernelGGL((f8_rows_kernel<t.NT, t.WK>), dim3(unsigned(a.nblocks), unsigned(a.mtiles)), dim3(64 * t.WK), lds, st, a);
    return hipGetLastError();
}

template <int I, bool SPLIT, bool EXACT>
hipError_t launch_tiles_of(const F8Args &a, hipStream_t st) {
    constexpr F8Cfg t = CFGS[I];
    constexpr size_t lds = tile_lds<t.WN, t.WK, t.MT, t.NT, t.S>();
    static_assert(lds <= LDS_BYTES_MAX, "fits");
    auto kern = f8_tile_kernel<t.WN, t.WK, t.MT, t.NT, t.S, SPLIT, EXACT>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, int(lds));
    if (e != hipSuccess) return e;
    // each XCD takes one of eight runs of equal length: whole eights of workgroups
    const unsigned grid = unsigned(ceil_div(int64_t(a.mtiles) * a.nblocks, 8) * 8);
    hipLaunchKernelGGL(kern, dim3(grid, unsigned(a.ks)), dim3(64 * t.WN * t.WK), lds, st, a);
    return hipGetLastError();
}

template <bool TALL, bool EXACT>
hipError_t launch_large(const F8Args &a, hipStream_t st) {
    constexpr int lds = large_lds<TALL ? 16 : 8>();
    static_assert(lds <= LDS_BYTES_MAX, "fits");
    auto kern = f8_large_kernel<TALL, EXACT>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, lds);
    if (e != hipSuccess) return e;
    const unsigned grid = unsigned((ceil_div(int64_t(a.mtiles) * a.nblocks, 8) + LAST_MORE) * 8);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(512), lds, st, a);
    return hipGetLastError();
}

template <int I>
hipError_t launch_tiles(const F8Args &a, hipStream_t st) {
    if (a.ks == 1) return a.out_f32 ? launch_tiles_of<I, false, true>(a, st) : launch_tiles_of<I, false, false>(a, st);
    const hipError_t e = a.out_f32 ? launch_tiles_of<I, true, true>(a, st) : launch_tiles_of<I, true, false>(a, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(f8_join_kernel, elementwise_grid(int64_t(a.r.rows) * a.ntiles * 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

// Up to 16 rows, an expert's on average, stream the weight through registers, a workgroup one column tile as long as
// that gives a compute unit at most one (4096 x 14336, one row: 11.4 us against 12.7 with two; 8192 x 8192, eight rows:
// 13.4 against 12.9; 8 experts of 28672 x 4096, 32 rows: 156 against 149).  An expert of more than 16 rows then has its
// weight read again for each further 16, which costs where counts are uneven and the average is near 16: 8 ragged experts of
// 28672 x 4096, 32, 64 and 128 rows, 134, 153 and 216 us (tiles of 32 x 64: 139, 142 and 148); 64 of 4096 x 7168, 256, 512 and
// 1024 rows, 285, 297 and 373 (64 x 256: 289, 293 and 302).  More take the schedule and the split of
// the input dimension whose time is least by the measured rates.  A grouped product's row blocks are taken to
// be half a block an expert more than its rows fill; it is not split.
F8Plan make_f8_plan(const F8Layout &L, int64_t M, bool grouped, bool f32) {
    F8Plan p;
    p.bps = int(L.kblocks);
    const int64_t used = grouped ? std::min(L.E, M) : 1;
    auto columns = [&](const F8Cfg &t) { return ceil_div(L.ntiles, t.NT * t.WN); };
    auto threads = [&](int c) {
        const F8Cfg &t = CFGS[c];
        const int64_t mt = most_row_blocks(M, L.E, grouped, 16 * t.MT);
        return (t.kind == 0 ? columns(t) : (ceil_div(mt * columns(t), 8) + LAST_MORE) * 8) * 64 * t.WK * t.WN;
    };
    const bool rows_fit = most_row_blocks(M, L.E, grouped, 16) <= 65535;    // the grid dimension that holds them
    if (M <= 16 * used && rows_fit) {
        p.cfg = L.ntiles * used <= 256 ? 0 : 1;
    } else {
        float best = 0.0f;
        for (int c = M <= 64 * used && rows_fit ? 1 : FIRST_TILE; c < NUM_CFGS; ++c) {
            const F8Cfg &t = CFGS[c];
            const F8Rate &rate = RATES[f32][c];
            const bool large = c == FIRST_TILE || c == TALL_TILE;
            const int largest = f32 ? FIRST_TILE : TALL_TILE;    // 256 x 256 has no registers for operands as bf16
            if (f32 && c == TALL_TILE) continue;
            if (c != largest && threads(c) > LAUNCH_THREADS_MAX) continue;    // where the largest do not fit, none does
            const int64_t block = 16 * t.MT, mt = grouped ? std::max(used, ceil_div(2 * M + used * block, 2 * block)) : ceil_div(M, block);
            for (int ks : {1, 2, 4, 8}) {
                const int64_t step = t.WK, bps = ks == 1 ? L.kblocks : ceil_div(ceil_div(L.kblocks, ks), step) * step;
                if (ks > 1 && (c < FIRST_TILE || large || grouped || bps < 4 * step || ceil_div(L.kblocks, bps) < ks)) break;
                const int64_t tiles = mt * columns(t) * ks;
                float more = float(ceil_div(tiles, 256) - 1), first = 1.0f;
                if (large && tiles % 256) {      // a last round of few tiles, cut: measured shares of a whole one
                    const int parts = last_parts(int(ceil_div(tiles % 256, 8)));
                    if (tiles < 256) first = parts == 4 ? 0.45f : (parts == 2 ? 0.62f : 1.0f);
                    else more += parts == 4 ? -0.67f : (parts == 2 ? -0.5f : 0.0f);
                }
                float us = (first + more * rate.block_more) * float(bps) * rate.block + (1.0f + more * rate.tile_more) * rate.tile;
                if (ks > 1) us += JOIN_US[f32] + float(ks) * float(M) * float(L.ntiles) * TILE_N * 8.0f / JOIN_BYTES_PER_US[f32];
                if (best == 0.0f || us < best) {
                    best = us;
                    p.cfg = c;
                    p.ks = ks;
                    p.bps = int(bps);
                }
            }
        }
    }
    const F8Cfg &t = CFGS[p.cfg];
    p.mtiles = most_row_blocks(M, L.E, grouped, 16 * t.MT);
    p.nblocks = columns(t);
    p.threads = threads(p.cfg);
    if (p.ks > 1) p.ws_bytes = round256(size_t(p.ks) * size_t(M) * size_t(L.ntiles) * TILE_N * 4);
    return p;
}

hipError_t launch_f8_forward(const F8Layout &L, const F8Plan &p, const F8Args &args, hipStream_t st) {
    F8Args a = args;
    a.w_stride = L.w_bytes;
    a.N = int(L.N);
    a.K = int(L.K);
    a.ntiles = int(L.ntiles);
    a.kblocks = int(L.kblocks);
    a.nbs = int(L.nblocks);
    a.mtiles = int(p.mtiles);
    a.nblocks = int(p.nblocks);
    a.ks = p.ks;
    a.bps = p.bps;
    switch (p.cfg) {
        case 0: return launch_rows<0>(a, st);
        case 1: return launch_rows<1>(a, st);
        case 2: return a.out_f32 ? launch_large<false, true>(a, st) : launch_large<false, false>(a, st);    // never split
        case 3: return launch_tiles<3>(a, st);
        case 4: return launch_tiles<4>(a, st);
        case 5: return launch_tiles<5>(a, st);
        case 6: return launch_tiles<6>(a, st);
        case 7: return launch_tiles<7>(a, st);
        default: return launch_large<true, false>(a, st);                  // bf16 alone
    }
}

}  // namespace ql
