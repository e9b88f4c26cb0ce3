// Backward products with frozen per-channel INT8 weights on the bf16 matrix cores.
//
//   linear   dx[m, k] = sum_n dy[m, n] s[n] q[n, k]
//   gated    du = dh act(g),  dg = dh u act'(g)  (one pass), then the same product over the
//            rows of both weights, up and gate tiles alternating as they are packed
//
// The product contracts over the weight's rows, across the direction it is packed in, and
// needs it in bf16.  A workgroup therefore turns each 32-row step of its weight columns
// into operand order once, through LDS, for all of its rows of dy: a thread takes the four
// inputs of one 32-bit word from four consecutive channels, and since a byte permute picks
// any byte of a word, the transposition costs no shuffles of its own.
//
// int8 codes are exact in bf16, the channel scales are not: they are folded into dy (or du
// and dg) in float32 before its rounding to bf16, in the pass that forms the product's
// operand.  That rounding is the only one before the float32 sums.  (Scaling the codes
// instead needs no pass over dy, but a multiplication and a rounding for every code in the
// inner loop, where decoding is what keeps the matrix cores waiting.)
//
// From memory, 2048 x 4096 x 14336 takes 213 us: 8 for the operand and 205 for the product,
// 1.17 PFLOP/s on 448 tiles, 1.75 rounds of the 256 compute units.  Gated 2048 x 14336 x 4096
// takes 481: 77 for du, dg and the operand (411 MB, memory-bound), 386 for the product, 1.25
// PFLOP/s in two splits on all compute units at once, 13 to join them.  The matrix cores are
// busy for 58% of the cycles; without any decoding the product would take some 4% less, with
// all data zero 13% less, as the clock then stays at 2.4 GHz in place of 2.17.
#include <hip/hip_runtime.h>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_i8.hpp"
#include "ql_launch.hpp"

namespace ql {
namespace {

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;   // a buffer offset that reads as zero
constexpr int NSTEP = 32;                        // weight rows (contraction) per step
constexpr int BACK_KP = 256, BACK_KQ = 4;        // inputs per workgroup, and chunks of them
constexpr int BACK_WAVES = 8;

// An LDS store of 8 bytes at p, or 16 KiB on (a decoded step's second place).  Written as
// assembly text because the compiler, which cannot tell the stages of the ring apart, would
// wait before every store for the buffer->LDS loads in flight; the step's barrier waits for
// the stores (lgkmcnt), and nothing reads them sooner.
__device__ inline void lds_store8(uint8_t *p, bool second, u32x2 v) {
    static_assert(BACK_KP * 64 == 16384, "the offset below");
    const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)p));
    if (second) asm volatile("ds_write_b64 %0, %1 offset:16384" : : "v"(at), "v"(v) : "memory");
    else asm volatile("ds_write_b64 %0, %1" : : "v"(at), "v"(v) : "memory");
}

// LDS: operand rows [MP][64] bf16 (two steps; 128-byte runs, whole cache lines), two stages;
// packed tiles [2][4] KiB, four; the decoded operand [16][1] KiB, two.
constexpr int back_lds(int mp) { return 2 * mp * 128 + 4 * 8 * 1024 + 2 * BACK_KP * 64; }

// One workgroup: MP = 16 MT WM rows of dy by 256 inputs, the contraction in steps of 32
// packed rows (two tiles).  While step s is multiplied out of registers, the operands of
// step s + 1 are read into registers, each wavefront decodes one of the eight packed tiles
// of step s + 2 (the one it loaded itself), and the buffer->LDS loads of tiles for s + 5 and,
// every other step, of the rows for s + 3 and s + 4 are issued; one barrier a step.
template <int WM, int WN, int MT, int NT, bool SPLIT>
__global__ void __launch_bounds__(64 * BACK_WAVES) i8_back_kernel(I8BackArgs a) {
    static_assert(WM * WN == BACK_WAVES && 16 * NT * WN == BACK_KP, "eight wavefronts over 256 inputs");
    constexpr int MP = 16 * MT * WM;
    constexpr int NA = MP / 8;                       // 1 KiB loads of rows for two steps
    // fewer loads than wavefronts: some are issued twice (the same bytes to the same place),
    // so that all wavefronts wait for the same count
    constexpr int NAW = NA < BACK_WAVES ? 1 : NA / BACK_WAVES;
    constexpr int A_BYTES = MP * 128, R_BYTES = 8 * 1024, D_BYTES = BACK_KP * 64;
    // The largest tile does not wait at a step's barrier for its last two reads of x, which it
    // uses last (213 us against 219.6 for 2048 x 4096 x 14336 from memory; the smaller tiles read
    // up to the end).  Rows loaded over the place those reads take theirs from then need a
    // barrier of their own, every other step.
    constexpr bool LATE = MT == 8;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint8_t *const ldsA = lds, *const ldsR = ldsA + 2 * A_BYTES, *const ldsD = ldsR + 4 * R_BYTES;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;
    const int g = lane >> 4, c = lane & 15;

    // XCD-aware numbering in bands of eight row blocks, as in the forward tile kernel
    const int tiles = a.mtiles * a.nblocks;
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int q8 = tiles >> 3, r8 = tiles & 7;
    const int lin = xcd * q8 + min(xcd, r8) + idx;
    const int band = lin / (8 * a.nblocks), in_band = lin - band * 8 * a.nblocks;
    const int band_rows = min(8, a.mtiles - 8 * band);
    const int mtile = 8 * band + in_band % band_rows, kblock = in_band / band_rows;
    const int m0 = mtile * MP, kq0 = kblock * BACK_KQ;
    const int m_here = min(MP, a.M - m0);

    const int steps = (a.ntiles + 1) / 2;
    const int st0 = SPLIT ? int(blockIdx.y) * a.nps : 0;
    const int st1 = SPLIT ? min(steps, st0 + a.nps) : steps;

    const __amdgpu_buffer_rsrc_t yr =
        make_rsrc(a.dy + int64_t(m0) * a.ldy, uint32_t(m_here) * uint32_t(a.ldy) * 2u);

    // piece p (eight packed rows) of row r of a pair of steps sits at piece p ^ r / 2 mod 8
    // (rows past the end lie past the buffer's range; load q is a fixed distance on from load 0)
    const int y_col = 8 * ((lane & 7) ^ ((lane >> 4) | ((wv & 1) << 2)));
    const uint32_t y_off = (uint32_t((wv % NA) * 8 + (lane >> 3)) * uint32_t(a.ldy) + uint32_t(y_col)) * 2u;
    const uint32_t y_far = uint32_t(BACK_WAVES * 16) * uint32_t(a.ldy);
    // u: the stage's place in the ring, (st - st0) mod 4, a constant where it matters; rows of
    // steps st and st + 1, st - st0 even
    auto issue_y = [&](int q, int st, int u) {
        const uint32_t past = st * NSTEP + y_col < a.ldy ? 0u : OUT_OF_RANGE;
        uint32_t far = st < st1 ? uint32_t(q) * y_far + uint32_t(st) * (NSTEP * 2) : OUT_OF_RANGE;
        asm("" : "+s"(far));           // one scalar: the sum with y_off is not worth a register
        ld128_lds(yr, (y_off + far) | past, ldsA + ((u >> 1) & 1) * A_BYTES + ((wv + BACK_WAVES * q) % NA) * 1024);
    };
    // This wavefront's packed tile of a step: tile wv / 4, chunk wv mod 4.  Its 16-byte piece
    // s lands at slot s ^ s / 16: the words that the 64 lanes read together then lie in 64
    // different banks.
    const int w_tile = wv >> 2, w_ch = wv & 3;
    const uint32_t r_off = kq0 + w_ch < a.kchunks ? uint32_t(kq0 + w_ch) * TILE_BYTES + 16u * (lane ^ (lane >> 4)) : OUT_OF_RANGE;
    auto issue_w = [&](int st, int u) {
        const int tile = 2 * st + w_tile;
        const uint32_t past = st < st1 && tile < a.ntiles ? 0u : OUT_OF_RANGE;
        const __amdgpu_buffer_rsrc_t wr =
            make_rsrc(a.w + int64_t(min(tile, a.ntiles - 1)) * a.kchunks * TILE_BYTES, uint32_t(a.kchunks) * TILE_BYTES);
        ld128_lds(wr, r_off | past, ldsR + (u & 3) * R_BYTES + wv * 1024);
    };

    // Decoding: lane = word j of channels 4 qd .. 4 qd + 3, 16-input group gg of the tile.
    const int dj = lane & 3, dq = (lane >> 2) & 3, dg = lane >> 4;
    struct Packed {
        uint32_t w[4];
    };
    const uint8_t *fetch_at[4];
    uint8_t *store_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        fetch_at[i] = ldsR + wv * 1024 + 4 * dj + 16 * ((dg * 16 + 4 * dq + i) ^ dg);
        store_at[i] = ldsD + ((4 * w_ch + dg) * 64 + (2 * w_tile + (dq >> 1)) * 16 + ((4 * dj + i) ^ dg ^ (dq & 2))) * 16 + (dq & 1) * 8;
    }
    auto fetch = [&](Packed &p, int u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.w[i] = *reinterpret_cast<const uint32_t *>(fetch_at[i] + (u & 3) * R_BYTES);
    };
    // Byte b (input 4 dj + b of the group) of four channels.  A byte u = q + 128 in the low
    // bits of 2^23 is the float 2^23 + u; 2^23 + 128 less gives q exactly, and so does its
    // upper half as bf16.  Permutes and subtractions run at the full vector rate, conversion
    // instructions at a quarter of it.
    uint32_t magic = 0x4B000000u;
    asm("" : "+v"(magic));             // in a vector register, which leaves the selectors scalar
    auto decode = [&](Packed &p, int u, int b) {
        if (b == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.w[i] ^= 0x80808080u;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __uint_as_float(__builtin_amdgcn_perm(magic, p.w[i], 0x07040400u | uint32_t(b))) - 8388736.0f;
        lds_store8(store_at[b], u & 1,
                   u32x2{__builtin_amdgcn_perm(__float_as_uint(v[1]), __float_as_uint(v[0]), 0x07060302u),
                         __builtin_amdgcn_perm(__float_as_uint(v[3]), __float_as_uint(v[2]), 0x07060302u)});
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // x[i] is free again after its group of matrix instructions, so only w needs two sets
    u32x4 x[MT], w0[NT], w1[NT];
    const uint8_t *const x_at[2] = {ldsA + (wm * MT * 16 + c) * 128 + ((g ^ (c >> 1)) * 16),
                                    ldsA + (wm * MT * 16 + c) * 128 + (((4 + g) ^ (c >> 1)) * 16)};
    const uint8_t *w_at[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int kt = wn * NT + j;
        w_at[j] = ldsD + kt * 1024 + (g * 16 + (c ^ (kt & 3) ^ (2 * (g & 1)))) * 16;
    }
    auto read_x = [&](int u, int i) {
        x[i] = *reinterpret_cast<const u32x4 *>(x_at[u & 1] + ((u >> 1) & 1) * A_BYTES + i * 2048);
    };
    auto read_w = [&](u32x4 (&w)[NT], int u, int j) {
        w[j] = *reinterpret_cast<const u32x4 *>(w_at[j] + (u & 1) * D_BYTES);
    };
    auto step = [&](int st, int u, const u32x4 (&w)[NT], u32x4 (&next)[NT]) {
        // Arrived by now: tiles of st + 2, and before an odd step the rows of st + 1.  Issued
        // since: tiles of st + 3 and st + 4, and in an odd step before its tiles the rows.
        if (u & 1) wait_vmcnt<2>();
        else wait_vmcnt<NAW + 2>();
        if constexpr (LATE) {
            // all but the last two reads of x: the stores of the last step, which are older, are
            // done, and so are its reads of w
            asm volatile("s_waitcnt lgkmcnt(2)" : : : "memory");
            __builtin_amdgcn_s_barrier();
            compiler_fence();
        } else {
            ring_barrier();
        }
        Packed p;
        fetch(p, u + 2);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j]),
                                                                    __builtin_bit_cast(bf16x8, x[i]), acc[j][i], 0, 0, 0);
            read_x(u + 1, i);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (LATE ? i == j + 1 : i == ((j + 1) * MT - 1) / NT) read_w(next, u + 1, j);
            // decoding starts behind a group of matrix instructions, under which its words
            // arrive, and ends before the last, under which its stores finish
            constexpr int D0 = MT >= 8 ? 2 : (MT >= 2 ? 1 : 0), D1 = MT >= 8 ? 6 : (MT >= 4 ? 3 : MT);
            if (i >= D0 && i < D1)
#pragma unroll
                for (int b = (i - D0) * 4 / (D1 - D0); b < (i - D0 + 1) * 4 / (D1 - D0); ++b) decode(p, u + 2, b);
            // rows of the pair of steps behind the next one, to the place of the last one
            if (LATE && (u & 1) && i == 3) {
                // this wavefront's last reads of that place are older than the words it has
                // decoded since; past this barrier, so are all the others'
                __builtin_amdgcn_s_barrier();
                compiler_fence();
            }
            if (u & 1)
#pragma unroll
                for (int q = 0; q < NAW; ++q)
                    if (i == (LATE ? 4 + q * (MT - 4) / NAW : ((q + 1) * MT - 1) / NAW)) issue_y(q, st + 3, u + 3);
            if (i == MT - 1) issue_w(st + 5, u + 5);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (st0 < st1) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            issue_w(st0 + u, u);
            if (u % 2 == 0)
#pragma unroll
                for (int q = 0; q < NAW; ++q) issue_y(q, st0 + u, u);
        }
        wait_vmcnt<0>();
        ring_barrier();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            Packed p;
            fetch(p, u);
#pragma unroll
            for (int b = 0; b < 4; ++b) decode(p, u, b);
        }
        ring_barrier();
#pragma unroll
        for (int j = 0; j < NT; ++j) read_w(w0, 0, j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MT; ++i) read_x(0, i);
        __builtin_amdgcn_sched_barrier(0);
        // the slot of step st0's tiles is decoded: those of step st0 + 4 go there
        issue_w(st0 + 4, 0);
        // whole groups of four: steps past the end read as zero and add nothing
        for (int st = st0; st < st1; st += 4) {
            step(st, 0, w0, w1);
            step(st + 1, 1, w1, w0);
            step(st + 2, 2, w0, w1);
            step(st + 3, 3, w1, w0);
        }
    }
    wait_vmcnt<0>();
    ring_barrier();                                  // LDS is free for the output rows

    if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = m0 + (wm * MT + i) * 16 + c;
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int k = kq0 * I8_CHUNK + (wn * NT + j) * 16 + 4 * g;
                if (k < a.K)                          // K is a multiple of 32
                    *reinterpret_cast<f32x4 *>(a.part + (int64_t(blockIdx.y) * a.M + m) * a.K + k) = acc[j][i];
            }
        }
        return;
    }
    // sixteen rows of the wavefront's inputs at a time through its own part of LDS, so that
    // stores are whole 16-byte pieces (as in the forward tile kernel)
    constexpr int PIECES = 2 * NT, STRIDE = NT * 32 + 16, ROWS = 64 / PIECES < 16 ? 64 / PIECES : 16;
    static_assert(BACK_WAVES * 16 * STRIDE <= 4 * R_BYTES, "output rows fit");
    uint8_t *const mine = ldsR + wv * (16 * STRIDE);
    const int p_row = lane / PIECES, k_mine = kq0 * I8_CHUNK + wn * NT * 16 + 8 * (lane % PIECES);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int mi = m0 + (wm * MT + i) * 16;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<u32x2 *>(mine + c * STRIDE + j * 32 + g * 8) =
                u32x2{pack_bf16(acc[j][i][0], acc[j][i][1]), pack_bf16(acc[j][i][2], acc[j][i][3])};
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += ROWS) {
            const int row = r0 + p_row, m = mi + row;
            const u32x4 piece = *reinterpret_cast<const u32x4 *>(mine + (row & 15) * STRIDE + (lane % PIECES) * 16);
            if (p_row < ROWS && m < a.M && k_mine < a.K) *reinterpret_cast<u32x4 *>(a.dx + int64_t(m) * a.K + k_mine) = piece;
        }
    }
}

// Adds the splits' float32 sums in split order and rounds: one thread per four inputs.
__global__ void __launch_bounds__(256) i8_back_join_kernel(const float *__restrict__ part, uint16_t *__restrict__ dx,
                                                           int64_t n4, int ks) {
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= n4) return;
    f32x4 t{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ks; ++k) {
        const f32x4 p = reinterpret_cast<const f32x4 *>(part)[int64_t(k) * n4 + e];
        t += p;
    }
    reinterpret_cast<u32x2 *>(dx)[e] = u32x2{pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3])};
}

// du, dg for V consecutive channels a thread: draw [M, 2N] = [du | dg] in bf16, and the
// product's operand [M][16 ntiles], both scaled by their channels and in packed tile order
// (zero past N).
template <int V>
__global__ void __launch_bounds__(256) gate_back_kernel(const uint16_t *__restrict__ dh, const uint16_t *__restrict__ raw,
                                                        const float *__restrict__ s, uint16_t *__restrict__ draw,
                                                        uint16_t *__restrict__ operand, int64_t M, int64_t N,
                                                        int64_t Np, int act) {
    const int64_t per_row = Np / V, e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= M * per_row) return;
    const int64_t m = e / per_row, n = (e % per_row) * V;
    const int64_t up_at = (n / TILE_N) * 2 * TILE_N + n % TILE_N;    // the gate's 16 further on
    uint16_t *const op = operand + m * 2 * Np + up_at;
    if constexpr (V == 8) {
        u32x4 du{0u, 0u, 0u, 0u}, dg = du, su = du, sg = du;
        if (n < N) {                                                  // N is a multiple of eight
            const u32x4 d = *reinterpret_cast<const u32x4 *>(dh + m * N + n);
            const u32x4 u = *reinterpret_cast<const u32x4 *>(raw + m * 2 * N + n);
            const u32x4 g = *reinterpret_cast<const u32x4 *>(raw + m * 2 * N + N + n);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float o[2], p[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float dv = bf16_bits_to_f32((d[w] >> (16 * b)) & 0xFFFFu);
                    const float uv = bf16_bits_to_f32((u[w] >> (16 * b)) & 0xFFFFu);
                    const float gv = bf16_bits_to_f32((g[w] >> (16 * b)) & 0xFFFFu);
                    float f, df;
                    gate_act_grad(gv, act, f, df);
                    o[b] = dv * f;
                    p[b] = dv * uv * df;
                }
                const float *us = s + up_at + 2 * w, *gs = us + TILE_N;
                du[w] = pack_bf16(o[0], o[1]);
                dg[w] = pack_bf16(p[0], p[1]);
                su[w] = pack_bf16(o[0] * us[0], o[1] * us[1]);
                sg[w] = pack_bf16(p[0] * gs[0], p[1] * gs[1]);
            }
            *reinterpret_cast<u32x4 *>(draw + m * 2 * N + n) = du;
            *reinterpret_cast<u32x4 *>(draw + m * 2 * N + N + n) = dg;
        }
        *reinterpret_cast<u32x4 *>(op) = su;
        *reinterpret_cast<u32x4 *>(op + TILE_N) = sg;
    } else {
        float o = 0.0f, p = 0.0f;
        if (n < N) {
            const float dv = bf16_bits_to_f32(dh[m * N + n]), uv = bf16_bits_to_f32(raw[m * 2 * N + n]);
            const float gv = bf16_bits_to_f32(raw[m * 2 * N + N + n]);
            float f, df;
            gate_act_grad(gv, act, f, df);
            o = dv * f;
            p = dv * uv * df;
            reinterpret_cast<__bf16 *>(draw)[m * 2 * N + n] = (__bf16)o;
            reinterpret_cast<__bf16 *>(draw)[m * 2 * N + N + n] = (__bf16)p;
            o *= s[up_at];
            p *= s[up_at + TILE_N];
        }
        reinterpret_cast<__bf16 *>(op)[0] = (__bf16)o;
        reinterpret_cast<__bf16 *>(op)[TILE_N] = (__bf16)p;
    }
}

// The linear product's operand: dy [M, N] times the channel scales, rows of Np, zero past N.
template <int V>
__global__ void __launch_bounds__(256) scale_back_kernel(const uint16_t *__restrict__ dy, const float *__restrict__ s,
                                                         uint16_t *__restrict__ operand, int64_t M, int64_t N,
                                                         int64_t Np) {
    const int64_t per_row = Np / V, e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= M * per_row) return;
    const int64_t m = e / per_row, n = (e % per_row) * V;
    if constexpr (V == 8) {
        const u32x4 d = *reinterpret_cast<const u32x4 *>(dy + m * N + n);
        u32x4 o;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            o[w] = pack_bf16(bf16_bits_to_f32(d[w] & 0xFFFFu) * s[n + 2 * w], bf16_bits_to_f32(d[w] >> 16) * s[n + 2 * w + 1]);
        *reinterpret_cast<u32x4 *>(operand + m * Np + n) = o;
    } else {
        reinterpret_cast<__bf16 *>(operand)[m * Np + n] = (__bf16)(n < N ? bf16_bits_to_f32(dy[m * N + n]) * s[n] : 0.0f);
    }
}

struct BackCfg { int WM, WN, MT, NT; };
constexpr BackCfg BACK_CFGS[] = {{2, 4, 8, 4}, {2, 4, 4, 4}, {2, 4, 2, 4}, {1, 8, 1, 2}};
constexpr int NUM_BACK_CFGS = 4;
constexpr int back_rows(const BackCfg &t) { return 16 * t.MT * t.WM; }
// Microseconds of a compute unit for one 32-row step of a workgroup, and for its start, first
// operands and stores; of a split's second launch, besides its sums' way to memory and back.
constexpr float STEP_US[NUM_BACK_CFGS] = {0.86f, 0.53f, 0.45f, 0.33f};
constexpr float START_US = 5.0f, JOIN_US = 5.0f, JOIN_BYTES_PER_US = 4.0e6f;

template <int I>
hipError_t launch_back(const I8BackArgs &a, hipStream_t st) {
    constexpr BackCfg t = BACK_CFGS[I];
    constexpr int lds = back_lds(back_rows(t));
    static_assert(lds <= LDS_BYTES_MAX, "the stages fit the LDS");
    const dim3 grid(unsigned(a.mtiles * a.nblocks), unsigned(a.ks)), block(64 * BACK_WAVES);
    if (a.ks == 1) {
        auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, false>;
        static const hipError_t set =
            hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (set != hipSuccess) return set;
        hipLaunchKernelGGL(kern, grid, block, lds, st, a);
        return hipGetLastError();
    }
    auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, true>;
    static const hipError_t set =
        hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (set != hipSuccess) return set;
    hipLaunchKernelGGL(kern, grid, block, lds, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n4 = int64_t(a.M) * a.K / 4;
    hipLaunchKernelGGL(i8_back_join_kernel, dim3(unsigned(ceil_div(n4, 256))), dim3(256), 0, st, a.part, a.dx, n4, a.ks);
    return hipGetLastError();
}

hipError_t launch_back_any(int cfg, const I8BackArgs &a, hipStream_t st) {
    switch (cfg) {
        case 0: return launch_back<0>(a, st);
        case 1: return launch_back<1>(a, st);
        case 2: return launch_back<2>(a, st);
        default: return launch_back<3>(a, st);
    }
}

}  // namespace

// Rows and split whose time is least by the measured rates, as for the forward tiles.
// Measured against every other choice at 1 to 4096 rows, 2000 to 4096 channels and 3008 to
// 14336 inputs, and gated 100 x 5000 x 2080 and 2048 x 14336 x 4096.
I8BackPlan make_i8_back_plan(const I8Layout &L, int64_t M) {
    I8BackPlan p;
    p.Np = L.gated ? ceil_div(L.N, TILE_N) * TILE_N : ceil_div(L.N, 8) * 8;
    const int64_t kblocks = ceil_div(L.kchunks, BACK_KQ), steps = ceil_div(L.ntiles, 2);
    p.nblocks = int(kblocks);
    float best = 0.0f;
    for (int c = 0; c < NUM_BACK_CFGS; ++c) {
        const int64_t mtiles = ceil_div(M, back_rows(BACK_CFGS[c]));
        for (int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
            const int64_t nps = ceil_div(ceil_div(steps, ks), 4) * 4;      // whole groups of four
            if (ks > 1 && (nps < 8 || ceil_div(steps, nps) < ks)) break;
            float us = float(ceil_div(mtiles * kblocks * ks, 256)) * (float(nps) * STEP_US[c] + START_US);
            if (ks > 1) us += JOIN_US + float(ks) * float(M) * float(L.K) * 8.0f / JOIN_BYTES_PER_US;
            if ((c == 0 && ks == 1) || us < best) {
                best = us;
                p.cfg = c;
                p.mtiles = int(mtiles);
                p.ks = ks;
                p.nps = int(nps);
            }
        }
    }
    p.operand_bytes = round256(size_t(M) * size_t(p.Np) * (L.gated ? 4 : 2));
    p.ws_bytes = p.operand_bytes + (p.ks > 1 ? round256(size_t(p.ks) * size_t(M) * size_t(L.K) * 4) : 0);
    return p;
}

hipError_t launch_i8_backward(const I8Layout &L, const I8BackPlan &p, const uint16_t *dy, const uint16_t *raw, int act,
                              int64_t M, const void *pw, const void *ps, uint16_t *dx, uint16_t *draw, void *ws,
                              hipStream_t st) {
    uint16_t *operand = static_cast<uint16_t *>(ws);
    const float *sc = static_cast<const float *>(ps);
    const bool vec = L.N % 8 == 0;
    const dim3 grid(unsigned(ceil_div(M * p.Np / (vec ? 8 : 1), 256)));
    if (L.gated) {
        if (vec) hipLaunchKernelGGL(gate_back_kernel<8>, grid, dim3(256), 0, st, dy, raw, sc, draw, operand, M, L.N, p.Np, act);
        else hipLaunchKernelGGL(gate_back_kernel<1>, grid, dim3(256), 0, st, dy, raw, sc, draw, operand, M, L.N, p.Np, act);
    } else {
        if (vec) hipLaunchKernelGGL(scale_back_kernel<8>, grid, dim3(256), 0, st, dy, sc, operand, M, L.N, p.Np);
        else hipLaunchKernelGGL(scale_back_kernel<1>, grid, dim3(256), 0, st, dy, sc, operand, M, L.N, p.Np);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    I8BackArgs a{};
    a.w = static_cast<const uint8_t *>(pw);
    a.dy = operand;
    a.ldy = (L.gated ? 2 : 1) * p.Np;
    a.dx = dx;
    a.part = p.ks > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.operand_bytes) : nullptr;
    a.M = int(M);
    a.K = int(L.K);
    a.ntiles = int(L.ntiles);
    a.kchunks = int(L.kchunks);
    a.mtiles = p.mtiles;
    a.nblocks = p.nblocks;
    a.ks = p.ks;
    a.nps = p.nps;
    return launch_back_any(p.cfg, a, st);
}

}  // namespace ql
