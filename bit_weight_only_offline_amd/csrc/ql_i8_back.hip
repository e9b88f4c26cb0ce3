// Backward products with frozen per-channel INT8 weights on the fp16 matrix cores.
//
//   linear   dx[m, k] = sum_n dy[m, n] s[n] q[n, k]
//   gated    du = dh act(g),  dg = dh u act'(g)  (one pass), then the same product over the
//            rows of both weights, up and gate tiles alternating as they are packed
//
// The product contracts over the weight's rows, across the direction it is packed in, and
// needs it in fp16.  A workgroup therefore turns each 32-row step of its weight columns
// into operand order once, through LDS, for all of its rows of dy: a thread takes the four
// inputs of one 32-bit word from four consecutive channels, and since a byte permute picks
// any byte of a word, the transposition costs no shuffles of its own.
//
// int8 codes are exact in fp16, the channel scales are not: they are folded into dy (or du
// and dg) in float32, in the pass that forms the product's operand.  That pass rounds the
// scaled gradient once, to fp16's eleven bits: an eighth of the error of the bf16 result's own
// rounding, so that the result is as good as one from a float32 operand.  (bf16 has eight
// bits, and as much error again as the result: 0.0023 in place of 0.0017 against 64 bits.)
// What fp16 lacks is range, which each row therefore gets by itself: it is scaled by a power
// of two, exact both ways, that takes its largest finite value to 2^14 .. 2^15 (the part of a
// row that one split contracts over, where the contraction is split).  Values down
// to 2^-28 of the row's largest keep eleven bits, smaller ones lose them one by one, and the
// sums stay below 2^43.  (Scaling the codes instead needs no pass over dy, but a
// multiplication and a rounding for every code in the inner loop, where decoding is what
// keeps the matrix cores waiting.)
//
// From memory, 2048 x 4096 x 14336 takes 208 to 217 us between cards: 10 for the operand and 198
// to 206 for the product, 1.17 to 1.21 PFLOP/s on 448 tiles, 1.75 rounds of the 256 compute units.
// Gated 2048 x 14336 x 4096 takes 467 to 476: 77 for du, dg and the operand (411 MB, memory-bound),
// 376 to 385 for the product, 1.25 to 1.28 PFLOP/s in two splits on all compute units at once, 13 to
// join them.  The matrix cores are busy for 63% of the cycles, at 2.18 GHz; power bounds them rather
// than decoding, which takes 6 instructions for four codes (11 for bf16, at the same times): with
// all codes zero the call takes 188 us where it takes 201 to 207 with random ones.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_i8.hpp"
#include "ql_launch.hpp"
#include "ql_lds_limit.hpp"

namespace ql {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

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

// LDS: operand rows [MP][64] fp16 (two steps; 128-byte runs, whole cache lines), two stages;
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
    // uses last (216 us against 220 for 2048 x 4096 x 14336 from memory; the smaller tiles read
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
    // bits of 2^10 is the fp16 number 2^10 + u, and 2^10 + 128 less gives q exactly.  One
    // permute takes the bytes of two channels, one XOR makes both numbers of them (0x80 turns
    // q into u), one subtraction both codes.
    auto decode = [&](Packed &p, int u, int b) {
        u32x2 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t two =
                __builtin_amdgcn_perm(p.w[2 * i + 1], p.w[2 * i], 0x0C040C00u | uint32_t(b) * 0x10001u) ^ 0x64806480u;
            o[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, two) - f16x2{(_Float16)1152.0f, (_Float16)1152.0f});
        }
        lds_store8(store_at[b], u & 1, o);
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
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w[j]),
                                                                   __builtin_bit_cast(f16x8, x[i]), acc[j][i], 0, 0, 0);
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

    // exponents of this lane's rows, ahead of the loop where there are registers for them
    int ex[MT];
    auto read_ex = [&] {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = m0 + (wm * MT + i) * 16 + c;
            ex[i] = m < a.M ? -a.ex[int64_t(SPLIT ? blockIdx.y : 0) * a.M + m] : 0;
        }
    };
    if (MT < 8) read_ex();

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
    if (MT == 8) read_ex();
    wait_vmcnt<0>();
    ring_barrier();                                  // LDS is free for the output rows
    // the rows' powers of two taken back
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][i][r] = __builtin_amdgcn_ldexpf(acc[j][i][r], ex[i]);

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

// Adds the splits' float32 sums in split order and rounds: a thread takes four inputs at a time.
__global__ void __launch_bounds__(256) i8_back_join_kernel(const float *__restrict__ part, uint16_t *__restrict__ dx,
                                                           int64_t n4, int ks) {
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < n4; e += int64_t(gridDim.x) * 256) {
        f32x4 t{0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < ks; ++k) {
            const f32x4 p = reinterpret_cast<const f32x4 *>(part)[int64_t(k) * n4 + e];
            t += p;
        }
        reinterpret_cast<u32x2 *>(dx)[e] = u32x2{pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3])};
    }
}

// ---- the operand -----------------------------------------------------------------------
// Groups of eight consecutive channels of a row.  Rows of dh, raw, dy and draw start at any
// element; of a group that the row ends in (`left` of it exist) the rest is zero.
__device__ inline u32x4 load8(const uint16_t *row, int64_t n, int64_t left) {
    if (left >= 8) return *reinterpret_cast<const u32x4_any *>(row + n);
    u32x4 v{0u, 0u, 0u, 0u};
    if (n >= 8) {
        // the row's last eight, moved to the front
        const u32x4 w = *reinterpret_cast<const u32x4_any *>(row + n + left - 8);
        const int gone = 8 - int(left), words = gone >> 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = 0; i + d < 4; ++d) v[i] |= words == d ? w[i + d] : 0u;
        }
        if (gone & 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (v[i] >> 16) | (i < 3 ? v[(i + 1) & 3] << 16 : 0u);
        return v;
    }
#pragma unroll 1
    for (int e = 0; e < left; ++e) {
        const uint32_t w = uint32_t(row[e]) << (16 * (e & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] |= (e >> 1) == i ? w : 0u;
    }
    return v;
}
__device__ inline void store8(uint16_t *p, int64_t left, const float (&v)[8]) {
    const u32x4 o{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    if (left >= 8) {
        *reinterpret_cast<u32x4_any *>(p) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) p[e] = uint16_t(o[e >> 1] >> (16 * (e & 1)));
    }
}
__device__ inline void unpack8(const u32x4 &r, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bf16_bits_to_f32((r[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
}

// TPR threads form the rows of the product's operand, one row at a time, from
//   plain  dy [M, N]:                    dy s
//   gated  dh [M, N], raw [M, 2N]:       [du us | dg gs], and draw = [du | dg] in bf16
// in packed tile order (zero past N) as fp16, and of each row the part of split blockIdx.y:
// scaled by a power of two that takes its largest finite value into [2^14, 2^15), whose exponent
// goes to `ex`.  (By splits, so that few rows too are spread over many compute units: the pass
// for gated 1 x 14336 takes 4.1 us, 7.8 with a workgroup for the whole row.)  A group stays in
// registers in float32 between the maximum and the rounding (NV groups a thread; NV = 0:
// rows of any length, read and formed again, and draw written the second time).  The threads
// walk the rows: their channels' scales stay in registers, and the next row is on its way
// while this one's maximum is found.
template <bool GATED, int TPR, int NV>
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR, 4) back_operand_kernel(I8BackOperand a) {
    struct Scales {
        f32x4 s[GATED ? 2 : 1][2];
    };
    constexpr int ROWS = TPR == 64 ? 4 : 1, KINDS = GATED ? 2 : 1, WAVES = TPR / 64;
    __shared__ float red[2][16];
    // this thread's groups: t, t + TPR, .. below `groups`
    const int64_t first = int64_t(blockIdx.y) * a.groups, t = first + threadIdx.x % TPR;
    const int64_t groups = min(a.Np / 8, first + a.groups);
    int32_t *const ex_out = a.ex + int64_t(blockIdx.y) * a.M;
    int turn = 0;
    // the operand's KINDS x 8 values of group j, and (draw) the stores of du and dg
    auto form = [&](int64_t m, int64_t j, const u32x4 (&in)[GATED ? 3 : 1], const Scales &s, bool draw, float (&v)[KINDS][8]) {
        const int64_t n = 8 * j, left = a.N - n;
        float d[8];
        unpack8(in[0], d);
        if constexpr (GATED) {
            float u[8], g[8];
            unpack8(in[1], u);
            unpack8(in[2], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float f, df;
                gate_act_grad(g[e], a.act, f, df);
                v[0][e] = d[e] * f;
                v[1][e] = d[e] * u[e] * df;
            }
            if (draw && left > 0) {
                store8(a.draw + m * 2 * a.N + n, left, v[0]);
                store8(a.draw + m * 2 * a.N + a.N + n, left, v[1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[0][e] = d[e];
        }
#pragma unroll
        for (int k = 0; k < KINDS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= s.s[k][e >> 2][e & 3];      // zero times zero past N
    };
    auto scales = [&](int64_t j, Scales &s) {
        const float *p = a.s + (GATED ? (j / 2) * 2 * TILE_N + 8 * (j & 1) : 8 * j);
#pragma unroll
        for (int k = 0; k < KINDS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) s.s[k][h] = *reinterpret_cast<const f32x4 *>(p + k * TILE_N + 4 * h);
    };
    auto fetch = [&](int64_t m, int64_t j, u32x4 (&in)[GATED ? 3 : 1]) {
        const int64_t n = 8 * j, left = a.N - n;
#pragma unroll
        for (int k = 0; k < (GATED ? 3 : 1); ++k) in[k] = u32x4{0u, 0u, 0u, 0u};
        if (j >= groups || left <= 0) return;
        in[0] = load8(a.dy + m * a.N, n, left);
        if constexpr (GATED) {
            in[1] = load8(a.raw + m * 2 * a.N, n, left);
            in[2] = load8(a.raw + m * 2 * a.N + a.N, n, left);
        }
    };
    auto largest = [&](const float (&v)[KINDS][8], float &top) {
#pragma unroll
        for (int k = 0; k < KINDS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = fabsf(v[k][e]);
                top = w < INFINITY ? fmaxf(top, w) : top;
            }
    };
    auto put = [&](int64_t m, int64_t j, const float (&v)[KINDS][8], int ex) {
        const int64_t n = 8 * j;
        uint16_t *const op = a.operand + m * KINDS * a.Np + (GATED ? (n / TILE_N) * 2 * TILE_N + n % TILE_N : n);
#pragma unroll
        for (int k = 0; k < KINDS; ++k) {
            f16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (_Float16)__builtin_amdgcn_ldexpf(v[k][e], ex);
            *reinterpret_cast<f16x8 *>(op + k * TILE_N) = o;
        }
    };
    // the exponent for a row's largest value, over the row's threads
    auto exponent = [&](float top) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        if constexpr (WAVES > 1) {
            // two halves in turn: one is written again only past the next row's barrier
            float *const half = red[turn];
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) half[threadIdx.x >> 6] = top;
            __syncthreads();
            top = half[0];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) top = fmaxf(top, half[w]);
        }
        return top > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
    };
    int64_t m = int64_t(blockIdx.x) * ROWS + threadIdx.x / TPR;
    const int64_t by = int64_t(gridDim.x) * ROWS;
    if constexpr (NV > 0) {
        Scales s[NV];
        u32x4 in[NV][GATED ? 3 : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (m < a.M) fetch(m, t + i * TPR, in[i]);
            if (t + i * TPR < groups) scales(t + i * TPR, s[i]);
        }
        for (; m < a.M; m += by) {
            float v[NV][KINDS][8], top = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * TPR < groups) {
                    form(m, t + i * TPR, in[i], s[i], true, v[i]);
                    largest(v[i], top);
                }
            if (m + by < a.M)
#pragma unroll
                for (int i = 0; i < NV; ++i) fetch(m + by, t + i * TPR, in[i]);
            const int ex = exponent(top);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * TPR < groups) put(m, t + i * TPR, v[i], ex);
            if (t == first) ex_out[m] = ex;
        }
    } else {
        for (; m < a.M; m += by) {
            Scales s;
            u32x4 in[GATED ? 3 : 1];
            float v[KINDS][8], top = 0.0f;
            for (int64_t j = t; j < groups; j += TPR) {
                fetch(m, j, in);
                scales(j, s);
                form(m, j, in, s, false, v);
                largest(v, top);
            }
            const int ex = exponent(top);
            for (int64_t j = t; j < groups; j += TPR) {
                fetch(m, j, in);
                scales(j, s);
                form(m, j, in, s, true, v);
                put(m, j, v, ex);
            }
            if (t == first) ex_out[m] = ex;
        }
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

// The operand pass: the fewest threads a row that hold it (its part of a split) in registers, one
// group each of a gated row and two of a plain one, and as many workgroups as the compute units
// hold.
template <bool GATED>
hipError_t launch_operand(const I8BackOperand &a, int ks, hipStream_t st) {
    constexpr int NV = GATED ? 1 : 2;
    const auto grid = [&](int64_t rows, int64_t most) {
        return dim3(unsigned(std::min(ceil_div(a.M, rows), ceil_div(most, ks))), unsigned(ks));
    };
    if (a.groups <= 64 * NV) hipLaunchKernelGGL((back_operand_kernel<GATED, 64, NV>), grid(4, 2048), dim3(256), 0, st, a);
    else if (a.groups <= 128 * NV) hipLaunchKernelGGL((back_operand_kernel<GATED, 128, NV>), grid(1, 4096), dim3(128), 0, st, a);
    else if (a.groups <= 256 * NV) hipLaunchKernelGGL((back_operand_kernel<GATED, 256, NV>), grid(1, 2048), dim3(256), 0, st, a);
    else if (a.groups <= 512 * NV) hipLaunchKernelGGL((back_operand_kernel<GATED, 512, NV>), grid(1, 1024), dim3(512), 0, st, a);
    else if (a.groups <= 1024 * NV) hipLaunchKernelGGL((back_operand_kernel<GATED, 1024, NV>), grid(1, 512), dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((back_operand_kernel<GATED, 1024, 0>), grid(1, 512), dim3(1024), 0, st, a);
    return hipGetLastError();
}

template <int I>
hipError_t launch_back(const I8BackArgs &a, hipStream_t st) {
    constexpr BackCfg t = BACK_CFGS[I];
    constexpr int lds = back_lds(back_rows(t));
    static_assert(lds <= LDS_BYTES_MAX, "the stages fit the LDS");
    const dim3 grid(unsigned(a.mtiles * a.nblocks), unsigned(a.ks)), block(64 * BACK_WAVES);
    if (a.ks == 1) {
        auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, false>;
        static LdsLimit limit;
        const hipError_t e = limit.raise((const void *)kern, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, grid, block, lds, st, a);
        return hipGetLastError();
    }
    auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, true>;
    static LdsLimit limit;
    hipError_t e = limit.raise((const void *)kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, grid, block, lds, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n4 = int64_t(a.M) * a.K / 4;
    hipLaunchKernelGGL(i8_back_join_kernel, elementwise_grid(n4), dim3(256), 0, st, a.part, a.dx, n4, a.ks);
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
        const int64_t mtiles = ceil_div(M, back_rows(BACK_CFGS[c])), threads = mtiles * kblocks * 64 * BACK_WAVES;
        if (c > 0 && threads > LAUNCH_THREADS_MAX) continue;
        for (int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
            const int64_t nps = ceil_div(ceil_div(steps, ks), 4) * 4;      // whole groups of four
            if (ks > 1 && (nps < 8 || ceil_div(steps, nps) < ks)) break;
            float us = float(ceil_div(mtiles * kblocks * ks, 256)) * (float(nps) * STEP_US[c] + START_US);
            if (ks > 1) us += JOIN_US + float(ks) * float(M) * float(L.K) * 8.0f / JOIN_BYTES_PER_US;
            if ((c == 0 && ks == 1) || us < best) {
                best = us;
                p.cfg = c;
                p.mtiles = int(mtiles);
                p.threads = threads;
                p.ks = ks;
                p.nps = int(nps);
            }
        }
    }
    p.operand_bytes = round256(size_t(M) * size_t(p.Np) * (L.gated ? 4 : 2));
    p.ex_bytes = round256(size_t(p.ks) * size_t(M) * 4);
    p.ws_bytes = p.operand_bytes + p.ex_bytes + (p.ks > 1 ? round256(size_t(p.ks) * size_t(M) * size_t(L.K) * 4) : 0);
    return p;
}

hipError_t launch_i8_backward(const I8Layout &L, const I8BackPlan &p, const uint16_t *dy, const uint16_t *raw, int act,
                              int64_t M, const void *pw, const void *ps, uint16_t *dx, uint16_t *draw, void *ws,
                              hipStream_t st) {
    uint8_t *const at = static_cast<uint8_t *>(ws);
    I8BackOperand o{};
    o.dy = dy;
    o.raw = raw;
    o.s = static_cast<const float *>(ps);
    o.draw = draw;
    o.operand = reinterpret_cast<uint16_t *>(at);
    o.ex = reinterpret_cast<int32_t *>(at + p.operand_bytes);
    o.M = M;
    o.N = L.N;
    o.Np = p.Np;
    // a step of the contraction is two packed tiles: 16 channels of a gated weight, 32 of a plain one
    o.groups = p.ks > 1 ? int64_t(p.nps) * (L.gated ? 2 : 4) : p.Np / 8;
    o.act = act;
    const hipError_t e = L.gated ? launch_operand<true>(o, p.ks, st) : launch_operand<false>(o, p.ks, st);
    if (e != hipSuccess) return e;
    I8BackArgs a{};
    a.w = static_cast<const uint8_t *>(pw);
    a.dy = o.operand;
    a.ex = o.ex;
    a.ldy = (L.gated ? 2 : 1) * p.Np;
    a.dx = dx;
    a.part = p.ks > 1 ? reinterpret_cast<float *>(at + p.operand_bytes + p.ex_bytes) : nullptr;
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
