// Forward products with per-channel INT8 weights on the INT8 matrix cores.
//
//   linear   y[m, n] = xs[m] s[n] sum_k x[m, k] q[n, k] + b[n]
//   gated    h[m, n] = act(g) u,  u and g two such products of one x
//
// The sums are exact int32 (K <= 131071), so how the input dimension is split -- over
// wavefronts, over workgroups -- cannot change a result.  They meet float32 once, at the
// end: one rounding of the sum to float32, the two scales, the bias, one rounding to the
// output type.  The weight is the A operand and the activations the B operand of
// v_mfma_i32_16x16x64_i8, so a lane ends up with four consecutive channels of one token
// and stores them together.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_i8.hpp"
#include "ql_launch.hpp"

namespace ql {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;   // a buffer offset that reads as zero

__device__ inline i32x4 mma(const u32x4 &a, const u32x4 &b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Scales and biases of four consecutive channels: tile `tile`, position `at` in it (a
// multiple of four), of which the first `count` exist and whose biases start at `bias_at`.
struct Channels {
    f32x4 s, b;
};
__device__ inline Channels channels(const I8Args &a, int tile, int at, int64_t bias_at, int count) {
    Channels q;
    q.s = *reinterpret_cast<const f32x4 *>(a.s + int64_t(tile) * TILE_N + at);
#pragma unroll
    for (int r = 0; r < 4; ++r) q.b[r] = (a.bias && r < count) ? bf16_bits_to_f32(a.bias[bias_at + r]) : 0.0f;
    return q;
}

// The float32 results of those channels for a token of scale xs whose sums are `sum`.
__device__ inline void scaled(const Channels &q, float xs, const i32x4 &sum, float (&v)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = fmaf(float(sum[r]) * xs, q.s[r], q.b[r]);
}

// Linear: channels n .. n + 3 of token m.
__device__ inline void emit_linear(const I8Args &a, int m, float xs, int n, const Channels &q, const i32x4 &sum) {
    const int count = a.N - n;
    if (count <= 0) return;
    float v[4];
    scaled(q, xs, sum, v);
    const int64_t i = int64_t(m) * a.N + n;
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, v, count, a.vec);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, v, count, a.vec);
}

// Gated: the same of an up and a gate tile.
__device__ inline void emit_gated(const I8Args &a, int m, float xs, int n, const Channels &uq, const Channels &gq,
                                  const i32x4 &up, const i32x4 &gt) {
    const int count = a.N - n;
    if (count <= 0) return;
    float u[4], g[4], h[4];
    scaled(uq, xs, up, u);
    scaled(gq, xs, gt, g);
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = gate_act(g[r], a.act) * u[r];
    const int64_t i = int64_t(m) * a.N + n;
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, h, count, a.vec);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, h, count, a.vec);
    if (a.raw) {
        const int64_t j = int64_t(m) * 2 * a.N + n;
        store4_bf16(a.raw, j, u, count, a.vec);
        store4_bf16(a.raw, j + a.N, g, count, a.vec);
    }
}

// One token's four channels of tile t (gated: of tile pair t), sums from `total(tile)`.
template <bool GATED, typename F>
__device__ inline void emit(const I8Args &a, int m, int t, int at, F total) {
    const int n = t * TILE_N + at, count = a.N - n;
    if constexpr (GATED)
        emit_gated(a, m, a.xs[m], n, channels(a, 2 * t, at, n, count), channels(a, 2 * t + 1, at, int64_t(a.N) + n, count),
                   total(2 * t), total(2 * t + 1));
    else
        emit_linear(a, m, a.xs[m], n, channels(a, t, at, n, count), total(t));
}

// ---- few rows: the weight streams through registers ----------------------------------
// One workgroup owns NT column tiles over the whole input dimension.  Its WK wavefronts
// take the chunks in turn (chunk i goes to wavefront i mod WK), so together they read one
// contiguous run per tile; U chunks are in flight while the U before them are multiplied.
// The wavefronts' int32 sums meet in LDS.
template <int MT, int NT, int WK, int U, bool GATED>
__global__ void __launch_bounds__(64 * WK) i8_rows_kernel(I8Args a) {
    static_assert(!GATED || NT % 2 == 0, "up and gate tiles go together");
    extern __shared__ __attribute__((aligned(16))) i32x4 red[];      // [WK][NT * MT][64]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int nt0 = blockIdx.x * NT, m0 = blockIdx.y * 16 * MT;
    const int nt_here = min(NT, a.ntiles - nt0), m_here = min(16 * MT, a.M - m0);

    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(a.w + int64_t(nt0) * a.kchunks * TILE_BYTES, uint32_t(nt_here) * uint32_t(a.kchunks) * TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + int64_t(m0) * a.K, uint32_t(m_here) * uint32_t(a.K));

    uint32_t w_off[NT], x_off[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        w_off[j] = j < nt_here ? uint32_t(j) * uint32_t(a.kchunks) * TILE_BYTES + 16u * lane : OUT_OF_RANGE;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        x_off[i] = 16 * i + c < m_here ? uint32_t(16 * i + c) * uint32_t(a.K) + 16u * g : OUT_OF_RANGE;

    i32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

    struct Batch {
        u32x4 w[U][NT], x[U][MT];
    };
    auto load = [&](int it, Batch &b) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kc = (it * U + u) * WK + wv;
            const uint32_t past = kc < a.kchunks ? 0u : OUT_OF_RANGE;
#pragma unroll
            for (int j = 0; j < NT; ++j) b.w[u][j] = ld128(wr, (w_off[j] + uint32_t(kc) * TILE_BYTES) | past);
#pragma unroll
            for (int i = 0; i < MT; ++i) b.x[u][i] = ld128(xr, (x_off[i] + uint32_t(kc) * I8_CHUNK) | past);
        }
    };
    auto multiply = [&](const Batch &b) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] = mma(b.w[u][j], b.x[u][i], acc[j][i]);
    };
    const int its = (a.kchunks + WK * U - 1) / (WK * U);
    Batch b0, b1;
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
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) red[(wv * NT * MT + j * MT + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    constexpr int UNITS = (GATED ? NT / 2 : NT) * MT * 64;
    for (int e = tid; e < UNITS; e += 64 * WK) {
        const int l = e & 63, i = (e >> 6) % MT, j = (e >> 6) / MT;
        const int m = m0 + 16 * i + (l & 15), at = 4 * (l >> 4);
        if (m >= a.M || (GATED ? 2 * j : j) >= nt_here) continue;
        emit<GATED>(a, m, (GATED ? nt0 / 2 : nt0) + j, at, [&](int tile) {
            i32x4 t = red[((tile - nt0) * MT + i) * 64 + l];
#pragma unroll
            for (int w = 1; w < WK; ++w) t += red[(w * NT * MT + (tile - nt0) * MT + i) * 64 + l];
            return t;
        });
    }
}

// ---- tiles: both operands staged through LDS ------------------------------------------
// WM x WN wavefronts, each 16 MT tokens x NT column tiles, WK times: the WK groups take
// alternate chunks (64 inputs) and their sums meet in LDS at the end, which keeps a compute
// unit's matrix cores busy where there are too few tiles for several workgroups.  A stage is
// WK chunks of 16 MT WM activation rows and of NT WN weight tiles; S stages form a ring that
// direct buffer->LDS loads fill.  Activation rows are loaded in 64-byte runs; a XOR swizzle of their
// 16-byte pieces, applied to the global address of each lane, spreads the 16 rows of an
// operand read over all banks.  Weight tiles are stored in operand order, so their reads are
// linear.
template <int WM, int WN, int WK, int MT, int NT, int S, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN * WK) i8_tile_kernel(I8Args a) {
    static_assert(!GATED || NT % 2 == 0, "up and gate tiles go together");
    constexpr int W = WM * WN * WK;
    constexpr int MP = 16 * MT * WM, NTT = NT * WN;
    constexpr int XA = MP / 16, XB = NTT;              // 1 KiB loads a chunk
    constexpr int NA = XA * WK, NB = XB * WK;          // and a stage
    // every wavefront issues the same number of loads; where they do not divide evenly some
    // are issued twice (the same bytes to the same place)
    constexpr int NAW = (NA + W - 1) / W, NBW = (NB + W - 1) / W, PER_STAGE = NAW + NBW;
    constexpr int STAGE = (NA + NB) * 1024;
    static_assert(S * STAGE <= LDS_BYTES_MAX && S >= 4 && S <= 6, "ring fits the LDS");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wv / (WM * WN), wm = wv / WN % WM, wn = wv % WN;
    const int g = lane >> 4, c = lane & 15;

    // Block b runs on XCD b mod 8: give each XCD one contiguous run of the tile order, and
    // order the tiles in bands of eight row blocks, so that the workgroups an XCD runs
    // together share rows and columns in its L2.
    const int tiles = a.mtiles * a.nblocks;
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int q8 = tiles >> 3, r8 = tiles & 7;
    const int lin = xcd * q8 + min(xcd, r8) + idx;
    const int band = lin / (8 * a.nblocks), in_band = lin - band * 8 * a.nblocks;
    const int band_rows = min(8, a.mtiles - 8 * band);
    const int mtile = 8 * band + in_band % band_rows, nblock = in_band / band_rows;
    const int m0 = mtile * MP, nt0 = nblock * NTT;
    const int nt_here = min(NTT, a.ntiles - nt0), m_here = min(MP, a.M - m0);

    const int kc0 = SPLIT ? int(blockIdx.y) * a.cps : 0;
    const int nck = SPLIT ? min(a.kchunks - kc0, a.cps) : a.kchunks;   // chunks, and stages of them
    const int nst = (nck + WK - 1) / WK;

    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(a.w + int64_t(nt0) * a.kchunks * TILE_BYTES, uint32_t(nt_here) * uint32_t(a.kchunks) * TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + int64_t(m0) * a.K, uint32_t(m_here) * uint32_t(a.K));

    // load l of a stage: chunk l / XA, 16 rows l mod XA; then chunk l / XB, tile l mod XB
    uint32_t off[PER_STAGE];
#pragma unroll
    for (int q = 0; q < NAW; ++q) {
        const int l = (wv + W * q) % NA, row = (l % XA) * 16 + lane / 4;
        off[q] = row < m_here ? uint32_t(row) * uint32_t(a.K) + uint32_t(kc0 + l / XA) * I8_CHUNK +
                                    16u * uint32_t((lane % 4) ^ row_swizzle(row))
                              : OUT_OF_RANGE;
    }
#pragma unroll
    for (int q = 0; q < NBW; ++q) {
        const int l = (wv + W * q) % NB, tile = l % XB;
        off[NAW + q] = tile < nt_here ? (uint32_t(tile) * uint32_t(a.kchunks) + uint32_t(kc0 + l / XB)) * TILE_BYTES + 16u * lane
                                      : OUT_OF_RANGE;
    }
    // load q of stage st; past the last chunk it reads as zero, so that every step of the
    // loop issues and waits for the same number of loads, and the sums stay as they are
    auto issue = [&](int q, int st, int buf) {
        uint8_t *base = lds + buf * STAGE;
        if (q < NAW) {
            const int l = (wv + W * q) % NA;
            const uint32_t past = st * WK + l / XA < nck ? 0u : OUT_OF_RANGE;
            ld128_lds(xr, (off[q] + uint32_t(st) * (WK * I8_CHUNK)) | past, base + l * 1024);
        } else {
            const int l = (wv + W * (q - NAW)) % NB;
            const uint32_t past = st * WK + l / XB < nck ? 0u : OUT_OF_RANGE;
            ld128_lds(wr, (off[q] + uint32_t(st) * (WK * TILE_BYTES)) | past, base + (NA + l) * 1024);
        }
    };

    i32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

    // A stage's operands in registers.  Reads of the next stage and loads further ahead are
    // spread between the matrix instructions of this one: issued together behind a barrier,
    // by all wavefronts at once, they would leave the matrix cores idle.
    struct Operands {
        u32x4 x[MT], w[NT];
    };
    constexpr int READS = MT + NT;
    const uint32_t x_at = uint32_t((wk * XA + wm * MT) * 1024 + c * 64 + ((g ^ row_swizzle(c)) * 16));
    const uint32_t w_at = uint32_t((NA + wk * XB + wn * NT) * 1024 + lane * 16);
    auto read = [&](Operands &f, const uint8_t *stage, int r) {
        if (r < MT) f.x[r] = *reinterpret_cast<const u32x4 *>(stage + x_at + r * 1024);
        else f.w[r - MT] = *reinterpret_cast<const u32x4 *>(stage + w_at + (r - MT) * 1024);
    };
    auto slot = [](int s, int by) { return s + by >= S ? s + by - S : s + by; };
    // Multiplies stage operands `f` while `next` is read from slot `from` and stage `st` is
    // loaded into slot `to`.
    auto multiply = [&](const Operands &f, Operands &next, int from, int st, int to) {
        const uint8_t *ahead = lds + from * STAGE;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = mma(f.w[j], f.x[i], acc[j][i]);
#pragma unroll
            for (int r = j * READS / (NT - 1); r < (j + 1) * READS / (NT - 1) && r < READS; ++r) read(next, ahead, r);
#pragma unroll
            for (int q = j * PER_STAGE / NT; q < (j + 1) * PER_STAGE / NT; ++q) issue(q, st, to);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // One barrier for two stages.  At the barrier before stages st and st + 1 the operands of
    // st are in registers, st + 1 and st + 2 have arrived, st + 3 .. st + S - 2 are on their
    // way, and the slots of st and of the stage before it are free: st + S - 1 and st + S go
    // there.  Past the last stage loads read as zero and nothing uses what is read.
#pragma unroll
    for (int u = 0; u < S - 1; ++u)
#pragma unroll
        for (int q = 0; q < PER_STAGE; ++q) issue(q, u, u);
    Operands f0, f1;
    wait_vmcnt<(S - 2) * PER_STAGE>();
    ring_barrier();
#pragma unroll
    for (int r = 0; r < READS; ++r) read(f0, lds, r);
    int st = 0, at = 0;                                   // at: slot of stage st
    while (true) {
        wait_vmcnt<(S - 4) * PER_STAGE>();
        ring_barrier();
        multiply(f0, f1, slot(at, 1), st + S - 1, slot(at, S - 1));
        if (st + 1 == nst) break;
        multiply(f1, f0, slot(at, 2), st + S, at);
        st += 2;
        at = slot(at, 2);
        if (st == nst) break;
    }
    wait_vmcnt<0>();
    ring_barrier();                                       // the ring is free for what follows
    if constexpr (WK > 1) {
        // the later groups hand their sums to the first: 1 KiB a tile, 16 bytes a lane
        static_assert((WK - 1) * XA * XB <= S * STAGE / 1024, "sums fit the ring");
        i32x4 *const at = reinterpret_cast<i32x4 *>(lds) + (wm * WN + wn) * (MT * NT) * 64 + lane;
        constexpr int GROUP = WM * WN * MT * NT * 64;
        if (wk > 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) at[(wk - 1) * GROUP + (j * MT + i) * 64] = acc[j][i];
        }
        ring_barrier();
        if (wk > 0) return;                               // no barrier follows
#pragma unroll
        for (int k = 0; k < WK - 1; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] += at[k * GROUP + (j * MT + i) * 64];
    }

    if constexpr (SPLIT) {
        const int64_t width = int64_t(a.ntiles) * TILE_N;
        int32_t *part = a.part + int64_t(blockIdx.y) * a.M * width;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = m0 + (wm * MT + i) * 16 + c;
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int tile = wn * NT + j;
                if (tile < nt_here)
                    *reinterpret_cast<i32x4 *>(part + int64_t(m) * width + (nt0 + tile) * TILE_N + 4 * g) = acc[j][i];
            }
        }
        return;
    }
    // All scales and biases first: behind the first stores their loads could not be shared.
    constexpr int CT = GATED ? NT / 2 : NT;                // channel tiles of the wavefront
    const int ct0 = GATED ? (nt0 + wn * NT) / 2 : nt0 + wn * NT;
    float xs[MT];
    Channels q[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + (wm * MT + i) * 16 + c;
        xs[i] = m < a.M ? a.xs[m] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = (ct0 + (GATED ? j / 2 : j)) * TILE_N + 4 * g;
        q[j] = Channels{};
        if (n < a.N) q[j] = channels(a, nt0 + wn * NT + j, 4 * g, (GATED && (j & 1) ? int64_t(a.N) : 0) + n, a.N - n);
    }
    // A lane holds four channels of a token, eight bytes of bf16.  Sixteen tokens of the
    // wavefront's columns go through LDS (its own part of the ring), so that
    // the stores cover whole 16-byte pieces of contiguous runs of each row: 256 x 256 bf16
    // tiles over 4096 inputs took 505 us a 4096 x 32768 output so, 629 with eight-byte stores,
    // and a gated product that also stores [up | gate] 509 against 721.
    if (a.vec8 && !a.out_f32) {
        constexpr int PIECES = 2 * CT, STRIDE = CT * 32 + 16, KINDS = GATED ? 3 : 1;
        constexpr int ROWS = 64 / PIECES < 16 ? 64 / PIECES : 16;
        // behind the sums of the other groups, which may still be read
        constexpr int SUMS = (WK - 1) * XA * XB * 1024;
        static_assert(SUMS + WM * WN * KINDS * 16 * STRIDE <= S * STAGE, "output rows fit the ring");
        uint8_t *const mine = lds + SUMS + wv * (KINDS * 16 * STRIDE);
        const int kinds = GATED && a.raw ? 3 : 1;
        const int p_row = lane / PIECES, n_mine = ct0 * TILE_N + 8 * (lane % PIECES);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int mi = m0 + (wm * MT + i) * 16;
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                float v[KINDS][4];
                if constexpr (GATED) {
                    scaled(q[2 * t], xs[i], acc[2 * t][i], v[1]);
                    scaled(q[2 * t + 1], xs[i], acc[2 * t + 1][i], v[2]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[0][r] = gate_act(v[2][r], a.act) * v[1][r];
                } else {
                    scaled(q[t], xs[i], acc[t][i], v[0]);
                }
#pragma unroll
                for (int k = 0; k < KINDS; ++k)
                    if (k < kinds)
                        *reinterpret_cast<u32x2 *>(mine + k * 16 * STRIDE + c * STRIDE + t * 32 + g * 8) =
                            u32x2{pack_bf16(v[k][0], v[k][1]), pack_bf16(v[k][2], v[k][3])};
            }
#pragma unroll
            for (int k = 0; k < KINDS; ++k) {
                if (k >= kinds) continue;
                uint16_t *const dst = k == 0 ? static_cast<uint16_t *>(a.out) : a.raw + (k == 1 ? 0 : a.N);
                const int64_t ld = k == 0 ? a.N : 2 * int64_t(a.N);
#pragma unroll
                for (int r0 = 0; r0 < 16; r0 += ROWS) {
                    const int row = r0 + p_row, m = mi + row;
                    const u32x4 piece =
                        *reinterpret_cast<const u32x4 *>(mine + k * 16 * STRIDE + (row & 15) * STRIDE + (lane % PIECES) * 16);
                    if (p_row < ROWS && m < a.M && n_mine < a.N)
                        *reinterpret_cast<u32x4 *>(dst + int64_t(m) * ld + n_mine) = piece;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + (wm * MT + i) * 16 + c;
        if (m >= a.M) continue;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int n = (ct0 + t) * TILE_N + 4 * g;
            if constexpr (GATED) emit_gated(a, m, xs[i], n, q[2 * t], q[2 * t + 1], acc[2 * t][i], acc[2 * t + 1][i]);
            else emit_linear(a, m, xs[i], n, q[t], acc[t][i]);
        }
    }
}

// Adds the splits' int32 sums and finishes: one thread per four channels of one token.
template <bool GATED>
__global__ void __launch_bounds__(256) i8_join_kernel(I8Args a) {
    const int per_row = (GATED ? a.ntiles / 2 : a.ntiles) * 4;
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= int64_t(a.M) * per_row) return;
    const int m = int(e / per_row), q = int(e % per_row), tile = q >> 2, at = 4 * (q & 3);
    const int64_t width = int64_t(a.ntiles) * TILE_N;
    emit<GATED>(a, m, tile, at, [&](int t) {
        i32x4 s{0, 0, 0, 0};
        for (int k = 0; k < a.ks; ++k)
            s += *reinterpret_cast<const i32x4 *>(a.part + (int64_t(k) * a.M + m) * width + int64_t(t) * TILE_N + at);
        return s;
    });
}

constexpr I8Cfg CFGS[] = {
    {0, 1, 1, 8, 1, 1, 0}, {0, 1, 2, 8, 1, 1, 0},      // up to 16 rows, one or two column tiles
    {0, 2, 1, 8, 1, 1, 0}, {0, 2, 2, 8, 1, 1, 0},      // 32 rows
    {1, 8, 4, 1, 2, 4, 5},      // 256 x 256
    {1, 4, 4, 1, 2, 4, 5},      // 128 x 256
    {1, 4, 2, 1, 2, 4, 5},      // 128 x 128
    {1, 2, 2, 1, 2, 4, 6},      // 64 x 128
    {1, 2, 2, 4, 2, 2, 5},      // 64 x 64, four groups
};
constexpr int NUM_CFGS = 9, FIRST_TILE = 4;
// Microseconds that a compute unit takes for one chunk of a workgroup's tile, and for the
// tile besides (start, first loads, stores): from runs with one workgroup a unit over 4096 to
// 14336 inputs.  128 x 128 and 64 x 128 with twice the groups on twice the wavefronts, and
// 64 x 128 tiles of four wavefronts, were slower wherever they were tried.
constexpr float CHUNK_US[NUM_CFGS] = {0, 0, 0.036f, 0.064f, 0.75f, 0.43f, 0.28f, 0.15f, 0.09f};
constexpr float TILE_US = 4.0f, JOIN_US = 5.0f, JOIN_BYTES_PER_US = 4.0e6f;
constexpr int ROWS_U = 4;

template <typename F>
hipError_t allow_lds(F kern, size_t lds) {
    return hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
}

template <int I, bool GATED>
hipError_t launch_rows(const I8Args &a, hipStream_t st) {
    constexpr I8Cfg t = CFGS[I];
    constexpr size_t lds = size_t(t.WK) * t.NT * t.MT * 1024;
    auto kern = i8_rows_kernel<t.MT, t.NT, t.WK, ROWS_U, GATED>;
    static const hipError_t set = allow_lds(kern, lds);
    if (set != hipSuccess) return set;
    hipLaunchKernelGGL(kern, dim3(unsigned(a.nblocks), unsigned(a.mtiles)), dim3(64 * t.WK), lds, st, a);
    return hipGetLastError();
}

template <int I, bool GATED>
hipError_t launch_tiles(const I8Args &a, hipStream_t st) {
    constexpr I8Cfg t = CFGS[I];
    constexpr size_t lds = size_t(t.S) * t.WK * (t.MT * t.WM + t.NT * t.WN) * TILE_BYTES;
    const dim3 grid(unsigned(a.mtiles * a.nblocks), unsigned(a.ks));
    const dim3 block(64 * t.WM * t.WN * t.WK);
    if (a.ks == 1) {
        auto kern = i8_tile_kernel<t.WM, t.WN, t.WK, t.MT, t.NT, t.S, GATED, false>;
        static const hipError_t set = allow_lds(kern, lds);
        if (set != hipSuccess) return set;
        hipLaunchKernelGGL(kern, grid, block, lds, st, a);
        return hipGetLastError();
    }
    auto kern = i8_tile_kernel<t.WM, t.WN, t.WK, t.MT, t.NT, t.S, GATED, true>;
    static const hipError_t set = allow_lds(kern, lds);
    if (set != hipSuccess) return set;
    hipLaunchKernelGGL(kern, grid, block, lds, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t units = int64_t(a.M) * (GATED ? a.ntiles / 2 : a.ntiles) * 4;
    hipLaunchKernelGGL(i8_join_kernel<GATED>, dim3(unsigned(ceil_div(units, 256))), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_any(int cfg, const I8Args &a, hipStream_t st) {
    switch (cfg) {
        // a gated weight's tiles come in pairs
        case 0: if constexpr (GATED) return hipErrorInvalidValue; else return launch_rows<0, false>(a, st);
        case 2: if constexpr (GATED) return hipErrorInvalidValue; else return launch_rows<2, false>(a, st);
        case 1: return launch_rows<1, GATED>(a, st);
        case 3: if constexpr (GATED) return launch_rows<3, true>(a, st); else return hipErrorInvalidValue;
        case 4: return launch_tiles<4, GATED>(a, st);
        case 5: return launch_tiles<5, GATED>(a, st);
        case 6: return launch_tiles<6, GATED>(a, st);
        case 7: return launch_tiles<7, GATED>(a, st);
        default: return launch_tiles<8, GATED>(a, st);
    }
}

}  // namespace

// Up to 16 rows stream the weight through registers, a workgroup one column tile of a plain
// weight as long as that gives a compute unit at most two (4096 x 14336, one row: 10.1 us
// against 10.4 with two tiles; 28672 x 4096, 16 rows: 19.8 against 18.9).  More rows take the
// schedule and the split of the input dimension whose time is least by the measured rates:
// rounds of workgroups over 256 compute units, and for a split the partial sums' way to
// memory and back and a launch.  Measured against every other tile at 17 to 2048 x 4096 x
// 4096 and 14336, 333 x 5001 x 4128, 1500 x 3000 x 2048, and gated 77 x 5003 x 2080, 32 and
// 64 x 14336 x 4096 and 700 x 2000 x 4096, its choice was the fastest or within 6% of it.
I8Plan make_i8_plan(const I8Layout &L, int64_t M) {
    I8Plan p;
    p.cps = int(L.kchunks);
    auto blocks = [&](int c, int64_t &mt, int64_t &nb) {
        const I8Cfg &t = CFGS[c];
        mt = ceil_div(M, 16 * t.MT * t.WM);
        nb = ceil_div(L.ntiles, t.NT * t.WN);
    };
    int64_t mt, nb;
    if (M <= 16) {
        p.cfg = !L.gated && L.ntiles <= 512 ? 0 : 1;
    } else {
        float best = 0.0f;
        for (int c = FIRST_TILE - 1; c < NUM_CFGS; ++c) {
            const bool rows = c < FIRST_TILE;
            if (rows && M > 64) continue;
            const int cfg = rows && !L.gated ? 2 : c;
            blocks(cfg, mt, nb);
            for (int ks : {1, 2, 3, 4, 6, 8}) {
                const int64_t cps = ceil_div(ceil_div(L.kchunks, ks), CFGS[cfg].WK) * CFGS[cfg].WK;
                if (ks > 1 && (rows || cps < 8 * CFGS[cfg].WK || ceil_div(L.kchunks, cps) < ks)) break;
                float us = float(ceil_div(mt * nb * ks, 256)) * (float(rows ? L.kchunks : cps) * CHUNK_US[cfg] + TILE_US);
                if (ks > 1) us += JOIN_US + float(ks) * float(M) * float(L.ntiles) * TILE_N * 8.0f / JOIN_BYTES_PER_US;
                if (best == 0.0f || us < best) {
                    best = us;
                    p.cfg = cfg;
                    p.ks = ks;
                    p.cps = int(cps);
                }
            }
        }
    }
    blocks(p.cfg, mt, nb);
    p.mtiles = int(mt);
    p.nblocks = int(nb);
    if (p.ks > 1) p.ws_bytes = round256(size_t(p.ks) * size_t(M) * size_t(L.ntiles) * TILE_N * 4);
    return p;
}

hipError_t launch_i8_forward(const I8Layout &L, const I8Plan &p, const I8Args &args, hipStream_t st) {
    I8Args a = args;
    a.N = int(L.N);
    a.K = int(L.K);
    a.ntiles = int(L.ntiles);
    a.kchunks = int(L.kchunks);
    a.mtiles = p.mtiles;
    a.nblocks = p.nblocks;
    a.ks = p.ks;
    a.cps = p.cps;
    return L.gated ? launch_any<true>(p.cfg, a, st) : launch_any<false>(p.cfg, a, st);
}

}  // namespace ql
