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

#include <algorithm>
#include <type_traits>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_i8.hpp"
#include "ql_launch.hpp"
#include "ql_lds_limit.hpp"

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
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, v, count);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, v, count);
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
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, h, count);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, h, count);
    if (a.raw) {
        const int64_t j = int64_t(m) * 2 * a.N + n;
        store4_bf16(a.raw, j, u, count);
        store4_bf16(a.raw, j + a.N, g, count);
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

// Outputs of a wavefront's MT x NT tiles: tokens m_first + 16 i + c, channel tiles ct0 ... (c, g:
// the lane's column and row group).  xs(i): the token's scale, ch(j): the channels of tile j.
//
// A lane holds four channels of a token, eight bytes of bf16.  Where rows allow it, sixteen
// tokens of the wavefront's columns go through LDS (`mine`, out_bytes() of the wavefront's
// own), so that the stores cover whole 16-byte pieces of contiguous runs of each row: 256 x
// 256 tiles over 4096 inputs took 505 us for a 4096 x 32768 output so, 629 with eight-byte
// stores, and a gated product that also stores [up | gate] 509 against 721.  STREAM: stores
// that ask the caches to let go of the lines: the large tiles' outputs otherwise push out the
// operands that the other workgroups read (468 against 409 us for 4096 x 32768 x 4096).
// Rows may start anywhere (channel counts off eight): the stores are whole pieces all the same,
// which memory takes at any address, and element by element only where a row ends (333 x 5001
// x 4128 to float32 from memory 15.4 us, 17.0 with elements throughout).  Such stores do not
// cover whole cache lines and are not streamed (gated 1500 x 5001 x 1024 with [up | gate]:
// 27.6 us, 37.7 with streaming stores).
template <int NT, bool GATED>
constexpr int out_stride() { return (GATED ? NT / 2 : NT) * 32 + 16; }
template <int NT, bool GATED>
constexpr int out_bytes() { return 16 * out_stride<NT, GATED>(); }

template <int MT, int NT, bool GATED, bool STREAM, typename X, typename C>
__device__ inline void store_tiles(const I8Args &a, int m_first, int ct0, const i32x4 (&acc)[NT][MT], X xs, C ch,
                                   uint8_t *mine, int lane) {
    constexpr int CT = GATED ? NT / 2 : NT;                // channel tiles of the wavefront
    constexpr int PIECES = 2 * CT, STRIDE = out_stride<NT, GATED>(), KINDS = GATED ? 3 : 1;
    constexpr int ROWS = 64 / PIECES < 16 ? 64 / PIECES : 16;
    const int g = lane >> 4, c = lane & 15;
    const int kinds = GATED && a.raw ? 3 : 1;
    const int p_row = lane / PIECES, n_mine = ct0 * TILE_N + 8 * (lane % PIECES);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int mi = m_first + i * 16;
        float v[KINDS][CT][4];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            if constexpr (GATED) {
                scaled(ch(2 * t), xs(i), acc[2 * t][i], v[1][t]);
                scaled(ch(2 * t + 1), xs(i), acc[2 * t + 1][i], v[2][t]);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[0][t][r] = gate_act(v[2][t][r], a.act) * v[1][t][r];
            } else {
                scaled(ch(t), xs(i), acc[t][i], v[0][t]);
            }
        }
        // one kind (h, up, gate) after another through the same bytes: a wavefront's LDS
        // accesses keep their order
#pragma unroll
        for (int k = 0; k < KINDS; ++k) {
            if (k >= kinds) continue;
            const int64_t ld = k == 0 ? a.N : 2 * int64_t(a.N);
            if (k == 0 && a.out_f32) {
                float *const out = static_cast<float *>(a.out);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const int n = (ct0 + t) * TILE_N + 4 * g;
                    if (mi + c < a.M && n < a.N) store4_f32(out, int64_t(mi + c) * ld + n, v[0][t], a.N - n);
                }
                continue;
            }
            uint16_t *const dst = k == 0 ? static_cast<uint16_t *>(a.out) : a.raw + (k == 1 ? 0 : a.N);
#pragma unroll
            for (int t = 0; t < CT; ++t)
                *reinterpret_cast<u32x2 *>(mine + c * STRIDE + t * 32 + g * 8) =
                    u32x2{pack_bf16(v[k][t][0], v[k][t][1]), pack_bf16(v[k][t][2], v[k][t][3])};
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += ROWS) {
                const int row = r0 + p_row, m = mi + row;
                const uint8_t *const from = mine + (row & 15) * STRIDE + (lane % PIECES) * 16;
                const u32x4 piece = *reinterpret_cast<const u32x4 *>(from);
                if (p_row < ROWS && m < a.M && n_mine < a.N) {
                    uint16_t *const to = dst + int64_t(m) * ld + n_mine;
                    if (n_mine + 8 > a.N) {
#pragma unroll 1
                        for (int e = 0; n_mine + e < a.N; ++e) to[e] = reinterpret_cast<const uint16_t *>(from)[e];
                    } else if (STREAM && a.pieces) {
                        __builtin_nontemporal_store(piece, reinterpret_cast<u32x4 *>(to));
                    } else {
                        *reinterpret_cast<u32x4_any *>(to) = piece;
                    }
                }
            }
        }
    }
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

// The end of a wavefront's MT x NT tiles (tokens from m, tiles from nt, of which those before
// nt_end exist): partial sums of a split, or outputs through `mine`.
template <int MT, int NT, bool GATED, bool SPLIT>
__device__ inline void finish_tiles(const I8Args &a, int m0, int nt, int nt_end, const i32x4 (&acc)[NT][MT], uint8_t *mine,
                                    int lane) {
    const int g = lane >> 4, c = lane & 15;
    if constexpr (SPLIT) {
        const int64_t width = int64_t(a.ntiles) * TILE_N;
        int32_t *part = a.part + int64_t(blockIdx.y) * a.M * width;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = m0 + i * 16 + c;
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (nt + j < nt_end)
                    *reinterpret_cast<i32x4 *>(part + int64_t(m) * width + (nt + j) * TILE_N + 4 * g) = acc[j][i];
        }
    } else {
        // All scales and biases first: behind the first stores their loads could not be shared.
        const int ct0 = GATED ? nt / 2 : nt;
        float xs[MT];
        Channels q[NT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = m0 + i * 16 + c;
            xs[i] = m < a.M ? a.xs[m] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = (ct0 + (GATED ? j / 2 : j)) * TILE_N + 4 * g;
            q[j] = Channels{};
            if (n < a.N) q[j] = channels(a, nt + j, 4 * g, (GATED && (j & 1) ? int64_t(a.N) : 0) + n, a.N - n);
        }
        store_tiles<MT, NT, GATED, false>(a, m0, ct0, acc, [&](int i) { return xs[i]; }, [&](int j) { return q[j]; }, mine, lane);
    }
}

// ---- tiles: activations through LDS, the weight straight to registers ------------------
// WN wavefronts, each all 16 MT tokens x its own NT column tiles, WK times on alternate stages
// (their sums meet in LDS at the end, which keeps a compute unit's matrix cores busy where
// there are too few tiles for several workgroups).  No two wavefronts of a group read the same
// weight tile, so it would gain nothing from LDS: packed in operand order it goes from memory
// to the registers it is multiplied from, S stages ahead, and LDS holds and serves the
// activations alone.  With both staged, LDS traffic was what the small tiles waited for: a
// chunk of a 64 x 128 tile took 0.15 us and takes 0.13, of a 128 x 128 tile 0.28 and 0.235.
// 2048 x 4096 x 14336 from memory went from 107 us to 98.3 (2.45 POP/s: power bounds it),
// 256 x 4096 x 14336 from 29.0 to 24.3, 64 x 8192 x 8192 from 16.4 to 13.5.  The small tiles
// are bound by their 6 to 12 KiB of operands a chunk, about 100 bytes a nanosecond and unit.
//
// A stage is two chunks: 128-byte runs of the rows, pieces swizzled as for the large
// tiles.  One barrier a stage, in its middle: by then every wavefront has read the stage's
// second half into registers and the next stage has arrived, so the loads of the stage S on
// go to this one's place.  The loop takes whole rounds of the ring; the stages left, already
// loaded, follow it without another wait (leaving the loop in the middle instead made the
// compiler wait for loads just issued at the loop's head, where it joins the paths).
template <int WN, int WK, int MT, int NT, int S, bool GATED>
constexpr int tile_lds() {
    const int ring = S * WK * MT * 2048, rows = (WK - 1) * WN * MT * NT * 1024 + WN * out_bytes<NT, GATED>();
    return ring > rows ? ring : rows;
}

template <int WN, int WK, int MT, int NT, int S, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(64 * WN * WK) i8_tile_kernel(I8Args a) {
    static_assert(!GATED || NT % 2 == 0, "up and gate tiles go together");
    constexpr int MP = 16 * MT, NTT = NT * WN;
    constexpr int XL = MP / 8 / WN;                       // 1 KiB loads of rows a wavefront and stage
    constexpr int PER_STAGE = XL + 2 * NT;
    static_assert(XL * WN * 8 == MP && WN % 2 == 0, "loads divide evenly");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wv / WN, wn = wv % WN;
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
    const int nck = SPLIT ? min(a.kchunks - kc0, a.cps) : a.kchunks;
    const int nst = (nck + 2 * WK - 1) / (2 * WK);

    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(a.w + int64_t(nt0) * a.kchunks * TILE_BYTES, uint32_t(nt_here) * uint32_t(a.kchunks) * TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + int64_t(m0) * a.K, uint32_t(m_here) * uint32_t(a.K));

    // Chunks past the last are multiplied with weights that read as zero, so the activations
    // there need only lie in the buffer's range or past it.
    uint32_t x_off[XL], w_off[NT];
#pragma unroll
    for (int q = 0; q < XL; ++q) {
        const int row = (wn + WN * q) * 8 + (lane >> 3), piece = (lane & 7) ^ ((row >> 1) & 7);
        x_off[q] = row < m_here ? uint32_t(row) * uint32_t(a.K) + uint32_t(kc0 + 2 * wk) * I8_CHUNK + 16u * uint32_t(piece)
                                : OUT_OF_RANGE;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int tile = wn * NT + j;
        w_off[j] = tile < nt_here ? (uint32_t(tile) * uint32_t(a.kchunks) + uint32_t(kc0 + 2 * wk)) * TILE_BYTES + 16u * lane
                                  : OUT_OF_RANGE;
    }
    uint8_t *const ring = lds + wk * (S * MP * 128);
    auto load_x = [&](int st, int u) {
        const uint32_t past = st < nst ? 0u : OUT_OF_RANGE;
#pragma unroll
        for (int q = 0; q < XL; ++q)
            ld128_lds(xr, (x_off[q] + uint32_t(st) * (WK * 2 * I8_CHUNK)) | past, ring + u * (MP * 128) + (wn + WN * q) * 1024);
    };
    u32x4 w[S][2][NT], x0[MT], x1[MT];
    auto load_w = [&](int st, int u, int h) {
        const uint32_t past = (st * WK + wk) * 2 + h < nck ? 0u : OUT_OF_RANGE;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            w[u][h][j] = ld128(wr, (w_off[j] + uint32_t(st) * (WK * 2 * TILE_BYTES) + uint32_t(h) * TILE_BYTES) | past);
    };
    const uint8_t *const x_at[2] = {ring + c * 128 + ((g ^ (c >> 1)) * 16), ring + c * 128 + (((4 + g) ^ (c >> 1)) * 16)};

    i32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

#pragma unroll
    for (int u = 0; u < S; ++u) {
        load_x(u, u);
        __builtin_amdgcn_sched_barrier(0);               // the waits count loads in this order
        load_w(u, u, 0);
        __builtin_amdgcn_sched_barrier(0);
        load_w(u, u, 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    wait_vmcnt<(S - 1) * PER_STAGE>();
    ring_barrier();
#pragma unroll
    for (int i = 0; i < MT; ++i) x0[i] = *reinterpret_cast<const u32x4 *>(x_at[0] + i * 2048);
    auto multiply = [&](const u32x4 (&wt)[NT], const u32x4 (&x)[MT], u32x4 (&next)[MT], const uint8_t *from) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][i] = mma(wt[j], x[i], acc[j][i]);
            next[i] = *reinterpret_cast<const u32x4 *>(from + i * 2048);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int st = 0;
    for (; st + S <= nst; st += S) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
            multiply(w[u][0], x0, x1, x_at[1] + u * (MP * 128));
            wait_vmcnt<(S - 2) * PER_STAGE>();
            ring_barrier();
            load_x(st + u + S, u);
            __builtin_amdgcn_sched_barrier(0);
            load_w(st + u + S, u, 0);
            multiply(w[u][1], x1, x0, x_at[0] + (u + 1) % S * (MP * 128));
            load_w(st + u + S, u, 1);
        }
    }
    // what is left has been loaded
    wait_vmcnt<0>();
    ring_barrier();
#pragma unroll
    for (int u = 0; u < S - 1; ++u) {
        if (st + u < nst) {
            multiply(w[u][0], x0, x1, x_at[1] + u * (MP * 128));
            multiply(w[u][1], x1, x0, x_at[0] + (u + 1) * (MP * 128));
        }
    }
    ring_barrier();                                       // the ring is free for what follows
    if constexpr (WK > 1) {
        // the later groups hand their sums to the first: 1 KiB a tile, 16 bytes a lane
        i32x4 *const at = reinterpret_cast<i32x4 *>(lds) + wn * (MT * NT) * 64 + lane;
        constexpr int GROUP = WN * MT * NT * 64;
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
    constexpr int SUMS = (WK - 1) * WN * MT * NT * 1024;   // sums of the other groups may still be read
    finish_tiles<MT, NT, GATED, SPLIT>(a, m0, nt0 + wn * NT, nt0 + nt_here, acc, lds + SUMS + wn * out_bytes<NT, GATED>(), lane);
}

// ---- large tiles ----------------------------------------------------------------------
// Eight wavefronts, each 16 MT tokens x NT column tiles; a workgroup stays on its compute unit
// and walks the tiles (item i, then i + the number of workgroups), so that the loads of the
// next tile's first stages are under way while this tile's outputs are scaled and stored.
//
// A stage is two chunks: 128-byte runs of the activation rows (whole cache lines; a XOR
// swizzle of their 16-byte pieces spreads the 16 rows of an operand read over all banks) and
// two weight tiles of each column tile.  Two stages, one barrier each, in the middle: by then
// every wavefront has read the stage's second half into registers and the next stage has
// arrived, so the loads of the one after go to this stage's place.  Operands are read half a
// stage ahead between the matrix instructions.  At 256 x 256 x 4096 a workgroup, stages of one
// chunk in a ring of five took 54.4 us a tile (64-byte runs), these 52.7.  What bounds the
// loop is power more than any unit: with all codes zero the same instructions take 43 us.
template <int WM, int WN, int MT, int NT>
constexpr int wide_stage() { return 2 * (MT * WM + NT * WN) * 1024; }
template <int WM, int WN, int MT, int NT, bool GATED>
constexpr int wide_lds() { return 2 * wide_stage<WM, WN, MT, NT>() + (16 * MT * WM + 2 * 16 * NT * WN) * 4 + WM * WN * out_bytes<NT, GATED>(); }

template <int WM, int WN, int MT, int NT, bool GATED>
__global__ void __launch_bounds__(64 * WM * WN) i8_wide_kernel(I8Args a) {
    static_assert(!GATED || NT % 2 == 0, "up and gate tiles go together");
    constexpr int W = WM * WN, T = 64 * W;
    constexpr int MP = 16 * MT * WM, NTT = NT * WN, NP = 16 * NTT;
    constexpr int XA = MP / 8, XB = 2 * NTT;               // 1 KiB loads a stage
    static_assert(XA % W == 0 && XB % W == 0 && W % 2 == 0, "every wavefront issues the same loads");
    constexpr int XAW = XA / W, LOADS = XAW + XB / W;
    constexpr int STAGE = wide_stage<WM, WN, MT, NT>();
    static_assert(wide_lds<WM, WN, MT, NT, GATED>() <= LDS_BYTES_MAX && MP <= T && NP <= T, "fits");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    float *const l_xs = reinterpret_cast<float *>(lds + 2 * STAGE), *const l_s = l_xs + MP, *const l_b = l_s + NP;
    uint8_t *const l_out = reinterpret_cast<uint8_t *>(l_b + NP);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;
    const int g = lane >> 4, c = lane & 15;

    // Offsets inside a tile of this wavefront's first loads of rows and of weights; the others
    // are a fixed distance on.  Rows and column tiles past the end lie past the buffers' ranges.
    const int row = wv * 8 + lane / 8, my_chunk = wv & 1;
    const uint32_t x_off = uint32_t(row) * uint32_t(a.K) + 16u * uint32_t((lane % 8) ^ ((row >> 1) & 7));
    const uint32_t w_off = (uint32_t(wv >> 1) * uint32_t(a.kchunks) + uint32_t(my_chunk)) * TILE_BYTES + 16u * lane;
    const uint32_t x_far = uint32_t(W * 8) * uint32_t(a.K), w_far = uint32_t(W / 2) * uint32_t(a.kchunks) * TILE_BYTES;

    struct Item {
        __amdgpu_buffer_rsrc_t xr, wr;
        int m0, nt0;
    };
    // Items in the order of bands of eight row blocks; workgroup b runs on XCD b mod 8 and each
    // XCD takes one contiguous run, so that what it runs together shares rows and columns.
    const int items = a.mtiles * a.nblocks;
    const int xcd = blockIdx.x & 7, q8 = items >> 3, r8 = items & 7;
    const int run = q8 + (xcd < r8 ? 1 : 0), first = xcd * q8 + min(xcd, r8);
    const int per_xcd = (int(gridDim.x) + 7 - xcd) >> 3;   // workgroups on this XCD
    auto open = [&](int at) {
        Item it;
        const bool real = at < run;
        const int tile = real ? first + at : 0;
        const int band = tile / (8 * a.nblocks), in_band = tile - band * 8 * a.nblocks;
        const int band_rows = min(8, a.mtiles - 8 * band);
        it.m0 = (8 * band + in_band % band_rows) * MP;
        it.nt0 = in_band / band_rows * NTT;
        it.xr = make_rsrc(a.x + int64_t(it.m0) * a.K, real ? uint32_t(min(MP, a.M - it.m0)) * uint32_t(a.K) : 0u);
        it.wr = make_rsrc(a.w + int64_t(it.nt0) * a.kchunks * TILE_BYTES,
                          real ? uint32_t(min(NTT, a.ntiles - it.nt0)) * uint32_t(a.kchunks) * TILE_BYTES : 0u);
        return it;
    };
    auto issue = [&](int q, const Item &it, int st, int buf) {
        uint8_t *const base = lds + buf * STAGE + (wv + W * (q < XAW ? q : q - XAW)) * 1024;
        if (q < XAW) {
            uint32_t far = uint32_t(q) * x_far + uint32_t(st) * (2 * I8_CHUNK);
            asm("" : "+s"(far));           // one scalar: the sum with x_off is not worth a register
            ld128_lds(it.xr, x_off + far, base);
        } else {
            // a chunk past the last reads as zero, and so adds nothing whatever its inputs
            uint32_t far = uint32_t(q - XAW) * w_far + uint32_t(st) * (2 * TILE_BYTES);
            if (2 * st + my_chunk >= a.kchunks) far = OUT_OF_RANGE;
            asm("" : "+s"(far));
            ld128_lds(it.wr, w_off + far, base + XA * 1024);
        }
    };
    // The lane number formed anew, where it is used once a tile: the compiler, which cannot
    // see through the empty statement, then keeps neither it nor the addresses that follow from
    // it in registers through the loop, whose operands and sums take all 256.
    auto lane_again = [] {
        uint32_t all = ~0u;
        asm volatile("" : "+s"(all));
        return int(__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0)));
    };
    // the tile's token and channel scales, 64 a wavefront
    auto issue_scales = [&](const Item &it) {
        const int lane = lane_again();
        constexpr int XW = MP / 64, SW = NP / 64;
        static_assert(MP % 64 == 0 && NP % 64 == 0 && XW + SW <= W, "one load a wavefront");
        if (wv < XW)
            ld32_lds(make_rsrc(a.xs + it.m0, uint32_t(min(MP, a.M - it.m0)) * 4u), uint32_t(wv * 64 + lane) * 4u,
                     reinterpret_cast<uint8_t *>(l_xs) + wv * 256);
        else if (wv < XW + SW)
            ld32_lds(make_rsrc(a.s + int64_t(it.nt0) * TILE_N, uint32_t(min(NTT, a.ntiles - it.nt0)) * TILE_N * 4u),
                     uint32_t((wv - XW) * 64 + lane) * 4u, reinterpret_cast<uint8_t *>(l_s) + (wv - XW) * 256);
    };

    struct Operands {
        u32x4 x[MT], w[NT];
    };
    constexpr int READS = MT + NT;
    const uint8_t *const x_at = lds + (wm * MT * 16 + c) * 128, *const w_at = lds + (XA + 2 * wn * NT) * 1024 + lane * 16;
    const int x_half[2] = {(g ^ (c >> 1)) * 16, ((4 + g) ^ (c >> 1)) * 16};
    auto read = [&](Operands &f, int buf, int h, int r) {
        if (r < MT) f.x[r] = *reinterpret_cast<const u32x4 *>(x_at + buf * STAGE + x_half[h] + r * 2048);
        else f.w[r - MT] = *reinterpret_cast<const u32x4 *>(w_at + buf * STAGE + (r - MT) * 2048 + h * 1024);
    };
    i32x4 acc[NT][MT];
    // half a stage: its operands f; reads of half h of buffer `from`; loads of stage st of `it`
    auto multiply = [&](const Operands &f, Operands &next, int from, int h, bool fill, const Item &it, int st, int to) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = mma(f.w[j], f.x[i], acc[j][i]);
#pragma unroll
            for (int r = j * READS / (NT - 1); r < (j + 1) * READS / (NT - 1) && r < READS; ++r) read(next, from, h, r);
            if (fill)
#pragma unroll
                for (int q = j * LOADS / NT; q < (j + 1) * LOADS / NT; ++q) issue(q, it, st, to);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    int at = int(blockIdx.x) >> 3;
    if (at >= run) return;
    Item cur = open(at);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < LOADS; ++q) issue(q, cur, u, u);
    wait_vmcnt<0>();
    ring_barrier();
    Operands f0, f1;
    int buf = 0;
    while (true) {
        const Item next = open(at + per_xcd);
        // at least two stages, so that the next tile's first two are loaded by this one's last
        const int stages = max(2, (a.kchunks + 1) / 2);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < READS; ++r) read(f0, buf, 0, r);
        for (int st = 0; st < stages; ++st) {
            multiply(f0, f1, buf, 1, false, cur, 0, 0);
            // a tile's first two stages had arrived before the last tile's stores, which
            // need not be waited for here
            if (st > 0) wait_vmcnt<0>();
            ring_barrier();
            const bool wrap = st + 2 >= stages;
            const Item &from = wrap ? next : cur;
            multiply(f1, f0, buf ^ 1, 0, true, from, wrap ? st + 2 - stages : st + 2, buf);
            if (st == 0) issue_scales(cur);      // every wavefront is past the last tile's stores
            buf ^= 1;
        }
        if (a.bias && wv * 64 < NP) {
            const int at_b = wv * 64 + lane_again(), tile = cur.nt0 + at_b / TILE_N;
            const int n = (GATED ? tile >> 1 : tile) * TILE_N + at_b % TILE_N;
            l_b[at_b] = n < a.N ? bf16_bits_to_f32(a.bias[(GATED && (tile & 1) ? int64_t(a.N) : 0) + n]) : 0.0f;
        }
        wait_vmcnt<0>();                                   // the next tile's first two stages
        ring_barrier();

        const int out_lane = lane_again();
        const int g = out_lane >> 4, c = out_lane & 15;
        const int ct0 = GATED ? (cur.nt0 + wn * NT) / 2 : cur.nt0 + wn * NT;
        store_tiles<MT, NT, GATED, true>(
            a, cur.m0 + wm * MT * 16, ct0, acc, [&](int i) { return l_xs[(wm * MT + i) * 16 + c]; },
            [&](int j) {
                const int at4 = (wn * NT + j) * TILE_N + 4 * g;
                return Channels{*reinterpret_cast<const f32x4 *>(l_s + at4),
                                a.bias ? *reinterpret_cast<const f32x4 *>(l_b + at4) : f32x4{0.f, 0.f, 0.f, 0.f}};
            },
            l_out + wv * out_bytes<NT, GATED>(), out_lane);
        at += per_xcd;
        if (at >= run) break;
        cur = next;
    }
}

// Adds the splits' int32 sums and finishes: a thread takes four channels of one token at a time.
template <bool GATED>
__global__ void __launch_bounds__(256) i8_join_kernel(I8Args a) {
    const int per_row = (GATED ? a.ntiles / 2 : a.ntiles) * 4;
    const int64_t width = int64_t(a.ntiles) * TILE_N;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < int64_t(a.M) * per_row; e += int64_t(gridDim.x) * 256) {
        const int m = int(e / per_row), q = int(e % per_row), tile = q >> 2, at = 4 * (q & 3);
        emit<GATED>(a, m, tile, at, [&](int t) {
            i32x4 s{0, 0, 0, 0};
            for (int k = 0; k < a.ks; ++k)
                s += *reinterpret_cast<const i32x4 *>(a.part + (int64_t(k) * a.M + m) * width + int64_t(t) * TILE_N + at);
            return s;
        });
    }
}

constexpr I8Cfg CFGS[] = {
    {0, 1, 1, 8, 1, 1, 0}, {0, 1, 2, 8, 1, 1, 0},      // 16 rows, one or two column tiles
    {2, 8, 4, 1, 2, 4, 2},      // 256 x 256
    {1, 8, 2, 1, 1, 8, 3},      // 128 x 256
    {1, 8, 1, 1, 1, 8, 4},      // 128 x 128
    {1, 4, 2, 1, 1, 4, 4},      // 64 x 128
    {1, 4, 1, 2, 1, 4, 4},      // 64 x 64, two groups
    {1, 2, 1, 2, 1, 4, 6},      // 32 x 64, two groups
};
constexpr int NUM_CFGS = 8, WIDE = 2, SHARED = 4;
// Microseconds that a compute unit takes for one chunk of a workgroup's tile, and for the
// tile besides: start, first loads, stores.  From SHARED on workgroups share a unit and hide
// those from each other: a second round's costs nothing, one of the rounds after it two fifths
// (128 x 128) or a fifth.  From runs with one workgroup a unit over 4096 to 14336 inputs and
// with several over 160 to 512.  Also tried, and slower at most sizes: 64 x 128 with two
// groups, 64 x 64 with one or four, 128 x 256 of four wavefronts, rings of up to six stages for
// the larger tiles.
constexpr float CHUNK_US[NUM_CFGS] = {0.039f, 0.039f, 0.75f, 0.36f, 0.235f, 0.13f, 0.087f, 0.06f};
constexpr float TILE_US[NUM_CFGS] = {4.0f, 4.0f, 8.0f, 6.0f, 6.2f, 4.7f, 4.5f, 4.5f};
constexpr float JOIN_US = 5.0f, JOIN_BYTES_PER_US = 4.0e6f;
constexpr int ROWS_U = 4;
constexpr int WIDE_WGS = 256;    // workgroups that walk the large tiles: one a compute unit

template <int I, bool GATED>
hipError_t launch_rows(const I8Args &a, hipStream_t st) {
    constexpr I8Cfg t = CFGS[I];
    constexpr size_t lds = size_t(t.WK) * t.NT * t.MT * 1024;
    auto kern = i8_rows_kernel<t.MT, t.NT, t.WK, ROWS_U, GATED>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, int(lds));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(a.nblocks), unsigned(a.mtiles)), dim3(64 * t.WK), lds, st, a);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_join(const I8Args &a, hipStream_t st) {
    const int64_t units = int64_t(a.M) * (GATED ? a.ntiles / 2 : a.ntiles) * 4;
    hipLaunchKernelGGL(i8_join_kernel<GATED>, elementwise_grid(units), dim3(256), 0, st, a);
    return hipGetLastError();
}

// 256 x 256 either way.  Gated wavefronts take twice the columns and half the rows, so that
// each of h, up and gate leaves in 128-byte lines.
template <int I, bool GATED>
hipError_t launch_wide(const I8Args &a, hipStream_t st) {
    constexpr I8Cfg t = CFGS[I];
    constexpr int WM = GATED ? 2 * t.WM : t.WM, WN = GATED ? t.WN / 2 : t.WN;
    constexpr int MT = GATED ? t.MT / 2 : t.MT, NT = GATED ? 2 * t.NT : t.NT;
    constexpr size_t lds = wide_lds<WM, WN, MT, NT, GATED>();
    auto kern = i8_wide_kernel<WM, WN, MT, NT, GATED>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, int(lds));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(std::min<int64_t>(int64_t(a.mtiles) * a.nblocks, WIDE_WGS))),
                       dim3(64 * WM * WN), lds, st, a);
    return hipGetLastError();
}

template <int I, bool GATED, bool SPLIT>
hipError_t launch_tiles_of(const I8Args &a, hipStream_t st) {
    constexpr I8Cfg t = CFGS[I];
    // a gated weight's tiles come in pairs
    constexpr int NT = GATED && t.NT == 1 ? 2 : t.NT, WN = t.WN * t.NT / NT;
    constexpr size_t lds = tile_lds<WN, t.WK, t.MT, NT, t.S, GATED>();
    auto kern = i8_tile_kernel<WN, t.WK, t.MT, NT, t.S, GATED, SPLIT>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, int(lds));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(a.mtiles * a.nblocks), unsigned(a.ks)), dim3(64 * WN * t.WK), lds, st, a);
    return hipGetLastError();
}

template <int I, bool GATED>
hipError_t launch_tiles(const I8Args &a, hipStream_t st) {
    if (a.ks == 1) return launch_tiles_of<I, GATED, false>(a, st);
    const hipError_t e = launch_tiles_of<I, GATED, true>(a, st);
    return e != hipSuccess ? e : launch_join<GATED>(a, st);
}

template <bool GATED>
hipError_t launch_any(int cfg, const I8Args &a, hipStream_t st) {
    switch (cfg) {
        // a gated weight's tiles come in pairs
        case 0: if constexpr (GATED) return hipErrorInvalidValue; else return launch_rows<0, false>(a, st);
        case 1: return launch_rows<1, GATED>(a, st);
        case 2: return launch_wide<2, GATED>(a, st);
        case 3: return launch_tiles<3, GATED>(a, st);
        case 4: return launch_tiles<4, GATED>(a, st);
        case 5: return launch_tiles<5, GATED>(a, st);
        case 6: return launch_tiles<6, GATED>(a, st);
        default: return launch_tiles<7, GATED>(a, st);
    }
}

}  // namespace

// Up to 16 rows stream the weight through registers, a workgroup one column tile of a plain
// weight as long as that gives a compute unit at most two (4096 x 14336, one row: 10.1 us
// against 10.4 with two tiles; 28672 x 4096, 16 rows: 19.8 against 18.9).  More rows take the
// schedule and the split of the input dimension whose time is least by the measured rates:
// rounds of workgroups over 256 compute units, and for a split the partial sums' way to
// memory and back and a launch.  Up to 32 rows the streaming kernel, 16 rows a workgroup, is
// one of them (32 x 4096 x 14336: 12.8 us, 32 x 64 tiles in two splits 13.9).  Measured
// against every other choice at 20 to 4096 x 4096 x 4096 and 14336, 32 to 4096 x 14336 x 4096,
// 32 to 128 x 8192 x 8192, 333 x 5008 x 4128, 1500 x 3008 x 2048, 2000 x 8192 x 256, 8192 x 1024 x
// 512 and 2100 x 4200 x 224, and gated at 20 to 4096 x 14336 x 4096, 77 x 5003 x 2080, 100 and 700
// x 2000 x 4096, 1000 x 8192 x 2048 and 1500 x 3000 x 2048, its choice was the fastest or within
// 8% of it.  The rates are of weights that do not wait for memory: for 17 to 32 rows of wide weights
// (28672 channels) the estimates are below the time of reading the weight once.
I8Plan make_i8_plan(const I8Layout &L, int64_t M) {
    I8Plan p;
    p.cps = int(L.kchunks);
    auto blocks = [&](int c, int64_t &mt, int64_t &nb) {
        const I8Cfg &t = CFGS[c];
        mt = ceil_div(M, 16 * t.MT * t.WM);
        nb = ceil_div(L.ntiles, t.NT * t.WN);
    };
    auto threads = [](int c, int64_t mt, int64_t nb) {
        const I8Cfg &t = CFGS[c];
        return (t.kind == 2 ? std::min<int64_t>(mt * nb, WIDE_WGS) : t.kind == 0 ? nb : mt * nb) * 64 * t.WK * t.WM * t.WN;
    };
    int64_t mt, nb;
    if (M <= 16) {
        p.cfg = !L.gated && L.ntiles <= 512 ? 0 : 1;
    } else {
        float best = 0.0f;
        for (int c = M <= 32 ? 1 : WIDE; c < NUM_CFGS; ++c) {
            blocks(c, mt, nb);
            if (threads(c, mt, nb) > LAUNCH_THREADS_MAX) continue;       // the large tiles always fit
            const int step = 2 * CFGS[c].WK;                             // chunks of a stage
            for (int ks : {1, 2, 3, 4, 6, 8}) {
                const int64_t cps = ks == 1 ? L.kchunks : ceil_div(ceil_div(L.kchunks, ks), step) * step;
                if (ks > 1 && (CFGS[c].kind != 1 || cps < 8 * CFGS[c].WK || ceil_div(L.kchunks, cps) < ks)) break;
                const float rounds = float(ceil_div(mt * nb * ks, 256));
                const float starts = c < SHARED ? rounds : 1.0f + std::max(0.0f, rounds - 2.0f) * (c == SHARED ? 0.4f : 0.2f);
                // compute units that a last round leaves idle leave their power to the others
                const float work = c == WIDE ? std::max(1.0f, float(mt * nb) / 256.0f) : rounds;
                float us = work * float(cps) * CHUNK_US[c] + starts * TILE_US[c];
                if (ks > 1) us += JOIN_US + float(ks) * float(M) * float(L.ntiles) * TILE_N * 8.0f / JOIN_BYTES_PER_US;
                if (best == 0.0f || us < best) {
                    best = us;
                    p.cfg = c;
                    p.ks = ks;
                    p.cps = int(cps);
                }
            }
        }
    }
    blocks(p.cfg, mt, nb);
    p.mtiles = int(mt);
    p.nblocks = int(nb);
    p.threads = threads(p.cfg, mt, nb);
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
