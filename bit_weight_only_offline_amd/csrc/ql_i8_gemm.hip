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

// The float32 results of four consecutive channels of token m (scale xs) whose sums are
// `sum`, tile `tile` holding them at position `at` (a multiple of four).
__device__ inline void scaled(const I8Args &a, float xs, int tile, int at, int64_t bias_at, int count, const i32x4 &sum,
                              float (&v)[4]) {
    const f32x4 s = *reinterpret_cast<const f32x4 *>(a.s + int64_t(tile) * TILE_N + at);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float b = (a.bias && r < count) ? bf16_bits_to_f32(a.bias[bias_at + r]) : 0.0f;
        v[r] = fmaf(float(sum[r]) * xs, s[r], b);
    }
}

// Linear: tile `tile`, channels 16 tile + at .. +3 of token m.
__device__ inline void emit_linear(const I8Args &a, int m, float xs, int tile, int at, const i32x4 &sum) {
    const int n = tile * TILE_N + at, count = a.N - n;
    if (count <= 0) return;
    float v[4];
    scaled(a, xs, tile, at, n, count, sum, v);
    const int64_t i = int64_t(m) * a.N + n;
    if (a.out_f32) store4_f32(static_cast<float *>(a.out), i, v, count, a.vec);
    else store4_bf16(static_cast<uint16_t *>(a.out), i, v, count, a.vec);
}

// Gated: tile pair `pair` (up tile 2 pair, gate tile 2 pair + 1).
__device__ inline void emit_gated(const I8Args &a, int m, float xs, int pair, int at, const i32x4 &up, const i32x4 &gt) {
    const int n = pair * TILE_N + at, count = a.N - n;
    if (count <= 0) return;
    float u[4], g[4], h[4];
    scaled(a, xs, 2 * pair, at, n, count, up, u);
    scaled(a, xs, 2 * pair + 1, at, int64_t(a.N) + n, count, gt, g);
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
        const float xs = a.xs[m];
        auto total = [&](int tile) {
            i32x4 t = red[(tile * MT + i) * 64 + l];
#pragma unroll
            for (int w = 1; w < WK; ++w) t += red[(w * NT * MT + tile * MT + i) * 64 + l];
            return t;
        };
        if constexpr (GATED) emit_gated(a, m, xs, nt0 / 2 + j, at, total(2 * j), total(2 * j + 1));
        else emit_linear(a, m, xs, nt0 + j, at, total(j));
    }
}

// ---- tiles: both operands staged through LDS ------------------------------------------
// WM x WN wavefronts, each 16 MT tokens x NT column tiles.  A stage holds CPS chunks of
// 16 MT WM activation rows and of NT WN weight tiles; S stages form a ring that direct
// buffer->LDS loads fill, S - 1 stages ahead of the one being multiplied.  Activation rows
// are loaded in whole 64 CPS-byte runs; a XOR swizzle of their 16-byte pieces, applied to
// the global address of each lane, spreads the 16 rows of an operand read over all banks.
// Weight tiles are stored in operand order, so their reads are linear.
template <int WM, int WN, int MT, int NT, int CPS, int S, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN) i8_tile_kernel(I8Args a) {
    static_assert(!GATED || NT % 2 == 0, "up and gate tiles go together");
    constexpr int W = WM * WN;
    constexpr int MP = 16 * MT * WM, NTT = NT * WN;
    constexpr int P = 4 * CPS, RPI = 64 / P;           // 16-byte pieces a row, rows a load
    constexpr int NA = MP / RPI, NB = NTT * CPS;       // 1 KiB loads a stage
    static_assert(NA % W == 0 && NB % W == 0, "every wavefront issues the same loads");
    constexpr int NAW = NA / W, NBW = NB / W, PER_STAGE = NAW + NBW;
    constexpr int STAGE = (NA + NB) * 1024;
    static_assert(S * STAGE <= LDS_BYTES_MAX && S >= 2 && S <= 6, "ring fits the LDS");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;
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
    const int kc1 = SPLIT ? min(a.kchunks, kc0 + a.cps) : a.kchunks;
    const int nst = (kc1 - kc0 + CPS - 1) / CPS;

    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(a.w + int64_t(nt0) * a.kchunks * TILE_BYTES, uint32_t(nt_here) * uint32_t(a.kchunks) * TILE_BYTES);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + int64_t(m0) * a.K, uint32_t(m_here) * uint32_t(a.K));

    auto xswz = [](int r) { return P == 8 ? ((r >> 1) & 7) : ((r >> 2) & 3); };
    uint32_t a_off[NAW], b_off[NBW];
    int b_chunk[NBW];
#pragma unroll
    for (int q = 0; q < NAW; ++q) {
        const int row = (wv + W * q) * RPI + lane / P;
        a_off[q] = row < m_here ? uint32_t(row) * uint32_t(a.K) + 16u * uint32_t((lane % P) ^ xswz(row)) : OUT_OF_RANGE;
    }
#pragma unroll
    for (int q = 0; q < NBW; ++q) {
        const int b = wv + W * q, tile = b / CPS;
        b_chunk[q] = b % CPS;
        b_off[q] = tile < nt_here ? (uint32_t(tile) * uint32_t(a.kchunks) + uint32_t(b_chunk[q])) * TILE_BYTES + 16u * lane
                                  : OUT_OF_RANGE;
    }
    auto issue = [&](int st, int buf) {
        uint8_t *base = lds + buf * STAGE;
        const int kc = kc0 + st * CPS;
#pragma unroll
        for (int q = 0; q < NAW; ++q) ld128_lds(xr, a_off[q] + uint32_t(kc) * I8_CHUNK, base + (wv + W * q) * 1024);
#pragma unroll
        for (int q = 0; q < NBW; ++q) {
            // a chunk past the range reads as zero, which leaves the sums as they are
            const uint32_t past = kc + b_chunk[q] < kc1 ? 0u : OUT_OF_RANGE;
            ld128_lds(wr, (b_off[q] + uint32_t(kc) * TILE_BYTES) | past, base + (NA + wv + W * q) * 1024);
        }
    };

    i32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

    auto compute = [&](int buf) {
        const uint8_t *A = lds + buf * STAGE, *B = A + NA * 1024;
#pragma unroll
        for (int h = 0; h < CPS; ++h) {
            u32x4 xf[MT], wf[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = (wm * MT + i) * 16 + c;
                xf[i] = *reinterpret_cast<const u32x4 *>(A + row * (P * 16) + (((4 * h + g) ^ xswz(row)) * 16));
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
                wf[j] = *reinterpret_cast<const u32x4 *>(B + ((wn * NT + j) * CPS + h) * 1024 + lane * 16);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] = mma(wf[j], xf[i], acc[j][i]);
        }
    };

#pragma unroll
    for (int u = 0; u < S - 1; ++u)
        if (u < nst) issue(u, u);
    for (int i0 = 0; i0 < nst; i0 += S) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const int i = i0 + u;
            if (i < nst) {
                const int later = min(S - 2, nst - 1 - i);   // stages issued after this one
                if (later >= 4) wait_vmcnt<4 * PER_STAGE>();
                else if (later == 3) wait_vmcnt<3 * PER_STAGE>();
                else if (later == 2) wait_vmcnt<2 * PER_STAGE>();
                else if (later == 1) wait_vmcnt<PER_STAGE>();
                else wait_vmcnt<0>();
                ring_barrier();
                if (i + S - 1 < nst) issue(i + S - 1, (u + S - 1) % S);
                compute(u);
            }
        }
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
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + (wm * MT + i) * 16 + c;
        if (m >= a.M) continue;
        const float xs = a.xs[m];
#pragma unroll
        for (int j = 0; j < NT; j += (GATED ? 2 : 1)) {
            const int tile = wn * NT + j;
            if (tile >= nt_here) continue;
            if constexpr (GATED) emit_gated(a, m, xs, (nt0 + tile) / 2, 4 * g, acc[j][i], acc[j + 1][i]);
            else emit_linear(a, m, xs, nt0 + tile, 4 * g, acc[j][i]);
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
    auto total = [&](int t) {
        i32x4 s{0, 0, 0, 0};
        for (int k = 0; k < a.ks; ++k)
            s += *reinterpret_cast<const i32x4 *>(a.part + (int64_t(k) * a.M + m) * width + int64_t(t) * TILE_N + at);
        return s;
    };
    if constexpr (GATED) emit_gated(a, m, a.xs[m], tile, at, total(2 * tile), total(2 * tile + 1));
    else emit_linear(a, m, a.xs[m], tile, at, total(tile));
}

constexpr I8Cfg CFGS[] = {
    {0, 1, 2, 8, 1, 1, 1, 0}, {0, 2, 2, 8, 1, 1, 1, 0}, {0, 4, 2, 8, 1, 1, 1, 0},
    {1, 2, 2, 1, 2, 2, 2, 4}, {1, 4, 4, 1, 2, 2, 2, 4}, {1, 8, 4, 1, 2, 4, 2, 2},
};
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
    constexpr size_t lds = size_t(t.S) * (16 * t.MT * t.WM + 16 * t.NT * t.WN) * t.CPS * I8_CHUNK;
    const dim3 grid(unsigned(a.mtiles * a.nblocks), unsigned(a.ks));
    const dim3 block(64 * t.WM * t.WN);
    if (a.ks == 1) {
        auto kern = i8_tile_kernel<t.WM, t.WN, t.MT, t.NT, t.CPS, t.S, GATED, false>;
        static const hipError_t set = allow_lds(kern, lds);
        if (set != hipSuccess) return set;
        hipLaunchKernelGGL(kern, grid, block, lds, st, a);
        return hipGetLastError();
    }
    auto kern = i8_tile_kernel<t.WM, t.WN, t.MT, t.NT, t.CPS, t.S, GATED, true>;
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
        case 0: return launch_rows<0, GATED>(a, st);
        case 1: return launch_rows<1, GATED>(a, st);
        case 2: return launch_rows<2, GATED>(a, st);
        case 3: return launch_tiles<3, GATED>(a, st);
        case 4: return launch_tiles<4, GATED>(a, st);
        default: return launch_tiles<5, GATED>(a, st);
    }
}

}  // namespace

I8Plan make_i8_plan(const I8Layout &L, int64_t M) {
    I8Plan p;
    if (M <= 64) p.cfg = M <= 16 ? 0 : (M <= 32 ? 1 : 2);
    else {
        p.cfg = 5;
        for (int c : {5, 4, 3}) {
            p.cfg = c;
            const I8Cfg &t = CFGS[c];
            if (ceil_div(M, 16 * t.MT * t.WM) * ceil_div(L.ntiles, t.NT * t.WN) >= 192) break;
        }
    }
    const I8Cfg &t = CFGS[p.cfg];
    p.mtiles = int(ceil_div(M, 16 * t.MT * t.WM));
    p.nblocks = int(ceil_div(L.ntiles, t.NT * t.WN));
    p.cps = int(L.kchunks);
    if (t.kind == 1) {
        const int64_t wgs = int64_t(p.mtiles) * p.nblocks;
        int64_t ks = wgs >= 192 ? 1 : ceil_div(256, wgs);
        ks = std::max<int64_t>(1, std::min<int64_t>(ks, L.kchunks / (4 * t.CPS)));
        p.cps = int(ceil_div(ceil_div(L.kchunks, ks), t.CPS) * t.CPS);
        p.ks = int(ceil_div(L.kchunks, p.cps));
        if (p.ks > 1) p.ws_bytes = round256(size_t(p.ks) * size_t(M) * size_t(L.ntiles) * TILE_N * 4);
    }
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
