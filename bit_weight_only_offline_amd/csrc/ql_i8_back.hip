// Backward products with frozen per-channel INT8 weights on the bf16 matrix cores.
//
//   linear   dx[m, k] = sum_n dy[m, n] s[n] q[n, k]
//   gated    du = dh act(g),  dg = dh u act'(g)  (one pass), then the same product over the
//            rows of both weights, up and gate tiles alternating as they are packed
//
// The product contracts over the weight's rows, across the direction it is packed in, and
// needs it in bf16.  A workgroup therefore turns each 64-row step of its weight columns
// into operand order once, through LDS, for all of its rows of dy: a thread takes the four
// inputs of one 32-bit word from eight consecutive channels, and since a conversion picks
// any byte of a word, the transposition costs no shuffles.  Per value: byte -> float32
// (exact), one fused multiply-add (u - 128) s that rounds once, and half of a packed
// rounding to bf16.  That bf16 rounding of the scaled weight is the only one before the
// float32 sums; scaling dy instead would round as much and need a second copy of it.
#include <hip/hip_runtime.h>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_i8.hpp"
#include "ql_launch.hpp"

namespace ql {
namespace {

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;   // a buffer offset that reads as zero
constexpr int NSTEP = 64;                        // weight rows (contraction) per step

// One workgroup: MP = 16 MT WM rows of dy by KP = 16 NT WN inputs, the contraction in steps
// of 64 packed rows (four tiles).  LDS, two buffers each: dy rows [MP][64] bf16 (XOR-swizzled
// 16-byte pieces), packed tiles as loaded [4][KP / 64] KiB, and the bf16 operand
// [KP / 16][2] KiB.  While step i is multiplied, the packed tiles of step i + 1 become its
// operand and the loads of dy for i + 1 and of packed tiles for i + 2 are in flight; one
// barrier a step.
template <int WM, int WN, int MT, int NT, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN) i8_back_kernel(I8BackArgs a) {
    constexpr int W = WM * WN, T = 64 * W;
    constexpr int MP = 16 * MT * WM, KP = 16 * NT * WN, KQ = KP / 64;
    static_assert(KP % 64 == 0, "whole chunks");
    constexpr int NA = MP / 8, NR = 4 * KQ;          // 1 KiB loads a step
    constexpr int A_BYTES = MP * 128, R_BYTES = NR * 1024, D_BYTES = KP * 128;
    constexpr int NAW = (NA + W - 1) / W, NRW = (NR + W - 1) / W;
    constexpr int TASKS = 2 * KP;                    // eight rows by four inputs each
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint8_t *const ldsA = lds, *const ldsR = lds + 2 * A_BYTES, *const ldsD = ldsR + 2 * R_BYTES;

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
    const int m0 = mtile * MP, kq0 = kblock * KQ;
    const int m_here = min(MP, a.M - m0);

    const int steps = (a.ntiles + 3) / 4;
    const int st0 = SPLIT ? int(blockIdx.y) * a.nps : 0;
    const int st1 = SPLIT ? min(steps, st0 + a.nps) : steps;

    const __amdgpu_buffer_rsrc_t yr =
        make_rsrc(a.dy + int64_t(m0) * a.ldy, uint32_t(m_here) * uint32_t(a.ldy) * 2u);

    auto yswz = [](int r) { return (r >> 1) & 7; };
    // piece p of a step's 64 packed rows: rows 8 p .. 8 p + 7, tile p / 2
    uint32_t y_off[NAW];
    int y_col[NAW];
#pragma unroll
    for (int q = 0; q < NAW; ++q) {
        const int row = ((wv + W * q) % NA) * 8 + lane / 8, p = (lane % 8) ^ yswz(row);
        y_col[q] = GATED ? 16 * (p >> 2) + 8 * (p & 1) : 8 * p;
        y_off[q] = uint32_t(row) * uint32_t(a.ldy) * 2u + uint32_t(y_col[q]) * 2u +
                   (GATED && (p & 2) ? uint32_t(a.half) * 2u : 0u);
        if (row >= m_here) y_off[q] = OUT_OF_RANGE;
    }
    constexpr int COLS = GATED ? NSTEP / 2 : NSTEP;   // channels a step
    auto issue_y = [&](int st, int buf) {
#pragma unroll
        for (int q = 0; q < NAW; ++q) {
            const uint32_t past = st * COLS + y_col[q] < a.N ? 0u : OUT_OF_RANGE;
            ld128_lds(yr, (y_off[q] + uint32_t(st) * (COLS * 2)) | past, ldsA + buf * A_BYTES + ((wv + W * q) % NA) * 1024);
        }
    };
    // 16-byte piece s of a packed tile lands at slot s ^ (s >> 4) << 1 ^ (chunk & 1): the
    // words that 64 threads read together then lie in 64 different banks
    uint32_t r_off[NRW];
#pragma unroll
    for (int q = 0; q < NRW; ++q) {
        const int b = (wv + W * q) % NR, tile = b / KQ, ch = b % KQ;
        const int piece = lane ^ ((lane >> 4) << 1) ^ (ch & 1);
        r_off[q] = kq0 + ch < a.kchunks
                       ? (uint32_t(tile) * uint32_t(a.kchunks) + uint32_t(kq0 + ch)) * TILE_BYTES + 16u * piece
                       : OUT_OF_RANGE;
    }
    auto issue_w = [&](int st, int buf) {
        const int here = min(4, a.ntiles - 4 * st);
        const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + int64_t(st) * 4 * a.kchunks * TILE_BYTES,
                                                    uint32_t(here) * uint32_t(a.kchunks) * TILE_BYTES);
#pragma unroll
        for (int q = 0; q < NRW; ++q) ld128_lds(wr, r_off[q], ldsR + buf * R_BYTES + ((wv + W * q) % NR) * 1024);
    };
    // tasks: four inputs (word j of group gg of chunk ch) of eight rows (octet o of the step)
    auto decode = [&](int st, int rbuf, int dbuf) {
        for (int t0 = 0; t0 < TASKS; t0 += T) {
            if (TASKS < T && ((wv / (TASKS / 64)) % (T / TASKS)) != (st % (T / TASKS))) break;   // in turn
            const int t = TASKS < T ? tid % TASKS : t0 + tid;
            const int j = t & 3, half = (t >> 2) & 1, gg = (t >> 3) & 3;
            const int ch = (t >> 5) % KQ, tile = (t >> 5) / KQ, o = 2 * tile + half;
            const uint8_t *raw = ldsR + rbuf * R_BYTES + (tile * KQ + ch) * 1024 + 4 * j;
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int piece = gg * 16 + half * 8 + i;
                w[i] = *reinterpret_cast<const uint32_t *>(raw + 16 * (piece ^ (gg << 1) ^ (ch & 1))) ^ 0x80808080u;
            }
            const int pt = 4 * st + tile;
            float s[8];
            const float *sp = a.s + int64_t(min(pt, a.ntiles - 1)) * TILE_N + 8 * half;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = pt < a.ntiles ? sp[i] : 0.0f;
            u32x4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = s[2 * i], a1 = s[2 * i + 1], b0 = -128.0f * a0, b1 = -128.0f * a1;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    v[b][i] = pack_bf16(fmaf(float((w[2 * i] >> (8 * b)) & 0xFFu), a0, b0),
                                        fmaf(float((w[2 * i + 1] >> (8 * b)) & 0xFFu), a1, b1));
            }
            const int kt = 4 * ch + gg;
            uint8_t *dst = ldsD + dbuf * D_BYTES + ((kt * 2 + (o >> 2)) * 64 + (o & 3) * 16) * 16;
#pragma unroll
            for (int b = 0; b < 4; ++b) *reinterpret_cast<u32x4 *>(dst + ((4 * j + b) ^ gg) * 16) = v[b];
        }
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](int buf) {
        const uint8_t *A = ldsA + buf * A_BYTES, *D = ldsD + buf * D_BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 yf[MT], wf[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = (wm * MT + i) * 16 + c;
                yf[i] = *reinterpret_cast<const u32x4 *>(A + row * 128 + (((4 * h + g) ^ yswz(row)) * 16));
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int kt = wn * NT + j;
                wf[j] = *reinterpret_cast<const u32x4 *>(D + ((kt * 2 + h) * 64 + g * 16 + (c ^ (kt & 3))) * 16);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[j]),
                                                                        __builtin_bit_cast(bf16x8, yf[i]), acc[j][i], 0, 0, 0);
        }
    };

    if (st0 < st1) {
        issue_w(st0, st0 & 1);
        issue_y(st0, st0 & 1);
        wait_vmcnt<0>();
        ring_barrier();
        if (st0 + 1 < st1) issue_w(st0 + 1, (st0 + 1) & 1);
        // every wavefront that takes a turn decodes in its own step; the first step's
        // operand is due now, whoever's turn it is
        decode(st0, st0 & 1, st0 & 1);
        for (int st = st0; st < st1; ++st) {
            wait_vmcnt<0>();
            ring_barrier();
            if (st + 1 < st1) issue_y(st + 1, (st + 1) & 1);
            if (st + 2 < st1) issue_w(st + 2, st & 1);
            if (st + 1 < st1) decode(st + 1, (st + 1) & 1, (st + 1) & 1);
            multiply(st & 1);
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + (wm * MT + i) * 16 + c;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int k = kq0 * 64 + (wn * NT + j) * 16 + 4 * g;
            if (k >= a.K) continue;                     // K is a multiple of 32
            if constexpr (SPLIT) {
                *reinterpret_cast<f32x4 *>(a.part + (int64_t(blockIdx.y) * a.M + m) * a.K + k) = acc[j][i];
            } else {
                *reinterpret_cast<u32x2 *>(a.dx + int64_t(m) * a.K + k) =
                    u32x2{pack_bf16(acc[j][i][0], acc[j][i][1]), pack_bf16(acc[j][i][2], acc[j][i][3])};
            }
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

// du, dg for V consecutive channels a thread; copy: the padded rows that the product reads
// when N is not a multiple of eight ([M][2][Np], zero past N), or null.
template <int V>
__global__ void __launch_bounds__(256) gate_back_kernel(const uint16_t *__restrict__ dh, const uint16_t *__restrict__ raw,
                                                        uint16_t *__restrict__ draw, uint16_t *__restrict__ copy,
                                                        int64_t M, int64_t N, int64_t Np, int act) {
    const int64_t per_row = Np / V, e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= M * per_row) return;
    const int64_t m = e / per_row, n = (e % per_row) * V;
    if constexpr (V == 8) {
        const u32x4 d = *reinterpret_cast<const u32x4 *>(dh + m * N + n);
        const u32x4 u = *reinterpret_cast<const u32x4 *>(raw + m * 2 * N + n);
        const u32x4 g = *reinterpret_cast<const u32x4 *>(raw + m * 2 * N + N + n);
        u32x4 du, dg;
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
            du[w] = pack_bf16(o[0], o[1]);
            dg[w] = pack_bf16(p[0], p[1]);
        }
        *reinterpret_cast<u32x4 *>(draw + m * 2 * N + n) = du;
        *reinterpret_cast<u32x4 *>(draw + m * 2 * N + N + n) = dg;
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
        }
        if (copy) {
            reinterpret_cast<__bf16 *>(copy)[m * 2 * Np + n] = (__bf16)o;
            reinterpret_cast<__bf16 *>(copy)[m * 2 * Np + Np + n] = (__bf16)p;
        }
    }
}

// dy [M, N] -> rows of Np, zero past N
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t *__restrict__ dy, uint16_t *__restrict__ out,
                                                       int64_t M, int64_t N, int64_t Np) {
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= M * Np) return;
    const int64_t m = e / Np, n = e % Np;
    out[e] = n < N ? dy[m * N + n] : uint16_t(0);
}

struct BackCfg { int WM, WN, MT, NT; };
constexpr BackCfg BACK_CFGS[] = {{4, 2, 4, 4}, {2, 2, 4, 4}, {2, 2, 1, 4}};
constexpr int back_lds(const BackCfg &t) {
    return 2 * (16 * t.MT * t.WM * 128 + 16 * t.NT * t.WN * (64 + 128));
}

template <int I, bool GATED>
hipError_t launch_back(const I8BackArgs &a, hipStream_t st) {
    constexpr BackCfg t = BACK_CFGS[I];
    constexpr int lds = back_lds(t);
    static_assert(lds <= LDS_BYTES_MAX, "two buffers fit the LDS");
    const dim3 grid(unsigned(a.mtiles * a.nblocks), unsigned(a.ks)), block(64 * t.WM * t.WN);
    if (a.ks == 1) {
        auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, GATED, false>;
        static const hipError_t set =
            hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (set != hipSuccess) return set;
        hipLaunchKernelGGL(kern, grid, block, lds, st, a);
        return hipGetLastError();
    }
    auto kern = i8_back_kernel<t.WM, t.WN, t.MT, t.NT, GATED, true>;
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

template <bool GATED>
hipError_t launch_back_any(int cfg, const I8BackArgs &a, hipStream_t st) {
    switch (cfg) {
        case 0: return launch_back<0, GATED>(a, st);
        case 1: return launch_back<1, GATED>(a, st);
        default: return launch_back<2, GATED>(a, st);
    }
}

}  // namespace

// Rows of dy the product cannot read in place (N not a multiple of eight) are copied to
// rows of Np first; a gated product's du and dg are written there as they are formed.
I8BackPlan make_i8_back_plan(const I8Layout &L, int64_t M) {
    I8BackPlan p;
    p.Np = ceil_div(L.N, 8) * 8;
    const int64_t kcols = L.kchunks * I8_CHUNK;
    for (int c = 0; c < 3; ++c) {
        const BackCfg &t = BACK_CFGS[c];
        p.cfg = c;
        p.mtiles = int(ceil_div(M, 16 * t.MT * t.WM));
        p.nblocks = int(ceil_div(kcols, 16 * t.NT * t.WN));
        if (int64_t(p.mtiles) * p.nblocks >= 192) break;
    }
    const int64_t steps = ceil_div(L.ntiles, 4), wgs = int64_t(p.mtiles) * p.nblocks;
    int64_t ks = wgs >= 192 ? 1 : ceil_div(256, wgs);
    ks = std::max<int64_t>(1, std::min<int64_t>(ks, steps / 4));
    p.nps = int(ceil_div(steps, ks));
    p.ks = int(ceil_div(steps, p.nps));
    p.copy_bytes = L.N % 8 ? round256(size_t(M) * size_t(p.Np) * (L.gated ? 4 : 2)) : 0;
    p.ws_bytes = p.copy_bytes + (p.ks > 1 ? round256(size_t(p.ks) * size_t(M) * size_t(L.K) * 4) : 0);
    return p;
}

hipError_t launch_i8_backward(const I8Layout &L, const I8BackPlan &p, const uint16_t *dy, const uint16_t *raw, int act,
                              int64_t M, const void *pw, const void *ps, uint16_t *dx, uint16_t *draw, void *ws,
                              hipStream_t st) {
    uint16_t *copy = p.copy_bytes ? static_cast<uint16_t *>(ws) : nullptr;
    I8BackArgs a{};
    if (L.gated) {
        const int V = copy ? 1 : 8;
        const int64_t n = M * ((copy ? p.Np : L.N) / V);
        const dim3 grid(unsigned(ceil_div(n, 256)));
        if (copy)
            hipLaunchKernelGGL(gate_back_kernel<1>, grid, dim3(256), 0, st, dy, raw, draw, copy, M, L.N, p.Np, act);
        else
            hipLaunchKernelGGL(gate_back_kernel<8>, grid, dim3(256), 0, st, dy, raw, draw, copy, M, L.N, L.N, act);
        a.dy = copy ? copy : draw;
        a.half = copy ? p.Np : L.N;
        a.ldy = 2 * a.half;
    } else {
        if (copy)
            hipLaunchKernelGGL(pad_rows_kernel, dim3(unsigned(ceil_div(M * p.Np, 256))), dim3(256), 0, st, dy, copy, M,
                               L.N, p.Np);
        a.dy = copy ? copy : dy;
        a.ldy = copy ? p.Np : L.N;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.w = static_cast<const uint8_t *>(pw);
    a.s = static_cast<const float *>(ps);
    a.dx = dx;
    a.part = p.ks > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.copy_bytes) : nullptr;
    a.M = int(M);
    a.N = int(copy ? p.Np : L.N);
    a.K = int(L.K);
    a.ntiles = int(L.ntiles);
    a.kchunks = int(L.kchunks);
    a.mtiles = p.mtiles;
    a.nblocks = p.nblocks;
    a.ks = p.ks;
    a.nps = p.nps;
    return L.gated ? launch_back_any<true>(p.cfg, a, st) : launch_back_any<false>(p.cfg, a, st);
}

}  // namespace ql
