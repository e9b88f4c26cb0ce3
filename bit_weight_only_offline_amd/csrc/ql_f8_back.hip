// Backward products through frozen block-scaled e4m3 weights, plain or over experts.
//
//   dx[m, k] = sum over channel blocks b of ws[b, k / 128] (sum over n in b of dy[m, n] w[n, k])
//
// dy is bf16, and an e4m3 code is exact in bf16: the products go through the bf16 matrix cores without
// rounding either, and float32 holds the sums.  The scale of a block multiplies what 128 channels have summed
// to.  Rather than a second set of sums, which registers have no room for, the running sums are kept in
// units of the current block's scale: between two blocks they are multiplied by the ratio of the scales, and
// at the end by the last.  Powers of two go into the codes' conversion, as far as that is exact: from 2^-124 to 2^119 a
// code times the power is a bf16 number (2^-9 times the least is bf16's smallest, which the matrix cores keep; 448 times the
// largest is finite).  So the unit left is between 1 and 2 for scales in that range, down to 2^-2 for other normal ones and
// 2^-25 for subnormal ones, and below 2^9: sums up to 2^102 overflow at no scale.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ql_f8_device.hpp"
#include "ql_gemm_lds.hpp"
#include "ql_launch.hpp"
#include "ql_lds_limit.hpp"

namespace ql {
namespace {

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;

__device__ inline f32x4 mma(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A block's scale as mantissa and power of two, the ratio of the sums' unit before to it, and how its codes are
// taken apart.  Scales outside the powers' range have a smaller or larger mantissa; NaN and infinity are
// mantissas.  A block with the scale 0 leaves the unit as it is, and its codes are taken as zeros.
struct Scale {
    float mantissa, power, ratio;
    uint32_t lo, hi;                                       // permutations: inputs 0 and 1, 2 and 3 of two channels
};
__device__ inline Scale split_scale(float s, float before) {
    asm("" : "+v"(s));                                     // selections, where a uniform value would make branches
    const uint32_t e = min(max((__float_as_uint(s) >> 23) & 0xFFu, 127u - 124u), 127u + 119u);
    const bool none = s == 0.0f;
    Scale r;
    r.power = __uint_as_float(e << 23);
    r.mantissa = none ? before : s * __uint_as_float((254u - e) << 23);
    r.ratio = none ? 1.0f : before / r.mantissa;           // an infinite unit by itself would be NaN
    r.lo = none ? 0x0C0C0C0Cu : 0x05010400u;
    r.hi = none ? 0x0C0C0C0Cu : 0x07030602u;
    return r;
}

// Two codes as bf16 times a power of two.
template <bool HI>
__device__ inline uint32_t widen2(uint32_t codes, float power) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, power, HI));
}

// Workgroup: WM x WN wavefronts, each 16 MT tokens x 64 inputs; three stages of 64 channels in LDS.
//
// Weight.  The operand of inputs (the A operand) needs eight channels of one input in a lane, packed tiles
// hold sixteen inputs of one channel.  A stage's 64 x 64 codes of a wavefront column lie in LDS as four planes of
// sixteen inputs, 64 channels of 16 bytes each; channel 32 h + 8 g + 4 p + q of the stage at 32 h + 16 p + 4 g + q.  Lane (c,
// g) reads inputs 4 c .. 4 c + 3 of channel 8 g + r of step h in one word, from plane c / 4; planes are 1040 bytes apart,
// so that the 64 words lie in 64 banks.  Loaded in this order, four lanes fetch 64 bytes in a row (8192 x 4096 x 14336:
// 934 us, 948 with 16 bytes from each of four places).  Eight such words are
// four operands, of inputs 4 c + j for j = 0 .. 3, after eight byte permutes and sixteen conversions.  Their sums
// leave a lane with sixteen consecutive inputs of a token, 32 bytes of bf16, which are stored as they are.
//
// Gradients.  128-byte runs of the rows, their 16-byte pieces swizzled; the B operand, read P tiles ahead.
//
// A stage is two steps of 32 channels.  During a step the next one's codes are read and turned into operands between
// the matrix instructions (8192 x 4096 x 14336 over 8 equal experts: 812 us, 1.18 PFLOP/s, the matrix cores busy half of the
// time; 934 while branches in the loop let the compiler move the decoding behind them, and 636 without the loads: they
// are what the wavefronts wait for, a quarter of their time).  A barrier before each step: the first of a stage frees the stage before it, whose place
// takes the loads of the stage after next; the second waits for the next stage.
constexpr int PLANE = 1040;
template <int WM, int WN, int MT>
constexpr int back_lds() { return 3 * (16 * MT * WM * 128 + WN * 4 * PLANE) + (2 * MT * WM < WM * WN ? 1024 : 0); }

template <int WM, int WN, int MT, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2))) f8_back_kernel(F8BackArgs a) {
    constexpr int S = 3, W = WM * WN, MP = 16 * MT * WM, KP = 64 * WN;
    constexpr int P = MT >= 4 ? 3 : 1, XB = MT >= 4 ? 4 : 2;
    constexpr int X_BYTES = MP * 128, STAGE = X_BYTES + WN * 4 * PLANE;
    constexpr int XL = MP / 8, WL = 4 * WN;                // 1 KiB loads of a stage
    constexpr int XLW = (XL + W - 1) / W, WLW = WL / W, LOADS = XLW + WLW;
    static_assert(WL % W == 0 && (XL % W == 0 || XL < W), "every wavefront issues the same loads");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN;
    const int g = lane >> 4, c = lane & 15;

    // as in the forward product: runs of the tile order to each XCD, bands of eight row blocks
    RowBlock rb;
    int mtiles = a.mtiles;
    if (a.r.counts) find_rows(a.r, MP, -1, lane, rb, mtiles);
    const int tiles = mtiles * a.nblocks;
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int q8 = tiles >> 3, r8 = tiles & 7;
    if (idx >= q8 + (xcd < r8 ? 1 : 0)) return;
    const int lin = xcd * q8 + min(xcd, r8) + idx;
    const int band = lin / (8 * a.nblocks), in_band = lin - band * 8 * a.nblocks;
    const int band_rows = min(8, mtiles - 8 * band);
    find_rows(a.r, MP, 8 * band + in_band % band_rows, lane, rb, mtiles);
    const int k0 = in_band / band_rows * KP;               // first input of the workgroup

    // channels nb0 * 128 .. in stages of 64
    const int nb0 = SPLIT ? int(blockIdx.y) * a.bps : 0;
    const int nbs = SPLIT ? min(a.nbs - nb0, a.bps) : a.nbs;
    const int n_end = min(a.N, (nb0 + nbs) * F8_BLOCK);
    const int nst = (n_end - nb0 * F8_BLOCK + 63) / 64;

    const __amdgpu_buffer_rsrc_t xr =
        make_uniform_rsrc(a.dy + int64_t(rb.first) * a.ldy, uint32_t(rb.count) * uint32_t(a.ldy) * 2u);
    const uint8_t *const w = a.w + uint64_t(rb.expert) * a.w_stride;
    const float *const ws = a.ws + (int64_t(rb.expert) * a.nbs + nb0) * a.kblocks;
    const int kb = min((k0 + 64 * wn) / F8_BLOCK, a.kblocks - 1);

    // A wavefront's first loads of a stage; the others lie a fixed distance on.  Rows past the last lie past the range.
    // Inputs past the last are read from whatever lies there, and their sums are not stored.
    const int row = wv * 8 + (lane >> 3), piece = (lane & 7) ^ ((row >> 1) & 7);
    static_assert(W % 2 == 0, "a wavefront's rows have one swizzle");
    const uint32_t x_off = uint32_t(row) * uint32_t(a.ldy) * 2u + uint32_t(nb0) * (2 * F8_BLOCK) + 16u * uint32_t(piece);
    const uint32_t x_far = uint32_t(W * 8) * uint32_t(a.ldy) * 2u;
    const int x_left = int(a.ldy) - nb0 * F8_BLOCK - 8 * piece;   // channels from the piece to the row's end
    // a load takes one plane of a wavefront column; the four channel tiles of a stage are kblocks tiles apart each
    const uint32_t tile_step = uint32_t(a.kblocks) * F8_TILE_BYTES;
    const int tiles_here = min(a.ntiles - nb0 * 8, nbs * 8);
    const int channel = 32 * (lane >> 5) + 8 * ((lane >> 2) & 3) + 4 * ((lane >> 4) & 1) + (lane & 3);   // of the stage
    const int k_load = k0 + 64 * (wv >> 2);
    static_assert(W % 4 == 0 && F8_TILE_BYTES == 2048, "four planes; a column is 1 KiB after the one before");
    const uint32_t w_off = uint32_t(channel >> 4) * tile_step + uint32_t(k_load >> 6) * 1024u + uint32_t(16 * (wv & 3) + (channel & 15)) * 16u;
    auto load = [&](int st, int place) {
        uint8_t *const base = lds + place;
        const bool more = (st < nst) & (st * 64 < x_left);
#pragma unroll
        for (int q = 0; q < XLW; ++q) {
            if (XL < W && wv >= XL) ld128_lds(xr, OUT_OF_RANGE, lds + S * STAGE);   // nothing left: zeros to a place of their own
            else ld128_lds(xr, more ? x_off + uint32_t(q) * x_far + uint32_t(st) * 128u : OUT_OF_RANGE, base + (wv + W * q) * 1024);
        }
        // four tiles a stage, those past the last read as zero
        const int left = max(0, min(4, tiles_here - 4 * st));
        const __amdgpu_buffer_rsrc_t wr = make_uniform_rsrc(w + int64_t(nb0 * 8 + min(4 * st, tiles_here)) * tile_step, uint32_t(left) * tile_step);
#pragma unroll
        for (int q = 0; q < WLW; ++q) ld128_lds(wr, w_off + uint32_t(q * (W / 4)) * 1024u, base + X_BYTES + (wv + W * q) * PLANE);
    };

    f32x4 acc[4][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint8_t *const x_at[2] = {lds + (wm * MT * 16 + c) * 128 + ((g ^ (c >> 1)) * 16),
                                    lds + (wm * MT * 16 + c) * 128 + (((4 + g) ^ (c >> 1)) * 16)};
    const uint8_t *const w_at = lds + X_BYTES + (4 * wn + (c >> 2)) * PLANE + g * 64 + (c & 3) * 4;
    struct Codes {
        uint32_t v[8];
    };
    auto read_w = [&](Codes &o, int stage, int h) {
#pragma unroll
        for (int q = 0; q < 8; ++q) o.v[q] = *reinterpret_cast<const uint32_t *>(w_at + stage + h * 512 + (q >> 2) * 256 + (q & 3) * 16);
    };
    // Channels 2 p and 2 p + 1 of each lane's eight.
    auto decode = [&](const Codes &o, int p, const Scale &s, u32x4 (&op)[4]) {
        const uint32_t lo = __builtin_amdgcn_perm(o.v[2 * p + 1], o.v[2 * p], s.lo);
        const uint32_t hi = __builtin_amdgcn_perm(o.v[2 * p + 1], o.v[2 * p], s.hi);
        op[0][p] = widen2<false>(lo, s.power);
        op[1][p] = widen2<true>(lo, s.power);
        op[2][p] = widen2<false>(hi, s.power);
        op[3][p] = widen2<true>(hi, s.power);
    };
    u32x4 x[XB], op[2][4];
    auto read_x = [&](int stage, int q) {                  // tile q of a stage's two steps
        x[q % XB] = *reinterpret_cast<const u32x4 *>(x_at[q / MT] + stage + q % MT * 2048);
    };

    load(0, 0);
    load(1, STAGE);
    wait_vmcnt<LOADS>();
    ring_barrier();
    float s_next = ws[kb];
    Scale now = split_scale(s_next, 1.0f), next = now;
    s_next = ws[int64_t(min(1, nbs - 1)) * a.kblocks + kb];
    {
        Codes first;
        read_w(first, 0, 0);
#pragma unroll
        for (int q = 0; q < P; ++q) read_x(0, q);
#pragma unroll
        for (int p = 0; p < 4; ++p) decode(first, p, now, op[0]);
    }
    int at = 0, after = STAGE;                             // places of this stage and of the next
    for (int st = 0; st < nst; st += 2) {                  // a block of channels, its second stage maybe empty
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int free = after == (S - 1) * STAGE ? 0 : after + STAGE;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1) wait_vmcnt<LOADS>();
                ring_barrier();
                if (h == 0) load(st + e + 2, free);
                if (e == 1 && h == 1) {
                    next = split_scale(s_next, now.mantissa);
                    next.ratio = st + 2 < nst ? next.ratio : 1.0f;
                    next.mantissa = st + 2 < nst ? next.mantissa : now.mantissa;
                    s_next = ws[int64_t(min((st >> 1) + 2, nbs - 1)) * a.kblocks + kb];
                }
                Codes codes;
                read_w(codes, h == 0 ? at : after, 1 - h);
                __builtin_amdgcn_sched_barrier(0);
                const Scale &s = e == 1 && h == 1 ? next : now;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int q = h * MT + i;
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j][i] = mma(op[h][j], x[q % XB], acc[j][i]);
                    if (q + P < 2 * MT) read_x(at, q + P);
                    else read_x(after, q + P - 2 * MT);
                    // the next step's operands, and behind a block's last products its sums in units of the next scale
                    if (MT >= 4 ? i >= MT - 4 : i == 0)
#pragma unroll
                        for (int p = MT >= 4 ? i - (MT - 4) : 0; p < (MT >= 4 ? i - (MT - 4) + 1 : 4); ++p) decode(codes, p, s, op[1 - h]);
                    if (e == 1 && h == 1 && i > 0)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[j][i - 1] *= next.ratio;
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (e == 1 && h == 1)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j][MT - 1] *= next.ratio;
            }
            at = after;
            after = free;
        }
        now = next;
    }

    wait_vmcnt<0>();                                       // zeros of stages past the last, on their way into LDS

    // A lane holds inputs 16 g .. of the wavefront's 64, element j of each four in acc[j].
    const float last = now.mantissa;
    const int k = k0 + 64 * wn + 16 * g;
    if (k >= a.K) return;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = (wm * MT + i) * 16 + c;
        if (row >= rb.count) continue;
        const int64_t at = int64_t(rb.first + row) * a.K + k;
        float v[16];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * r + j] = acc[j][i][r] * last;
        if constexpr (SPLIT) {
            float *const to = a.part + int64_t(blockIdx.y) * a.r.rows * a.K + at;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f32x4 *>(to + 4 * r) = f32x4{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r)
                *reinterpret_cast<u32x4 *>(a.dx + at + 8 * r) =
                    u32x4{pack_bf16(v[8 * r], v[8 * r + 1]), pack_bf16(v[8 * r + 2], v[8 * r + 3]),
                          pack_bf16(v[8 * r + 4], v[8 * r + 5]), pack_bf16(v[8 * r + 6], v[8 * r + 7])};
        }
    }
}

// Adds the splits' sums in their order.
__global__ void __launch_bounds__(256) f8_back_join_kernel(const float *part, uint16_t *dx, int64_t n, int ks) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n / 4; i += int64_t(gridDim.x) * 256) {
        f32x4 s = *reinterpret_cast<const f32x4 *>(part + 4 * i);
        for (int k = 1; k < ks; ++k) s += *reinterpret_cast<const f32x4 *>(part + k * n + 4 * i);
        *reinterpret_cast<u32x2 *>(dx + 4 * i) = u32x2{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
    }
}

// Rows of N channels in rows of ldy, a multiple of eight, zeros behind: loads into LDS need rows on 16 bytes.
__global__ void __launch_bounds__(256) f8_back_copy_kernel(const uint16_t *dy, uint16_t *to, int64_t M, int N, int64_t ldy) {
    const int64_t per_row = ldy / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < M * per_row; i += int64_t(gridDim.x) * 256) {
        const int64_t m = i / per_row, n = (i - m * per_row) * 8;
        const uint16_t *from = dy + m * N + n;
        u32x4 v{0u, 0u, 0u, 0u};
        if (n + 8 <= N) {
            const u32x4_any p = *reinterpret_cast<const u32x4_any *>(from);
            v = u32x4{p[0], p[1], p[2], p[3]};
        } else {
            for (int j = 0; n + j < N; ++j) v[j >> 1] |= uint32_t(from[j]) << (16 * (j & 1));
        }
        *reinterpret_cast<u32x4 *>(to + m * ldy + n) = v;
    }
}

struct BackCfg { int WM, WN, MT; };
constexpr BackCfg CFGS[] = {
    {2, 4, 8},      // 256 x 256
    {1, 4, 4},      // 64 x 256
    {1, 4, 2},      // 32 x 256
    {1, 4, 1},      // 16 x 256
};
constexpr int NUM_CFGS = 4;
// Microseconds that a compute unit takes for a block of 128 channels, and for a tile besides (start, first loads, stores),
// and what a round of 256 workgroups after the first takes of either, less where several share a unit.  Fitted to 84
// sizes, 1 to 8192 x 4096 x 14336, 14336 x 4096, 4096 x 4096, 5000 x 4128, 2048 x 2048 and 1024 x 8192, every tile in
// one to twelve splits.  Tiles of 128 rows were the fastest at none.  Of 66 sizes of the same layers, 1 to 4096 rows, the
// choice is the fastest at the median and loses more than 9% at two: 333 x 4096 x 14336, where the 16-row tile's second
// round is taken for too short (94 us against 60 with 64 rows), and 1400 x 5001 x 4128 (94 against 84).  Grouped products have no
// sizes in the fit: over 8 experts of 4096 x 14336, 512 rows take 172 us (64-row tiles 98), 2048 rows 240 (256-row 220).  A
// grouped product is not split, so that few rows leave most compute units idle: one row over 8 experts of 14336 x 4096
// takes 97 us, where the plain product in splits takes 18.
struct BackRate { float block, tile, tile_more, block_more; };
constexpr BackRate RATES[NUM_CFGS] = {
    {3.19f, 8.0f, 1.07f, 0.85f}, {1.19f, 5.2f, 0.05f, 0.74f}, {0.91f, 4.9f, 0.01f, 0.67f}, {0.69f, 4.4f, 0.19f, 0.4f},
};
constexpr float JOIN_US = 4.1f, JOIN_BYTES_PER_US = 4.8e6f;

template <int I, bool SPLIT>
hipError_t launch_of(const F8BackArgs &a, hipStream_t st) {
    constexpr BackCfg t = CFGS[I];
    constexpr size_t lds = back_lds<t.WM, t.WN, t.MT>();
    static_assert(lds <= LDS_BYTES_MAX, "fits");
    auto kern = f8_back_kernel<t.WM, t.WN, t.MT, SPLIT>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)kern, int(lds));
    if (e != hipSuccess) return e;
    const unsigned grid = unsigned(ceil_div(int64_t(a.mtiles) * a.nblocks, 8) * 8);
    hipLaunchKernelGGL(kern, dim3(grid, unsigned(a.ks)), dim3(64 * t.WM * t.WN), lds, st, a);
    return hipGetLastError();
}

template <int I>
hipError_t launch(const F8BackArgs &a, hipStream_t st) {
    if (a.ks == 1) return launch_of<I, false>(a, st);
    const hipError_t e = launch_of<I, true>(a, st);
    if (e != hipSuccess) return e;
    const int64_t n = int64_t(a.r.rows) * a.K;
    hipLaunchKernelGGL(f8_back_join_kernel, elementwise_grid(n / 4), dim3(256), 0, st, a.part, a.dx, n, a.ks);
    return hipGetLastError();
}

}  // namespace

// The tile and the split of the channels whose time is least by the measured rates.  A grouped product's row
// blocks are taken to be half a block an expert more than its rows fill; it is not split.
F8BackPlan make_f8_back_plan(const F8Layout &L, int64_t M, bool grouped) {
    F8BackPlan p;
    p.ldy = ceil_div(L.N, 8) * 8;
    const int64_t used = grouped ? std::min(L.E, M) : 1;
    auto columns = [&](const BackCfg &t) { return ceil_div(L.K, 64 * t.WN); };
    auto threads = [&](const BackCfg &t) {
        return ceil_div(most_row_blocks(M, L.E, grouped, 16 * t.MT * t.WM) * columns(t), 8) * 8 * 64 * t.WM * t.WN;
    };
    float best = 0.0f;
    for (int c = 0; c < NUM_CFGS; ++c) {
        const BackCfg &t = CFGS[c];
        const BackRate &rate = RATES[c];
        if (c > 0 && threads(t) > LAUNCH_THREADS_MAX) continue;             // where the tallest do not fit, none does
        const int64_t block = 16 * t.MT * t.WM, mt = grouped ? std::max(used, ceil_div(2 * M + used * block, 2 * block)) : ceil_div(M, block);
        for (int ks : {1, 2, 3, 4, 6, 8, 12}) {
            const int64_t bps = ceil_div(L.nblocks, ks);
            if (ks > 1 && (grouped || bps < 2 || ceil_div(L.nblocks, bps) < ks)) break;
            const float more = float(ceil_div(mt * columns(t) * ks, 256) - 1);
            float us = (1.0f + more * rate.block_more) * float(bps) * rate.block + (1.0f + more * rate.tile_more) * rate.tile;
            if (ks > 1) us += JOIN_US + float(ks) * float(M) * float(L.K) * 8.0f / JOIN_BYTES_PER_US;
            if (best == 0.0f || us < best) {
                best = us;
                p.cfg = c;
                p.ks = ks;
                p.bps = int(bps);
            }
        }
    }
    const BackCfg &t = CFGS[p.cfg];
    p.mtiles = most_row_blocks(M, L.E, grouped, 16 * t.MT * t.WM);
    p.nblocks = columns(t);
    p.threads = threads(t);
    p.operand_bytes = L.N % 8 != 0 ? round256(size_t(M) * size_t(p.ldy) * 2) : 0;
    p.ws_bytes = p.operand_bytes + (p.ks > 1 ? round256(size_t(p.ks) * size_t(M) * size_t(L.K) * 4) : 0);
    return p;
}

hipError_t launch_f8_backward(const F8Layout &L, const F8BackPlan &p, const F8BackArgs &args, void *workspace, hipStream_t st) {
    F8BackArgs a = args;
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
    a.ldy = p.ldy;
    uint8_t *const space = static_cast<uint8_t *>(workspace);
    a.part = p.ks > 1 ? reinterpret_cast<float *>(space + p.operand_bytes) : nullptr;
    if (p.operand_bytes) {
        uint16_t *const to = reinterpret_cast<uint16_t *>(space);
        hipLaunchKernelGGL(f8_back_copy_kernel, elementwise_grid(int64_t(a.r.rows) * (p.ldy / 8)), dim3(256), 0, st, a.dy, to,
                           int64_t(a.r.rows), a.N, p.ldy);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.dy = to;
    }
    switch (p.cfg) {
        case 0: return launch<0>(a, st);
        case 1: return launch<1>(a, st);
        case 2: return launch<2>(a, st);
        default: return launch<3>(a, st);
    }
}

}  // namespace ql
