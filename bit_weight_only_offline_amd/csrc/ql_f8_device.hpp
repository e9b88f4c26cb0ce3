// Device code that the block-scaled e4m3 kernels share: the quantisation of eight values a lane,
// and how a grouped product's workgroup finds its rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_f8.hpp"

namespace ql {

// The largest magnitude of the 128 values of a block, eight in each of sixteen lanes; infinity if
// one is NaN.  Magnitudes compare as integers do, and NaN lies above them all (a maximum of floats would drop it).  The
// sixteen lanes are a row of the wavefront, whose rotations need no LDS.
template <int BY>
__device__ inline uint32_t row_rotate(uint32_t m) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x120 + BY, 0xF, 0xF, true));
}
__device__ inline float block_amax(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = max(m, row_rotate<8>(m));
    m = max(m, row_rotate<4>(m));
    m = max(m, row_rotate<2>(m));
    m = max(m, row_rotate<1>(m));
    return __uint_as_float(min(m, 0x7F800000u));
}

// amax / 448; NaN for a block with NaN or infinity, whose codes are then 0.
__device__ inline float block_scale(float amax) {
    return amax < INFINITY ? __fdiv_rn(amax, F8_MAX) : __uint_as_float(0x7FC00000u);
}

// Codes of v / s, each the e4m3 value nearest to the exact quotient (ties to even).
//
// A quotient rounded to float32 first may land on the border between two codes from either side;
// bf16 values in particular often lie next to one.  So the quotient, taken by a reciprocal (off by one unit of its
// last place itself) and off by at most four, is rounded to a multiple q of sixteen units, which every border is; the sign of the remainder
// v - q s, which one fused operation gives whatever its size, says on which side of q the exact quotient lies, less
// than sixteen units away, and q is moved by one unit to that side.  The mantissa of s alone is divided by:
// scales at the ends of float32's range stay exact.  Nine operations a value; a value's three bytes leave time for about
// twenty, which reading it, its maximum and its address take some of.
struct BlockDivisor {
    float s, inv;
    int e;
    bool some;
    __device__ explicit BlockDivisor(float scale) {
        some = scale > 0.0f;                               // neither 0 nor NaN
        int x = 0;
        s = some ? frexpf(scale, &x) : 1.0f;
        e = -x;
        inv = __builtin_amdgcn_rcpf(s);
    }
    __device__ float quotient(float v) const {
        const float a = ldexpf(fabsf(v), e);
        const int q = (__float_as_int(a * inv) + 8) & ~15;
        const int r = __float_as_int(fmaf(-__int_as_float(q), s, a));   // negative, zero or positive as an integer too
        const int b = min(q + min(max(r, -1), 1), __float_as_int(F8_MAX));    // a scale with few bits may leave more
        return copysignf(__int_as_float(b), v);
    }
    __device__ u32x2 codes(const float (&v)[8]) const {
        if (!some) return u32x2{0u, 0u};
        u32x2 c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = 0;
            w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h]), quotient(v[4 * h + 1]), w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h + 2]), quotient(v[4 * h + 3]), w, true);
            c[h] = uint32_t(w);
        }
        return c;
    }
};

// Eight values of a row at any element's address, of which the first `count` exist; zeros behind them.
__device__ inline void load8(const void *p, int64_t i, int count, bool f32, float (&v)[8]) {
    if (count >= 8) {
        if (f32) {
            const float *q = static_cast<const float *>(p) + i;
            const f32x4_any a = *reinterpret_cast<const f32x4_any *>(q), b = *reinterpret_cast<const f32x4_any *>(q + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
        } else {
            const u32x4_any a = *reinterpret_cast<const u32x4_any *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = bf16_bits_to_f32((a[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (j < count)
            v[j] = f32 ? static_cast<const float *>(p)[i + j] : bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i + j]);
    }
}
__device__ inline void store8(void *p, int64_t i, int count, bool f32, const float (&v)[8]) {
    if (count >= 8) {
        if (f32) {
            float *q = static_cast<float *>(p) + i;
            *reinterpret_cast<f32x4_any *>(q) = f32x4_any{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_any *>(q + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(p) + i) =
                u32x4_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < count) {
            if (f32) static_cast<float *>(p)[i + j] = v[j];
            else static_cast<__bf16 *>(p)[i + j] = (__bf16)v[j];
        }
}

// Where the rows of a workgroup lie: `first` .. first + count - 1 of expert `expert`.
struct RowBlock {
    int expert, first, count;
};

// Row block `at` of blocks of `block` rows, expert after expert, and the number of all.  A plain
// product has one expert.  Every wavefront scans the counts by itself, 64 at a time: a load and two
// scans of six steps for up to 64 experts, about a microsecond, less than another launch takes.  With 256 experts of
// 4096 x 7168, 8 rows of 8 of them take 40.5 us and 64 rows of 64 303: the weights' bytes take 39 and 315 at 5.97 TB/s.  A
// negative count is 0, and counts past the rows are clipped.
__device__ inline int64_t scan64(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ inline bool find_rows(const F8Rows &r, int block, int at, int lane, RowBlock &found, int &blocks) {
    if (!r.counts) {
        blocks = (r.rows + block - 1) / block;
        found = RowBlock{0, at * block, min(block, r.rows - at * block)};
        return at < blocks;
    }
    int64_t rows = 0;
    int done = 0;
    bool have = false;
    for (int e0 = 0; e0 < r.E; e0 += 64) {
        const int own = e0 + lane < r.E ? min(max(r.counts[e0 + lane], 0), r.rows) : 0;
        const int64_t upto = rows + scan64(own, lane);
        const int start = int(min(upto - own, int64_t(r.rows))), end = int(min(upto, int64_t(r.rows)));
        const int mine = (end - start + block - 1) / block;
        const int last = done + int(scan64(mine, lane)), first = last - mine;
        const uint64_t here = __ballot(at >= first && at < last);
        if (here) {
            const int l = __builtin_amdgcn_readfirstlane(__builtin_ctzll(here));
            const int s = __shfl(start, l, 64), n = __shfl(end, l, 64), f = __shfl(first, l, 64);
            const int row = s + (at - f) * block;
            found = RowBlock{e0 + l, __builtin_amdgcn_readfirstlane(row), __builtin_amdgcn_readfirstlane(min(block, n - row))};
            have = true;
        }
        rows = min(__shfl(upto, 63, 64), int64_t(r.rows));
        done = __builtin_amdgcn_readfirstlane(__shfl(last, 63, 64));
    }
    blocks = done;
    return have;
}

}  // namespace ql
