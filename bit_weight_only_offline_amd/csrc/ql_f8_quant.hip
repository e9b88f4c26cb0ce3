// e4m3 with a float32 scale for each block of 128: activations by rows, weights by 128 x 128, the
// way back, the gradient through the SwiGLU in front, and the packing of weights.
//
//   s = max |x| / 448 (float32),  c = the e4m3 value nearest to x / s;   x = up silu(gate) optionally
//   backward, the quantisation passed straight through, p = logistic(gate):
//   dup = dh gate p,  dgate = dh up p (1 + gate (1 - p))
//
// All of these are bound by memory at large sizes and by their launch at small ones: each value is
// read once, in 16-byte pieces, and each result written once.  Sixteen lanes hold a block, eight
// values each, so its maximum takes four exchanges inside a wavefront and no LDS.  4096 x 14336 in bf16: the gradient
// 103 us (5.7 TB/s), the way back 31 (5.7), quantising 40 (4.5), with the SwiGLU 71 (4.2): there a value's operations
// take nearly as long as its bytes (float32, with twice the bytes: 49 and 97, 6.0 and 5.4 TB/s).  A weight of that size:
// quantising 40 us from bf16 (4.5 TB/s) and 55 from float32 (5.4), packing and unpacking 20 each (5.8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ql_f8_device.hpp"

namespace ql {
namespace {

template <bool SWIGLU>
__global__ void __launch_bounds__(256) f8_quantize_kernel(F8Quant a) {
    const int kb = (a.K + F8_BLOCK - 1) / F8_BLOCK, l = threadIdx.x & 15;
    const int64_t n = a.R * kb, by = int64_t(gridDim.x) * 16;
    const bool f32 = a.f32;
    for (int64_t i = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4); i < n; i += by) {
        const int64_t row = i / kb;
        const int b = int(i - row * kb), k = b * F8_BLOCK + 8 * l;
        const int count = k < a.K ? 8 : 0;
        float v[8];
        if constexpr (SWIGLU) {
            float g[8];
            load8(a.x, row * 2 * a.K + k, count, f32, v);
            load8(a.x, row * 2 * a.K + a.K + k, count, f32, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= gate_act(g[j], GATE_SILU);
        } else {
            load8(a.x, row * a.K + k, count, f32, v);
        }
        const float s = block_scale(block_amax(v));
        const u32x2 c = BlockDivisor(s).codes(v);
        if (count) *reinterpret_cast<u32x2 *>(a.codes + row * a.K + k) = c;
        if (l == 0) a.scales[i] = s;
    }
}

__global__ void __launch_bounds__(256) f8_quantize_back_kernel(const uint16_t *dh, const uint16_t *raw, uint16_t *draw,
                                                               int64_t n, int K) {
    const int per_row = K / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per_row, k = (i - row * per_row) * 8;
        float d[8], u[8], g[8], du[8], dg[8];
        load8(dh, row * K + k, 8, false, d);
        load8(raw, row * 2 * K + k, 8, false, u);
        load8(raw, row * 2 * K + K + k, 8, false, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float act, slope;
            gate_act_grad(g[j], GATE_SILU, act, slope);
            du[j] = d[j] * act;
            dg[j] = d[j] * u[j] * slope;
        }
        store8(draw, row * 2 * K + k, 8, false, du);
        store8(draw, row * 2 * K + K + k, 8, false, dg);
    }
}

__global__ void __launch_bounds__(256) f8_dequantize_kernel(const uint8_t *codes, const float *scales, void *out, int64_t n,
                                                            int K, int f32) {
    const int per_row = K / 8, kb = (K + F8_BLOCK - 1) / F8_BLOCK;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per_row;
        const int k = int(i - row * per_row) * 8;
        const u32x2 c = *reinterpret_cast<const u32x2 *>(codes + row * K + k);
        const float s = scales[row * kb + k / F8_BLOCK];
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[h]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[h]), true);
            v[4 * h] = lo[0] * s;
            v[4 * h + 1] = lo[1] * s;
            v[4 * h + 2] = hi[0] * s;
            v[4 * h + 3] = hi[1] * s;
        }
        store8(out, row * K + k, 8, f32 != 0, v);
    }
}

// A block of 128 x 128 a workgroup, eight values a thread and step, held through the maximum.
__global__ void __launch_bounds__(256) f8_quantize_weight_kernel(const void *w, int f32, uint8_t *codes, float *scales,
                                                                 int64_t blocks, int nbs, int kbs, int N, int K) {
    __shared__ float red[4];
    const int l = threadIdx.x & 15, r = threadIdx.x >> 4;
    for (int64_t i = blockIdx.x; i < blocks; i += gridDim.x) {
        const int64_t en = i / kbs;
        const int b = int(i - en * kbs), k = b * F8_BLOCK + 8 * l;
        const int64_t e = en / nbs;
        const int n0 = int(en - e * nbs) * F8_BLOCK;
        float v[8][8];
        float m = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int n = n0 + 16 * q + r;
            load8(w, (e * N + n) * K + k, n < N && k < K ? 8 : 0, f32 != 0, v[q]);
            m = fmaxf(m, block_amax(v[q]));
        }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        const float s = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const BlockDivisor by(s);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int n = n0 + 16 * q + r;
            if (n < N && k < K) *reinterpret_cast<u32x2 *>(codes + (e * N + n) * K + k) = by.codes(v[q]);
        }
        if (threadIdx.x == 0) scales[i] = s;
    }
}

// Sixteen bytes of the packed weight a thread: expert, tile, block, half and lane in that order.
template <bool PACK>
__global__ void __launch_bounds__(256) f8_pack_kernel(const uint8_t *from, uint8_t *to, int64_t n, int ntiles, int kblocks,
                                                      int N, int K) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t unit = i >> 7, tile = unit / kblocks;
        const int lane = int(i & 63), half = int(i >> 6) & 1, b = int(unit - tile * kblocks);
        const int64_t e = tile / ntiles;
        const int c = int(tile - e * ntiles) * TILE_N + (lane & 15), k = b * F8_BLOCK + 64 * half + 16 * (lane >> 4);
        const bool real = c < N && k < K;
        const int64_t at = (e * N + c) * K + k;
        if constexpr (PACK)
            *reinterpret_cast<u32x4 *>(to + 16 * i) = real ? *reinterpret_cast<const u32x4 *>(from + at) : u32x4{0u, 0u, 0u, 0u};
        else if (real)
            *reinterpret_cast<u32x4 *>(to + at) = *reinterpret_cast<const u32x4 *>(from + 16 * i);
    }
}

}  // namespace

hipError_t launch_f8_quantize(const F8Quant &a, hipStream_t st) {
    const int64_t threads = a.R * ceil_div(a.K, F8_BLOCK) * 16;
    if (a.swiglu) hipLaunchKernelGGL(f8_quantize_kernel<true>, elementwise_grid(threads), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(f8_quantize_kernel<false>, elementwise_grid(threads), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_f8_quantize_backward(const uint16_t *dh, const uint16_t *raw, uint16_t *draw, int64_t R, int K,
                                       hipStream_t st) {
    const int64_t n = R * (K / 8);
    hipLaunchKernelGGL(f8_quantize_back_kernel, elementwise_grid(n), dim3(256), 0, st, dh, raw, draw, n, K);
    return hipGetLastError();
}

hipError_t launch_f8_dequantize(const uint8_t *codes, const float *scales, void *out, int64_t R, int K, bool f32,
                                hipStream_t st) {
    const int64_t n = R * (K / 8);
    hipLaunchKernelGGL(f8_dequantize_kernel, elementwise_grid(n), dim3(256), 0, st, codes, scales, out, n, K, f32 ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_f8_quantize_weight(const F8Layout &L, const void *w, bool f32, uint8_t *codes, float *scales,
                                     hipStream_t st) {
    const int64_t blocks = L.E * L.nblocks * L.kblocks;
    hipLaunchKernelGGL(f8_quantize_weight_kernel, elementwise_grid(blocks * 256), dim3(256), 0, st, w, f32 ? 1 : 0, codes,
                       scales, blocks, int(L.nblocks), int(L.kblocks), int(L.N), int(L.K));
    return hipGetLastError();
}

hipError_t launch_f8_pack(const F8Layout &L, const uint8_t *codes, uint8_t *packed, hipStream_t st) {
    const int64_t n = L.E * int64_t(L.w_bytes / 16);
    hipLaunchKernelGGL(f8_pack_kernel<true>, elementwise_grid(n), dim3(256), 0, st, codes, packed, n, int(L.ntiles),
                       int(L.kblocks), int(L.N), int(L.K));
    return hipGetLastError();
}

hipError_t launch_f8_unpack(const F8Layout &L, const uint8_t *packed, uint8_t *codes, hipStream_t st) {
    const int64_t n = L.E * int64_t(L.w_bytes / 16);
    hipLaunchKernelGGL(f8_pack_kernel<false>, elementwise_grid(n), dim3(256), 0, st, packed, codes, n, int(L.ntiles),
                       int(L.kblocks), int(L.N), int(L.K));
    return hipGetLastError();
}

}  // namespace ql
