// Packing of per-channel INT8 weights into operand tiles, and its exact inverse.  Runs
// once per weight; one thread per 16-byte operand slice, bytes read one by one so that
// the canonical rows need no alignment.
#include <hip/hip_runtime.h>

#include "ql_decode.hpp"
#include "ql_i8.hpp"

namespace ql {
namespace {

__global__ void __launch_bounds__(256) i8_pack_kernel(const int8_t *__restrict__ codes, const int8_t *__restrict__ gate,
                                                      int64_t N, int64_t K, int64_t kchunks, int64_t slices,
                                                      uint8_t *__restrict__ pw) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < slices; i += int64_t(gridDim.x) * 256) {
        const int lane = int(i & 63);
        const int64_t blk = i >> 6, tile = blk / kchunks, kc = blk % kchunks;
        const int8_t *src = (gate && (tile & 1)) ? gate : codes;
        const int64_t n = (gate ? tile >> 1 : tile) * TILE_N + (lane & 15);
        const int64_t k0 = kc * I8_CHUNK + 16 * (lane >> 4);
        u32x4 v{0u, 0u, 0u, 0u};
        if (n < N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k0 + j < K) v[j >> 2] |= uint32_t(uint8_t(src[n * K + k0 + j])) << (8 * (j & 3));
        }
        reinterpret_cast<u32x4 *>(pw)[i] = v;
    }
}

__global__ void __launch_bounds__(256) i8_pack_scales_kernel(const float *__restrict__ s, const float *__restrict__ gs,
                                                             int64_t N, int64_t n_packed, float *__restrict__ ps) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n_packed) return;
    const int64_t tile = i / TILE_N;
    const int64_t n = (gs ? tile >> 1 : tile) * TILE_N + i % TILE_N;
    ps[i] = n < N ? ((gs && (tile & 1)) ? gs[n] : s[n]) : 0.0f;
}

__global__ void __launch_bounds__(256) i8_unpack_kernel(const uint8_t *__restrict__ pw, int64_t N, int64_t K,
                                                        int64_t kchunks, int64_t slices, int8_t *__restrict__ codes,
                                                        int8_t *__restrict__ gate) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < slices; i += int64_t(gridDim.x) * 256) {
        const int lane = int(i & 63);
        const int64_t blk = i >> 6, tile = blk / kchunks, kc = blk % kchunks;
        int8_t *dst = (gate && (tile & 1)) ? gate : codes;
        const int64_t n = (gate ? tile >> 1 : tile) * TILE_N + (lane & 15);
        const int64_t k0 = kc * I8_CHUNK + 16 * (lane >> 4);
        if (n >= N) continue;
        const u32x4 v = reinterpret_cast<const u32x4 *>(pw)[i];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (k0 + j < K) dst[n * K + k0 + j] = int8_t(v[j >> 2] >> (8 * (j & 3)));
    }
}

__global__ void __launch_bounds__(256) i8_unpack_scales_kernel(const float *__restrict__ ps, int64_t N, int64_t n_packed,
                                                               float *__restrict__ s, float *__restrict__ gs) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n_packed) return;
    const int64_t tile = i / TILE_N;
    const int64_t n = (gs ? tile >> 1 : tile) * TILE_N + i % TILE_N;
    if (n < N) ((gs && (tile & 1)) ? gs : s)[n] = ps[i];
}

}  // namespace

hipError_t launch_i8_pack(const I8Layout &L, const int8_t *codes, const float *scales, const int8_t *gate_codes,
                          const float *gate_scales, void *pw, void *ps, hipStream_t st) {
    const int64_t slices = int64_t(L.w_bytes / 16), np = L.ntiles * TILE_N;
    hipLaunchKernelGGL(i8_pack_kernel, elementwise_grid(slices), dim3(256), 0, st, codes, gate_codes, L.N,
                       L.K, L.kchunks, slices, static_cast<uint8_t *>(pw));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(i8_pack_scales_kernel, elementwise_grid(np), dim3(256), 0, st, scales, gate_scales,
                       L.N, np, static_cast<float *>(ps));
    return hipGetLastError();
}

hipError_t launch_i8_unpack(const I8Layout &L, const void *pw, const void *ps, int8_t *codes, float *scales,
                            int8_t *gate_codes, float *gate_scales, hipStream_t st) {
    const int64_t slices = int64_t(L.w_bytes / 16), np = L.ntiles * TILE_N;
    hipLaunchKernelGGL(i8_unpack_kernel, elementwise_grid(slices), dim3(256), 0, st,
                       static_cast<const uint8_t *>(pw), L.N, L.K, L.kchunks, slices, codes, gate_codes);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(i8_unpack_scales_kernel, elementwise_grid(np), dim3(256), 0, st,
                       static_cast<const float *>(ps), L.N, np, scales, gate_scales);
    return hipGetLastError();
}

}  // namespace ql
