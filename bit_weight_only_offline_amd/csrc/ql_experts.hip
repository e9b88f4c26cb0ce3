// Tokens into expert order and back.
//
//   slot (t, j) = t k + j is choice j of token t, with expert ids[t, j]
//   order    counts[e] = slots of expert e;  rows[t, j] = the slot's place among all slots sorted by
//            (expert, slot), -1 for an id that names no expert;  source = the inverse, -1 behind the last
//   dispatch out[rows[t, j]] = x[t], as it is or quantised to e4m3 blocks;  backward: combine without weights
//   combine  out[t] = sum_j w[t, j] y[rows[t, j]], in the order of j
//            backward: dy[rows[t, j]] = w[t, j] dout[t],  dw[t, j] = sum_d dout[t, d] y[rows[t, j], d]
//
// All of them are bound by memory, the small ones by their launches: 4099 tokens of 5000 bf16 values to 6 places each 49 to
// 52 us (5.5 TB/s), 4096 x 4096 back from 8 places 61 us (5.0 TB/s), the gradient of 8192 x 4096 from 2 places 64 us (5.2
// TB/s).  No result depends on the order in which workgroups or atomics run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ql_experts.hpp"
#include "ql_f8_device.hpp"
#include "ql_lds_limit.hpp"

namespace ql {
namespace {

constexpr int ORDER_WAVES = 16;

__device__ inline int expert_of(const OrderArgs &a, int64_t i) {
    if (i >= a.n) return -1;
    const int64_t e = a.wide ? static_cast<const int64_t *>(a.ids)[i] : int64_t(static_cast<const int32_t *>(a.ids)[i]);
    return e >= 0 && e < a.E ? int(e) : -1;
}

// Lanes of the wavefront that hold the same value.
__device__ inline uint64_t same(int e, int bits) {
    uint64_t m = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        m &= ((e >> b) & 1) ? set : ~set;
    }
    return m;
}

// Counts of each workgroup's run, where there are several.
__global__ void __launch_bounds__(1024) order_count_kernel(OrderArgs a) {
    extern __shared__ int32_t hist[];                      // [E]
    for (int e = threadIdx.x; e < a.E; e += 1024) hist[e] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * a.per, last = min(a.n, first + a.per);
    for (int64_t i = first + threadIdx.x; i < last; i += 1024) {
        const int e = expert_of(a, i);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 1024) a.part[int64_t(blockIdx.x) * a.E + e] = hist[e];
}

// A run of slots a workgroup, a part of it to each wavefront in order.  A slot's place is the number of
// slots of smaller experts, of its own in earlier workgroups and wavefronts, and of its own before it in this
// wavefront: the first from the counts, the last from a comparison of ids over the lanes, 64 slots at a time.
// One launch for up to 4096 slots; more have their runs counted by a launch before.
__global__ void __launch_bounds__(64 * ORDER_WAVES) order_place_kernel(OrderArgs a) {
    extern __shared__ int32_t hist[];                      // [ORDER_WAVES][E], later the next place of each; [2][E]
    __shared__ int32_t sums[ORDER_WAVES + 1];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int bits = 1;                                          // of an expert's number; -1 has more set
    while ((a.E - 1) >> bits) ++bits;
    for (int i = tid; i < (ORDER_WAVES + 2) * a.E; i += 64 * ORDER_WAVES) hist[i] = 0;
    __syncthreads();
    int32_t *const everywhere = hist + ORDER_WAVES * a.E, *const earlier = everywhere + a.E;
    if (gridDim.x > 1)
        for (int i = tid; i < int(gridDim.x) * a.E; i += 64 * ORDER_WAVES) {
            const int h = a.part[i], g = i / a.E, e = i - g * a.E;
            if (h) {
                atomicAdd(&everywhere[e], h);
                if (g < int(blockIdx.x)) atomicAdd(&earlier[e], h);
            }
        }
    const int64_t part = a.per / ORDER_WAVES, first = int64_t(blockIdx.x) * a.per + wv * part;
    for (int64_t i = first; i < first + part && i < a.n; i += 64) {
        const int e = expert_of(a, i + lane);
        if (e >= 0) atomicAdd(&hist[wv * a.E + e], 1);
    }
    __syncthreads();

    // thread e: this expert's counts; EXPERTS_MAX threads
    int before = 0, all = 0, own = 0;                      // in earlier workgroups, everywhere, here
    if (tid < a.E) {
        for (int w = 0; w < ORDER_WAVES; ++w) {
            const int h = hist[w * a.E + tid];
            hist[w * a.E + tid] = own;
            own += h;
        }
        all = own;
        if (gridDim.x > 1) {
            all = everywhere[tid];
            before = earlier[tid];
        }
    }
    // experts before this one
    int upto = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d, 64);
        if (lane >= d) upto += o;
    }
    if (lane == 63) sums[wv] = upto;
    __syncthreads();
    if (tid == 0) {
        int run = 0;
        for (int w = 0; w < ORDER_WAVES; ++w) {
            const int s = sums[w];
            sums[w] = run;
            run += s;
        }
        sums[ORDER_WAVES] = run;
    }
    __syncthreads();
    if (tid < a.E) {
        const int base = sums[wv] + upto - all + before;
        for (int w = 0; w < ORDER_WAVES; ++w) hist[w * a.E + tid] += base;
        if (blockIdx.x == 0) a.counts[tid] = all;
    }
    __syncthreads();

    int32_t *const next = hist + wv * a.E;
    for (int64_t i = first; i < first + part && i < a.n; i += 64) {
        const int64_t slot = i + lane;
        const int e = expert_of(a, slot);
        const uint64_t mine = same(e, bits) & __ballot(e >= 0);
        if (e >= 0) {
            const int row = next[e] + __popcll(mine & ((uint64_t(1) << lane) - 1));
            a.rows[slot] = row;
            if (uint32_t(row) < a.n) a.source[row] = int32_t(slot);   // counts in a workspace that another call writes may say otherwise
        } else if (slot < a.n) {
            a.rows[slot] = -1;
        }
        __builtin_amdgcn_wave_barrier();                   // every lane has its place before the counters move on
        if (e >= 0 && (mine >> lane) == 1) next[e] += __popcll(mine);
        __builtin_amdgcn_wave_barrier();
    }
    for (int64_t i = sums[ORDER_WAVES] + int64_t(blockIdx.x) * 1024 + tid; i < a.n; i += int64_t(gridDim.x) * 1024) a.source[i] = -1;
}

// ---- rows ------------------------------------------------------------------------------
// Eight values a thread: a thread reads its piece of the token's row once and writes it to each of the k
// rows.  Rows outside 0 .. T k - 1 are not written.
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs a) {
    const int per_row = (a.D + 7) / 8;
    const int64_t n = a.T * per_row, slots = a.T * a.k;
    const bool f32 = a.f32;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t t = i / per_row;
        const int d = int(i - t * per_row) * 8, count = a.D - d;
        const int32_t *const rows = a.rows + t * a.k;
        if (f32) {
            float v[8];
            load8(a.x, t * a.D + d, count, true, v);
            for (int j = 0; j < a.k; ++j)
                if (const uint32_t r = uint32_t(rows[j]); r < slots) store8(a.out, int64_t(r) * a.D + d, count, true, v);
        } else if (count >= 8) {
            const u32x4_any v = *reinterpret_cast<const u32x4_any *>(static_cast<const uint16_t *>(a.x) + t * a.D + d);
            for (int j = 0; j < a.k; ++j)
                if (const uint32_t r = uint32_t(rows[j]); r < slots)
                    *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(a.out) + int64_t(r) * a.D + d) = v;
        } else {
            for (int j = 0; j < a.k; ++j)
                if (const uint32_t r = uint32_t(rows[j]); r < slots)
                    for (int q = 0; q < count; ++q)
                        static_cast<uint16_t *>(a.out)[int64_t(r) * a.D + d + q] = static_cast<const uint16_t *>(a.x)[t * a.D + d + q];
        }
    }
}

// The same to e4m3 codes: sixteen lanes a block of 128, quantised once and written k times.
__global__ void __launch_bounds__(256) dispatch_f8_kernel(DispatchArgs a) {
    const int kb = (a.D + F8_BLOCK - 1) / F8_BLOCK, l = threadIdx.x & 15;
    const int64_t n = a.T * kb, slots = a.T * a.k;
    const bool f32 = a.f32;
    for (int64_t i = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4); i < n; i += int64_t(gridDim.x) * 16) {
        const int64_t t = i / kb;
        const int b = int(i - t * kb), d = b * F8_BLOCK + 8 * l, count = d < a.D ? 8 : 0;
        float v[8];
        load8(a.x, t * a.D + d, count, f32, v);
        const float s = block_scale(block_amax(v));
        const u32x2 c = BlockDivisor(s).codes(v);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t r = uint32_t(a.rows[t * a.k + j]);
            if (r >= slots) continue;
            if (count) *reinterpret_cast<u32x2 *>(a.codes + int64_t(r) * a.D + d) = c;
            if (l == 0) a.scales[int64_t(r) * kb + b] = s;
        }
    }
}

// Eight values a thread, added up over the token's rows in their order.
template <bool F32>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
    const int per_row = (a.D + 7) / 8;
    const int64_t n = a.T * per_row, slots = a.T * a.k;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t t = i / per_row;
        const int d = int(i - t * per_row) * 8, count = a.D - d;
        float sum[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const uint32_t r = uint32_t(a.rows[t * a.k + j]);
            const bool real = r < slots;
            const float w = a.w ? a.w[t * a.k + j] : 1.0f;
            float v[8];
            load8(a.y, int64_t(real ? r : 0) * a.D + d, real ? count : 0, F32, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) sum[q] = real ? fmaf(w, v[q], sum[q]) : sum[q];
        }
        store8(a.out, t * a.D + d, count, F32, sum);
    }
}

// Gradients: WAVES wavefronts take a token (four for rows of more than 1024 values), read its gradient and each of its
// rows once, write the rows' gradients and keep up to four of the weights' sums at a time.
template <bool F32, int WAVES>
__global__ void __launch_bounds__(256) combine_back_kernel(CombineArgs a) {
    constexpr int PER = 4 / WAVES;                         // tokens of a workgroup
    __shared__ float red[4][4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, in = threadIdx.x % (64 * WAVES);
    const int64_t slots = a.T * a.k;
    for (int64_t t0 = int64_t(blockIdx.x) * PER; t0 < a.T; t0 += int64_t(gridDim.x) * PER) {
        const int64_t t = t0 + wv / WAVES;
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (t < a.T) {
                uint32_t r[4];
                float w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r[j] = j0 + j < a.k ? uint32_t(a.rows[t * a.k + j0 + j]) : ~0u;
                    w[j] = j0 + j < a.k ? a.w[t * a.k + j0 + j] : 0.0f;
                }
                for (int d = in * 8; d < a.D; d += 64 * WAVES * 8) {
                    const int count = a.D - d;
                    float g[8];
                    load8(a.dout, t * a.D + d, count, F32, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (r[j] >= slots) continue;
                        float y[8], dy[8];
                        load8(a.y, int64_t(r[j]) * a.D + d, count, F32, y);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            dot[j] = fmaf(g[q], y[q], dot[j]);
                            dy[q] = w[j] * g[q];
                        }
                        store8(a.dy, int64_t(r[j]) * a.D + d, count, F32, dy);
                    }
                }
            }
#pragma unroll
            for (int s = 32; s >= 1; s >>= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) dot[j] += __shfl_xor(dot[j], s, 64);
            if constexpr (WAVES > 1) {
                __syncthreads();
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j) red[wv][j] = dot[j];
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dot[j] = red[0][j];
#pragma unroll
                    for (int w = 1; w < 4; ++w) dot[j] += red[w][j];
                }
            }
            if (t < a.T && in < 4 && j0 + in < a.k) a.dw[t * a.k + j0 + in] = in == 0 ? dot[0] : in == 1 ? dot[1] : in == 2 ? dot[2] : dot[3];
        }
    }
}

}  // namespace

// One workgroup takes up to 4096 slots, four steps of its wavefronts.  More slots are cut into runs of 1024, one step
// each, after a launch that counts them (24594 slots of 60 experts, from a graph: 7.7 us, 12.0 in runs of 4096), and into longer ones
// past 64 runs, whose counts every workgroup reads.
OrderPlan make_order_plan(int64_t n, int64_t E) {
    OrderPlan p;
    p.per = n <= 4096 ? 4096 : std::max<int64_t>(1024, ceil_div(ceil_div(n, 64), 1024) * 1024);
    p.wgs = std::max<int64_t>(1, ceil_div(n, p.per));
    p.ws_bytes = p.wgs > 1 ? round256(size_t(p.wgs) * size_t(E) * 4) : 0;
    return p;
}

hipError_t launch_expert_order(const OrderArgs &args, const OrderPlan &p, hipStream_t st) {
    OrderArgs a = args;
    // a run's parts are whole steps of 64 slots; a short run is divided over all wavefronts
    a.per = p.wgs > 1 ? p.per : std::max<int64_t>(1024, ceil_div(a.n, 1024) * 1024);
    if (p.wgs > 1) {
        hipLaunchKernelGGL(order_count_kernel, dim3(unsigned(p.wgs)), dim3(1024), size_t(a.E) * 4, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void *)order_place_kernel, int((ORDER_WAVES + 2) * EXPERTS_MAX * 4));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(order_place_kernel, dim3(unsigned(p.wgs)), dim3(64 * ORDER_WAVES), size_t(ORDER_WAVES + 2) * a.E * 4, st, a);
    return hipGetLastError();
}

hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t st) {
    if (a.codes) hipLaunchKernelGGL(dispatch_f8_kernel, elementwise_grid(a.T * ceil_div(a.D, F8_BLOCK) * 16), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(dispatch_kernel, elementwise_grid(a.T * ceil_div(a.D, 8)), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t st) {
    const dim3 grid = elementwise_grid(a.T * ceil_div(a.D, 8));
    if (a.f32) hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineArgs &a, hipStream_t st) {
    // a wavefront covers 512 values at a time; rows of more than 1024 take four
    const bool wide = a.D > 1024;
    const dim3 grid(unsigned(std::min<int64_t>(ceil_div(a.T, wide ? 1 : 4), int64_t(1) << 20)));
    if (a.f32) {
        if (wide) hipLaunchKernelGGL((combine_back_kernel<true, 4>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((combine_back_kernel<true, 1>), grid, dim3(256), 0, st, a);
    } else {
        if (wide) hipLaunchKernelGGL((combine_back_kernel<false, 4>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((combine_back_kernel<false, 1>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace ql
