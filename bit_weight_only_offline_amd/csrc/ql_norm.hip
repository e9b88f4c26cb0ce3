// Norms before and after a block, fused with the block's gate and the residual scale.
//
//   t  = y rsqrt(mean y^2 + eps) w_post        the block's output, normed (or t = y)
//   r' = alpha r + gate t                      the residual stream
//   x  = r' rsqrt(mean r'^2 + eps) w_pre       the next block's input, as bf16 or as int8
//                                              codes with one scale a row (s = max|x| / 127)
//
// Backward, with v = y ip and u = r' iq the normed rows (ip, iq the inverse norms):
//   D  = dr' + iq (n - u mean(n u)),  n = dx w_pre;     dr = alpha D
//   dv = D gate w_post;  dy = ip (dv - v mean(dv v))
//   dw_pre = sum_rows dx u,  dw_post = sum_rows D gate v,  dgate = sum_rows D v w_post
//
// Both are bound by memory: each row is read once, held in registers in float32 through all
// of its reductions, and written once.  x is formed from the float32 r', not from its
// rounded copy.  One workgroup walks several rows, so the weight vectors stay in registers and
// the next row is on its way while this one is reduced.  8192 x 4096, float32 stream: 79 us,
// 5.1 TB/s; backward, bf16 stream: 87 us, 4.6 TB/s, and 5.5 us for the column sums.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ql_act.hpp"
#include "ql_decode.hpp"
#include "ql_launch.hpp"
#include "ql_norm.hpp"

namespace ql {
namespace {

// Rows are read and written through ranged buffers of exactly their own bytes: what lies past
// the row's end, or belongs to an absent tensor (no bytes at all), reads as zero and is not
// written, so no access is predicated.  (The whole offset stands in the lane's part of the
// address: the scalar part takes no part in the range check.)
// Zeros past the end add nothing to any sum, and whatever is formed from them stays there.
template <int V>
struct Raw { uint32_t w[V == 8 ? 8 : 1]; };   // V values as stored: bf16 (half used) or float32

__device__ inline __amdgpu_buffer_rsrc_t row_of(const void *p, int64_t row, int C, bool f32) {
    const int64_t es = f32 ? 4 : 2;
    return make_rsrc(static_cast<const uint8_t *>(p) + row * C * es, p ? uint32_t(C) * uint32_t(es) : 0u);
}

// V values at element `lane + skip` of a row; V = 8 needs 16-byte aligned rows
template <int V>
__device__ inline Raw<V> load_raw(__amdgpu_buffer_rsrc_t p, int lane, int skip, bool f32) {
    Raw<V> r;
    if constexpr (V == 8) {
        if (f32) {
            const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(p, (lane + skip) * 4, 0, 0);
            const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(p, (lane + skip) * 4 + 16, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) { r.w[j] = a[j]; r.w[4 + j] = b[j]; }
        } else {
            const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(p, (lane + skip) * 2, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[j] = a[j];
        }
    } else {
        r.w[0] = f32 ? __builtin_amdgcn_raw_buffer_load_b32(p, (lane + skip) * 4, 0, 0)
                     : uint32_t(__builtin_amdgcn_raw_buffer_load_b16(p, (lane + skip) * 2, 0, 0));
    }
    return r;
}
template <int V>
__device__ inline void widen(const Raw<V> &r, bool f32, float *v) {
    if constexpr (V == 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = f32 ? __uint_as_float(r.w[j]) : bf16_bits_to_f32((r.w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
    } else {
        v[0] = f32 ? __uint_as_float(r.w[0]) : bf16_bits_to_f32(r.w[0]);
    }
}
template <int V>
__device__ inline void store_row(__amdgpu_buffer_rsrc_t p, int lane, int skip, bool f32, const float *v) {
    if constexpr (V == 8) {
        if (f32) {
            const u32x4 a{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            const u32x4 b{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
            __builtin_amdgcn_raw_buffer_store_b128(a, p, (lane + skip) * 4, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(b, p, (lane + skip) * 4 + 16, 0, 0);
        } else {
            const u32x4 a{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
            __builtin_amdgcn_raw_buffer_store_b128(a, p, (lane + skip) * 2, 0, 0);
        }
    } else {
        if (f32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), p, (lane + skip) * 4, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (__bf16)v[0]), p, (lane + skip) * 2, 0, 0);
    }
}

// Workgroup-wide sums (or maxima) of N values: a shuffle tree in each wavefront, then every
// thread adds the wavefronts' values in the same order.  `red` alternates between two
// halves, so one barrier a reduction is enough: a half is written again only after the
// barrier of the reduction in between.
template <int N, bool MAX>
__device__ inline void reduce(float (&v)[N], float *red, int &turn, int waves) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o = __shfl_xor(v[i], d, 64);
            v[i] = MAX ? fmaxf(v[i], o) : v[i] + o;
        }
    if (waves == 1) return;
    float *half = red + turn * (16 * 4);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) half[(threadIdx.x >> 6) * 4 + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = half[i];
    for (int w = 1; w < waves; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = MAX ? fmaxf(v[i], half[w * 4 + i]) : v[i] + half[w * 4 + i];
}

// ---- forward ---------------------------------------------------------------------------
// V values per load, NV loads per thread and row: load v covers values (v T + t) V ..; rows
// of up to 8 values a thread keep their weight vectors in registers and fetch a row ahead,
// longer ones read the vectors again for each row.
template <int V, int NV, int TMAX, bool RF32>
__global__ void __launch_bounds__(TMAX) block_norm_kernel(NormArgs a) {
    constexpr int E = V * NV;
    constexpr bool KEEP = E <= 8;
    __shared__ float red[2 * 16 * 4];
    const int T = blockDim.x, waves = T >> 6, t = threadIdx.x * V;
    int turn = 0;
    const int64_t row0 = blockIdx.x, row1 = a.R, by = gridDim.x;
    const float inv_c = 1.0f / float(a.C);
    const bool pf32 = !a.p_bf16;

    const int step = T * V;
    // vector `index` of a parameter, ones where it is absent
    auto param = [&](const void *p, int64_t index, int v, float *out) {
        if (p) widen<V>(load_raw<V>(row_of(p, index, a.C, pf32), t, v * step, pf32), pf32, out);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = 1.0f;
    };
    float post[KEEP ? E : V], pre[KEEP ? E : V], gate[KEEP ? E : V];
    if constexpr (KEEP) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            param(a.post, 0, v, post + v * V);
            param(a.pre, 0, v, pre + v * V);
        }
    }
    int64_t gate_of = -1;

    Raw<V> ny[NV], nr[NV];
    auto fetch = [&](int64_t row) {
        const __amdgpu_buffer_rsrc_t py = row_of(a.y, row, a.C, false), pr = row_of(a.r, row, a.C, RF32);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ny[v] = load_raw<V>(py, t, v * step, false);
            nr[v] = load_raw<V>(pr, t, v * step, RF32);
        }
    };
    if (KEEP && row0 < row1) fetch(row0);
    for (int64_t row = row0; row < row1; row += by) {
        float y[E], r[E];
        if (!KEEP) fetch(row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            widen<V>(ny[v], false, y + v * V);
            widen<V>(nr[v], RF32, r + v * V);
        }
        if (KEEP && row + by < row1) fetch(row + by);

        if (a.y) {
            float ip = 1.0f;
            if (a.post) {
                float ss[1] = {0.0f};
#pragma unroll
                for (int e = 0; e < E; ++e) ss[0] = fmaf(y[e], y[e], ss[0]);
                reduce<1, false>(ss, red, turn, waves);
                ip = rsqrtf(fmaf(ss[0], inv_c, a.eps));
            }
            const int64_t gb = a.gate_rows ? row / a.gate_rows : 0;
            const bool new_gate = gb != gate_of;
            gate_of = gb;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float *w = KEEP ? post + v * V : post, *g = KEEP ? gate + v * V : gate;
                if (!KEEP) param(a.post, 0, v, w);
                if (!KEEP || new_gate) param(a.gate, gb, v, g);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    r[v * V + j] = fmaf(g[j], y[v * V + j] * ip * w[j], a.alpha * r[v * V + j]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] *= a.alpha;
        }
        const __amdgpu_buffer_rsrc_t po = row_of(a.r_out, row, a.C, RF32);
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row<V>(po, t, v * step, RF32, r + v * V);
        if (!a.pre) continue;

        float ss[1] = {0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) ss[0] = fmaf(r[e], r[e], ss[0]);
        reduce<1, false>(ss, red, turn, waves);
        const float iq = rsqrtf(fmaf(ss[0], inv_c, a.eps));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float *w = KEEP ? pre + v * V : pre;
            if (!KEEP) param(a.pre, 0, v, w);
#pragma unroll
            for (int j = 0; j < V; ++j) r[v * V + j] = r[v * V + j] * iq * w[j];
        }
        if (a.x) {
            const __amdgpu_buffer_rsrc_t px = row_of(a.x, row, a.C, false);
#pragma unroll
            for (int v = 0; v < NV; ++v) store_row<V>(px, t, v * step, false, r + v * V);
            continue;
        }
        float am[1] = {0.0f};
        bool bad = false;                               // a maximum would drop NaN
#pragma unroll
        for (int e = 0; e < E; ++e) {
            am[0] = fmaxf(am[0], fabsf(r[e]));
            bad |= r[e] != r[e];
        }
        if (bad) am[0] = INFINITY;
        reduce<1, true>(am, red, turn, waves);
        // a row with NaN or infinity has the scale NaN and codes 0, so its products are NaN
        const float s = am[0] < INFINITY ? __fdiv_rn(am[0], 127.0f) : __uint_as_float(0x7FC00000u);
        if (threadIdx.x == 0) a.scales[row] = s;
        const __amdgpu_buffer_rsrc_t pq = make_rsrc(a.codes + int64_t(row) * a.C, uint32_t(a.C));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            uint32_t q[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(r[v * V + j], s)), -127.0f), 127.0f) : 0.0f;
                q[j >> 2] |= (uint32_t(int(f)) & 0xFFu) << (8 * (j & 3));
            }
            if constexpr (V == 8) __builtin_amdgcn_raw_buffer_store_b64(u32x2{q[0], q[1]}, pq, t + v * step, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b8((unsigned char)q[0], pq, t + v * step, 0, 0);
        }
    }
}

// ---- backward --------------------------------------------------------------------------
// Workgroup i walks every cpb-th row of one gate (from i mod cpb, gate i / cpb), or, where there are
// more gates than workgroups (cpb = 1), all rows of gpw gates.  The column sums stay in
// registers and leave once a workgroup (dgate: once a gate where cpb = 1).
template <int V, int NV, int TMAX, bool RF32>
__global__ void __launch_bounds__(TMAX, NV <= (V == 8 ? 1 : 4) ? 4 : 1) block_norm_back_kernel(NormBackArgs a) {
    constexpr int E = V * NV;
    constexpr bool KEEP = E <= 8;
    __shared__ float red[2 * 16 * 4];
    const int T = blockDim.x, waves = T >> 6, t = threadIdx.x * V;
    int turn = 0;
    const float inv_c = 1.0f / float(a.C);
    const bool pf32 = !a.p_bf16;
    const int i = blockIdx.x;
    int64_t row0, row1, by;
    if (a.cpb > 1) {
        row0 = int64_t(i / a.cpb) * a.gate_rows + i % a.cpb;
        row1 = int64_t(i / a.cpb + 1) * a.gate_rows;
        by = a.cpb;
    } else {
        row0 = int64_t(i) * a.rows_per_wg;
        row1 = min(int64_t(a.R), row0 + a.rows_per_wg);
        by = 1;
    }

    const int step = T * V;
    auto param = [&](const void *p, int64_t index, int v, float *out) {
        if (p) widen<V>(load_raw<V>(row_of(p, index, a.C, pf32), t, v * step, pf32), pf32, out);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = 1.0f;
    };
    auto sums_out = [&](float *dst, int64_t index, const float *v0) {
        const __amdgpu_buffer_rsrc_t p = row_of(dst, index, a.C, true);
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row<V>(p, t, v * step, true, v0 + v * V);
    };
    float post[KEEP ? E : V], pre[KEEP ? E : V], gate[KEEP ? E : V];
    if constexpr (KEEP) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            param(a.post, 0, v, post + v * V);
            param(a.pre, 0, v, pre + v * V);
        }
    }
    int64_t gate_of = -1;
    float s_post[E], s_pre[E], s_gate[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s_post[e] = s_pre[e] = s_gate[e] = 0.0f;

    Raw<V> ny[NV], nr[NV], nx[NV], nd[NV];
    auto fetch = [&](int64_t row) {
        const __amdgpu_buffer_rsrc_t py = row_of(a.y, row, a.C, false), pr = row_of(a.pre ? a.r : nullptr, row, a.C, RF32),
                                     px = row_of(a.dx, row, a.C, false), pd = row_of(a.dres, row, a.C, RF32);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ny[v] = load_raw<V>(py, t, v * step, false);
            nr[v] = load_raw<V>(pr, t, v * step, RF32);
            nx[v] = load_raw<V>(px, t, v * step, false);
            nd[v] = load_raw<V>(pd, t, v * step, RF32);
        }
    };
    if (KEEP && row0 < row1) fetch(row0);
    for (int64_t row = row0; row < row1; row += by) {
        float y[E], r[E], x[E], d[E];
        if (!KEEP) fetch(row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            widen<V>(ny[v], false, y + v * V);
            widen<V>(nr[v], RF32, r + v * V);
            widen<V>(nx[v], false, x + v * V);
            widen<V>(nd[v], RF32, d + v * V);
        }
        if (KEEP && row + by < row1) fetch(row + by);

        // n = dx w_pre replaces x in the second half: x itself is needed for dw_pre
        float ss[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float *w = KEEP ? pre + v * V : pre;
            if (!KEEP) param(a.pre, 0, v, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = v * V + j;
                ss[0] = fmaf(y[e], y[e], ss[0]);
                ss[1] = fmaf(r[e], r[e], ss[1]);
                ss[2] = fmaf(x[e] * w[j], r[e], ss[2]);
            }
        }
        reduce<3, false>(ss, red, turn, waves);
        const float ip = a.post ? rsqrtf(fmaf(ss[0], inv_c, a.eps)) : 1.0f;
        if (a.pre) {
            const float iq = rsqrtf(fmaf(ss[1], inv_c, a.eps));
            const float along = ss[2] * iq * inv_c;          // mean(n u)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float *w = KEEP ? pre + v * V : pre;
                if (!KEEP) param(a.pre, 0, v, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = v * V + j;
                    const float u = r[e] * iq;
                    d[e] = fmaf(iq, x[e] * w[j] - u * along, d[e]);
                    s_pre[e] = fmaf(x[e], u, s_pre[e]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = a.alpha * d[e];
        const __amdgpu_buffer_rsrc_t po = row_of(a.dr, row, a.C, RF32);
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row<V>(po, t, v * step, RF32, r + v * V);
        if (!a.y) continue;

        const int64_t gb = a.gate_rows ? row / a.gate_rows : 0;
        const bool new_gate = gb != gate_of;
        gate_of = gb;
        float dot[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float *w = KEEP ? post + v * V : post, *g = KEEP ? gate + v * V : gate;
            if (!KEEP) param(a.post, 0, v, w);
            if (!KEEP || new_gate) param(a.gate, gb, v, g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = v * V + j;
                const float u = y[e] * ip;
                s_gate[e] = fmaf(d[e] * w[j], u, s_gate[e]);
                const float dt = d[e] * g[j];
                s_post[e] = fmaf(dt, u, s_post[e]);
                d[e] = dt * w[j];
                dot[0] = fmaf(d[e], u, dot[0]);
            }
        }
        if (a.post) {
            reduce<1, false>(dot, red, turn, waves);
            const float along = dot[0] * inv_c;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = ip * (d[e] - y[e] * ip * along);
        }
        const __amdgpu_buffer_rsrc_t pz = row_of(a.dy, row, a.C, false);
#pragma unroll
        for (int v = 0; v < NV; ++v) store_row<V>(pz, t, v * step, false, d + v * V);
        if (a.dgate && (row + 1) % a.gate_rows == 0) {        // this gate is complete
            sums_out(a.dgate, gb, s_gate);
#pragma unroll
            for (int e = 0; e < E; ++e) s_gate[e] = 0.0f;
        }
    }
    if (a.part_post) sums_out(a.part_post, i, s_post);
    if (a.part_pre) sums_out(a.part_pre, i, s_pre);
    if (a.part_gate) sums_out(a.part_gate, i, s_gate);
}

// out[b][c] = sum over `count` consecutive rows of part, in a fixed order: 16 row groups of
// one workgroup take every 16th row, then the groups are added in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(ColumnSums a) {
    __shared__ float red[16][64];
    const int q = blockIdx.z, lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t c = int64_t(blockIdx.x) * 64 + lane;
    for (int64_t b = blockIdx.y; b < a.outs[q]; b += gridDim.y) {
        const float *p = a.part[q] + b * a.count[q] * a.C;
        float s = 0.0f;
        if (c < a.C)
#pragma unroll 8
            for (int g = grp; g < a.count[q]; g += 16) s += p[int64_t(g) * a.C + c];
        red[grp][lane] = s;
        __syncthreads();
        if (grp == 0 && c < a.C) {
            float t = red[0][lane];
#pragma unroll
            for (int g = 1; g < 16; ++g) t += red[g][lane];
            a.out[q][b * a.C + c] = t;
        }
        __syncthreads();
    }
}

// The least number of loads per thread among those compiled with which `most` threads cover
// a row, and that many threads in whole wavefronts.
template <int N>
int loads_per_thread(int64_t C, int V, int most, const int (&choices)[N], int &T) {
    int nv = choices[N - 1];
    for (int i = N - 1; i >= 0; --i)
        if (int64_t(choices[i]) * V * most >= C) nv = choices[i];
    T = int(ceil_div(ceil_div(C, int64_t(V) * nv), 64) * 64);
    return nv;
}

template <int V, int NV, int TMAX>
hipError_t launch_fwd(const NormArgs &a, int T, int wgs, hipStream_t st) {
    if (a.r_f32) hipLaunchKernelGGL((block_norm_kernel<V, NV, TMAX, true>), dim3(wgs), dim3(T), 0, st, a);
    else hipLaunchKernelGGL((block_norm_kernel<V, NV, TMAX, false>), dim3(wgs), dim3(T), 0, st, a);
    return hipGetLastError();
}
template <int V, int NV, int TMAX>
hipError_t launch_bwd(const NormBackArgs &a, int T, int wgs, hipStream_t st) {
    if (a.r_f32) hipLaunchKernelGGL((block_norm_back_kernel<V, NV, TMAX, true>), dim3(wgs), dim3(T), 0, st, a);
    else hipLaunchKernelGGL((block_norm_back_kernel<V, NV, TMAX, false>), dim3(wgs), dim3(T), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &args, bool vec, hipStream_t st) {
    NormArgs a = args;
    int T, NV;
    // as few values a thread as 512 threads allow (a short row's latency), then 1024 threads
    if (vec) NV = loads_per_thread(a.C, 8, a.C > 512 * 16 ? 1024 : 512, {1, 2, 4}, T);
    else NV = loads_per_thread(a.C, 1, a.C > 512 * 16 ? 1024 : 512, {4, 8, 16, 32}, T);
    // Workgroup i takes rows i, i + grid, ..: rows in flight together are neighbours in memory
    // (runs of rows to each instead: 95 against 79 us for 8192 x 4096 from memory).
    const int grid = int(std::min<int64_t>(a.R, 512 * (2048 / std::max(T, 256))));
    if (vec) {
        if (NV == 1) return launch_fwd<8, 1, 1024>(a, T, grid, st);
        if (NV == 2) return launch_fwd<8, 2, 1024>(a, T, grid, st);
        return launch_fwd<8, 4, 1024>(a, T, grid, st);
    }
    if (NV == 4) return launch_fwd<1, 4, 512>(a, T, grid, st);
    if (NV == 8) return launch_fwd<1, 8, 1024>(a, T, grid, st);
    if (NV == 16) return launch_fwd<1, 16, 1024>(a, T, grid, st);
    return launch_fwd<1, 32, 1024>(a, T, grid, st);
}

NormBackPlan make_norm_back_plan(int64_t R, int64_t C, int64_t gates) {
    NormBackPlan p;
    const int64_t target = std::min<int64_t>(std::max<int64_t>(R, 1), 512);
    const int64_t B = gates > 0 ? gates : 1, gr = R / B;
    p.gate_rows = gr;
    if (R > 0 && B >= target) {
        p.cpb = 1;
        p.rows_per_wg = ceil_div(B, target) * gr;
        p.wgs = ceil_div(R, p.rows_per_wg);
    } else {
        const int64_t want = ceil_div(target, B);
        p.rows_per_wg = std::max<int64_t>(1, ceil_div(gr, want));
        p.cpb = ceil_div(gr, p.rows_per_wg);
        p.wgs = B * p.cpb;
    }
    const size_t one = round256(size_t(p.wgs) * size_t(C) * 4);
    p.off_post = 0;
    p.off_pre = one;
    p.off_gate = 2 * one;
    p.ws_bytes = (gates > 0 && p.cpb > 1 ? 3 : 2) * one;
    return p;
}

hipError_t launch_block_norm_back(const NormBackArgs &args, const NormBackPlan &p, float *dpost, float *dpre,
                                  float *dgate, int64_t gates, void *ws, bool vec, hipStream_t st) {
    NormBackArgs a = args;
    uint8_t *const w = static_cast<uint8_t *>(ws);
    const bool has_post = a.post != nullptr, has_gate = a.gate != nullptr;
    a.gate_rows = int(p.gate_rows);
    a.rows_per_wg = int(p.rows_per_wg);
    a.cpb = int(p.cpb);
    a.part_post = has_post ? reinterpret_cast<float *>(w + p.off_post) : nullptr;
    a.part_pre = a.pre ? reinterpret_cast<float *>(w + p.off_pre) : nullptr;
    a.part_gate = has_gate && p.cpb != 1 ? reinterpret_cast<float *>(w + p.off_gate) : nullptr;
    a.dgate = has_gate && p.cpb == 1 ? dgate : nullptr;

    // 512 threads leave 256 registers each; only rows past 16384 need 1024
    int T, NV;
    const int most = a.C > 512 * 32 ? 1024 : 512;
    if (vec) NV = loads_per_thread(a.C, 8, most, {1, 2, 4}, T);
    else NV = loads_per_thread(a.C, 1, most, {4, 8, 16, 32}, T);
    const int grid = int(p.wgs);
    hipError_t e = hipSuccess;
    if (grid == 0) {
        // no rows: the sums below are empty and write zeros
    } else if (vec) {
        if (NV == 1) e = launch_bwd<8, 1, 512>(a, T, grid, st);
        else if (NV == 2) e = launch_bwd<8, 2, 512>(a, T, grid, st);
        else if (most == 512) e = launch_bwd<8, 4, 512>(a, T, grid, st);
        else e = launch_bwd<8, 4, 1024>(a, T, grid, st);
    } else if (NV == 4) e = launch_bwd<1, 4, 512>(a, T, grid, st);
    else if (NV == 8) e = launch_bwd<1, 8, 512>(a, T, grid, st);
    else if (NV == 16) e = launch_bwd<1, 16, 512>(a, T, grid, st);
    else if (most == 512) e = launch_bwd<1, 32, 512>(a, T, grid, st);
    else e = launch_bwd<1, 32, 1024>(a, T, grid, st);
    if (e != hipSuccess) return e;

    ColumnSums c{};
    int n = 0, outs = 1;
    auto add = [&](float *out, const float *part, int64_t count, int64_t rows) {
        c.out[n] = out;
        c.part[n] = part;
        c.count[n] = int(count);
        c.outs[n] = int(rows);
        outs = std::max(outs, int(rows));
        ++n;
    };
    if (has_post) add(dpost, a.part_post, p.wgs, 1);
    if (a.pre) add(dpre, a.part_pre, p.wgs, 1);
    if (has_gate && p.cpb != 1) add(dgate, a.part_gate, p.cpb, gates);
    if (n == 0) return hipSuccess;
    c.C = a.C;
    hipLaunchKernelGGL(column_sum_kernel, dim3(unsigned(ceil_div(a.C, 64)), unsigned(std::min(outs, 65535)), unsigned(n)), dim3(1024), 0,
                       st, c);
    return hipGetLastError();
}

}  // namespace ql
