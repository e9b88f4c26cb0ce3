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
// rounded copy.  One workgroup walks a run of rows, so the weight vectors stay in registers
// and the next row is on its way while this one is reduced.
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

template <int V>
struct Raw { uint32_t w[V == 8 ? 8 : 1]; };   // V values as stored: bf16 (half used) or float32

// V values at element i of a bf16 or float32 array; V = 8 needs 16-byte aligned addresses
template <int V>
__device__ inline Raw<V> load_raw(const void *p, int64_t i, bool f32) {
    Raw<V> r;
    if constexpr (V == 8) {
        if (f32) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(p) + i);
            const u32x4 b = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(p) + i + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { r.w[j] = a[j]; r.w[4 + j] = b[j]; }
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[j] = a[j];
        }
    } else {
        r.w[0] = f32 ? static_cast<const uint32_t *>(p)[i] : uint32_t(static_cast<const uint16_t *>(p)[i]);
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
__device__ inline void store_row(void *p, int64_t i, bool f32, const float *v) {
    if constexpr (V == 8) {
        if (f32) {
            float *q = static_cast<float *>(p) + i;
            *reinterpret_cast<f32x4 *>(q) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4 *>(q + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + i) =
                u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        }
    } else {
        if (f32) static_cast<float *>(p)[i] = v[0];
        else static_cast<__bf16 *>(p)[i] = (__bf16)v[0];
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
// V values per load, NV loads per thread and row; KEEP: weight vectors stay in registers.
template <int V, int NV, int TMAX, bool RF32>
__global__ void __launch_bounds__(TMAX) block_norm_kernel(NormArgs a) {
    constexpr bool KEEP = V * NV <= 16;
    constexpr int E = V * NV;
    __shared__ float red[2 * 16 * 4];
    const int t = threadIdx.x, T = blockDim.x, waves = T >> 6;
    int turn = 0;
    const int row0 = blockIdx.x * a.rows_per_wg, row1 = min(a.R, row0 + a.rows_per_wg);
    const float inv_c = 1.0f / float(a.C);
    const bool pf32 = !a.p_bf16;

    int at[NV];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        at[v] = (v * T + t) * V;
        in[v] = at[v] < a.C;
    }
    auto params = [&](const void *p, int64_t base, float one, float *out) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (p && in[v]) widen<V>(load_raw<V>(p, base + at[v], pf32), pf32, out + v * V);
            else
#pragma unroll
                for (int j = 0; j < V; ++j) out[v * V + j] = one;
        }
    };
    float post[KEEP ? E : 1], pre[KEEP ? E : 1], gate[KEEP ? E : 1];
    if constexpr (KEEP) {
        params(a.post, 0, 1.0f, post);
        params(a.pre, 0, 1.0f, pre);
    }
    int64_t gate_of = -1;

    Raw<V> ny[NV], nr[NV];
    auto fetch = [&](int row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ny[v] = Raw<V>{};
            nr[v] = Raw<V>{};
            if (in[v]) {
                if (a.y) ny[v] = load_raw<V>(a.y, int64_t(row) * a.C + at[v], false);
                nr[v] = load_raw<V>(a.r, int64_t(row) * a.C + at[v], RF32);
            }
        }
    };
    if (row0 < row1) fetch(row0);
    for (int row = row0; row < row1; ++row) {
        float y[E], r[E];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            widen<V>(ny[v], false, y + v * V);
            widen<V>(nr[v], RF32, r + v * V);
        }
        if (row + 1 < row1) fetch(row + 1);

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
            float gl[KEEP ? 1 : E], pl[KEEP ? 1 : E];
            if constexpr (KEEP) {
                if (gb != gate_of) params(a.gate, gb * a.C, 1.0f, gate);
                gate_of = gb;
            } else {
                params(a.gate, gb * a.C, 1.0f, gl);
                params(a.post, 0, 1.0f, pl);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float w = KEEP ? post[KEEP ? e : 0] : pl[KEEP ? 0 : e];
                const float gv = KEEP ? gate[KEEP ? e : 0] : gl[KEEP ? 0 : e];
                r[e] = fmaf(gv, y[e] * ip * w, a.alpha * r[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] *= a.alpha;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (in[v]) store_row<V>(a.r_out, int64_t(row) * a.C + at[v], RF32, r + v * V);
        if (!a.pre) continue;

        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < V; ++j) ss[0] = in[v] ? fmaf(r[v * V + j], r[v * V + j], ss[0]) : ss[0];
        reduce<1, false>(ss, red, turn, waves);
        const float iq = rsqrtf(fmaf(ss[0], inv_c, a.eps));
        float ql[KEEP ? 1 : E];
        if constexpr (!KEEP) params(a.pre, 0, 1.0f, ql);
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = r[e] * iq * (KEEP ? pre[KEEP ? e : 0] : ql[KEEP ? 0 : e]);
        if (a.x) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (in[v]) store_row<V>(a.x, int64_t(row) * a.C + at[v], false, r + v * V);
            continue;
        }
        float am[1] = {0.0f};
        bool bad = false;                               // a maximum would drop NaN
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in[v]) {
                    am[0] = fmaxf(am[0], fabsf(r[v * V + j]));
                    bad |= r[v * V + j] != r[v * V + j];
                }
        if (bad) am[0] = INFINITY;
        reduce<1, true>(am, red, turn, waves);
        // a row with NaN or infinity has the scale NaN and codes 0, so its products are NaN
        const float s = am[0] < INFINITY ? __fdiv_rn(am[0], 127.0f) : __uint_as_float(0x7FC00000u);
        if (t == 0) a.scales[row] = s;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!in[v]) continue;
            uint32_t q[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(r[v * V + j], s)), -127.0f), 127.0f) : 0.0f;
                q[j >> 2] |= (uint32_t(int(f)) & 0xFFu) << (8 * (j & 3));
            }
            int8_t *dst = a.codes + int64_t(row) * a.C + at[v];
            if constexpr (V == 8) *reinterpret_cast<u32x2 *>(dst) = u32x2{q[0], q[1]};
            else dst[0] = int8_t(q[0]);
        }
    }
}

// ---- backward --------------------------------------------------------------------------
// Workgroup i walks rows of one gate (chunk i mod cpb of gate i / cpb), or, where there are
// more gates than workgroups (cpb = 1), all rows of gpw gates.  The column sums stay in
// registers and leave once a workgroup (dgate: once a gate where cpb = 1).
template <int V, int NV, int TMAX, bool RF32>
__global__ void __launch_bounds__(TMAX) block_norm_back_kernel(NormBackArgs a) {
    constexpr bool KEEP = V * NV <= 8;
    constexpr int E = V * NV;
    __shared__ float red[2 * 16 * 4];
    const int t = threadIdx.x, T = blockDim.x, waves = T >> 6;
    int turn = 0;
    const float inv_c = 1.0f / float(a.C);
    const bool pf32 = !a.p_bf16;
    const int i = blockIdx.x;
    int64_t row0, row1;
    if (a.cpb > 1) {
        row0 = int64_t(i / a.cpb) * a.gate_rows + int64_t(i % a.cpb) * a.rows_per_wg;
        row1 = min(row0 + a.rows_per_wg, int64_t(i / a.cpb + 1) * a.gate_rows);
    } else {
        row0 = int64_t(i) * a.rows_per_wg;
        row1 = min(int64_t(a.R), row0 + a.rows_per_wg);
    }

    int at[NV];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        at[v] = (v * T + t) * V;
        in[v] = at[v] < a.C;
    }
    auto params = [&](const void *p, int64_t base, float *out) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (p && in[v]) widen<V>(load_raw<V>(p, base + at[v], pf32), pf32, out + v * V);
            else
#pragma unroll
                for (int j = 0; j < V; ++j) out[v * V + j] = 1.0f;
        }
    };
    auto sums_out = [&](float *dst, const float *v0) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (in[v]) store_row<V>(dst, at[v], true, v0 + v * V);
    };
    float post[KEEP ? E : 1], pre[KEEP ? E : 1], gate[KEEP ? E : 1];
    if constexpr (KEEP) {
        params(a.post, 0, post);
        params(a.pre, 0, pre);
    }
    int64_t gate_of = -1;
    float s_post[E], s_pre[E], s_gate[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s_post[e] = s_pre[e] = s_gate[e] = 0.0f;

    Raw<V> ny[NV], nr[NV], nx[NV], nd[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ny[v] = nr[v] = nx[v] = nd[v] = Raw<V>{};
            if (in[v]) {
                const int64_t j = row * a.C + at[v];
                if (a.y) ny[v] = load_raw<V>(a.y, j, false);
                if (a.pre) {
                    nr[v] = load_raw<V>(a.r, j, RF32);
                    nx[v] = load_raw<V>(a.dx, j, false);
                }
                if (a.dres) nd[v] = load_raw<V>(a.dres, j, RF32);
            }
        }
    };
    if (row0 < row1) fetch(row0);
    for (int64_t row = row0; row < row1; ++row) {
        float y[E], r[E], x[E], d[E];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            widen<V>(ny[v], false, y + v * V);
            widen<V>(nr[v], RF32, r + v * V);
            widen<V>(nx[v], false, x + v * V);
            widen<V>(nd[v], RF32, d + v * V);
        }
        if (row + 1 < row1) fetch(row + 1);

        float ql[KEEP ? 1 : E];
        if constexpr (!KEEP) params(a.pre, 0, ql);
        auto pre_of = [&](int e) { return KEEP ? pre[KEEP ? e : 0] : ql[KEEP ? 0 : e]; };
        float ss[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ss[0] = fmaf(y[e], y[e], ss[0]);
            ss[1] = fmaf(r[e], r[e], ss[1]);
            ss[2] = fmaf(x[e] * pre_of(e), r[e], ss[2]);
        }
        reduce<3, false>(ss, red, turn, waves);
        const float ip = a.post ? rsqrtf(fmaf(ss[0], inv_c, a.eps)) : 1.0f;
        if (a.pre) {
            const float iq = rsqrtf(fmaf(ss[1], inv_c, a.eps));
            const float along = ss[2] * iq * inv_c;          // mean(n u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float u = r[e] * iq;
                d[e] = fmaf(iq, x[e] * pre_of(e) - u * along, d[e]);
                s_pre[e] = fmaf(x[e], u, s_pre[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = a.alpha * d[e];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (in[v]) store_row<V>(a.dr, row * a.C + at[v], RF32, r + v * V);
        if (!a.y) continue;

        const int64_t gb = a.gate_rows ? row / a.gate_rows : 0;
        float gl[KEEP ? 1 : E], pl[KEEP ? 1 : E];
        if constexpr (KEEP) {
            if (gb != gate_of) params(a.gate, gb * a.C, gate);
            gate_of = gb;
        } else {
            params(a.gate, gb * a.C, gl);
            params(a.post, 0, pl);
        }
        float dot[1] = {0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float w = KEEP ? post[KEEP ? e : 0] : pl[KEEP ? 0 : e];
            const float gv = KEEP ? gate[KEEP ? e : 0] : gl[KEEP ? 0 : e];
            const float v = y[e] * ip;
            s_gate[e] = fmaf(d[e] * w, v, s_gate[e]);
            const float dt = d[e] * gv;
            s_post[e] = fmaf(dt, v, s_post[e]);
            d[e] = dt * w;
            dot[0] = fmaf(d[e], v, dot[0]);
        }
        if (a.post) {
            reduce<1, false>(dot, red, turn, waves);
            const float along = dot[0] * inv_c;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = ip * (d[e] - y[e] * ip * along);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (in[v]) store_row<V>(a.dy, row * a.C + at[v], false, d + v * V);
        if (a.dgate && a.cpb == 1 && (row + 1) % a.gate_rows == 0) {   // this gate is complete
            sums_out(a.dgate + gb * a.C, s_gate);
#pragma unroll
            for (int e = 0; e < E; ++e) s_gate[e] = 0.0f;
        }
    }
    const int64_t slot = int64_t(i) * a.C;
    if (a.part_post) sums_out(a.part_post + slot, s_post);
    if (a.part_pre) sums_out(a.part_pre + slot, s_pre);
    if (a.part_gate) sums_out(a.part_gate + slot, s_gate);
}

// out[b][c] = sum over `count` consecutive rows of part, in a fixed order: 16 row groups of
// one workgroup take every 16th row, then the groups are added in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(ColumnSums a) {
    __shared__ float red[16][64];
    const int q = blockIdx.z, lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    if (blockIdx.y >= unsigned(a.outs[q])) return;
    const int64_t c = int64_t(blockIdx.x) * 64 + lane;
    const float *p = a.part[q] + int64_t(blockIdx.y) * a.count[q] * a.C;
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
        a.out[q][int64_t(blockIdx.y) * a.C + c] = t;
    }
}

int threads_for(int64_t C, int V, int NV, int most) {
    const int64_t t = ceil_div(ceil_div(C, int64_t(V) * NV), 64) * 64;
    return int(std::min<int64_t>(t, most));
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
    const int V = vec ? 8 : 1;
    // loads per thread: as few as 512 threads allow, so that a row's latency is short
    int NV = 1;
    const int64_t pieces = ceil_div(a.C, V);
    const int most = pieces > 512 * 4 * (vec ? 1 : 8) ? 1024 : 512;
    if (vec) while (int64_t(most) * NV < pieces) NV *= 2;
    else NV = int64_t(most) * 8 >= pieces ? 8 : 32;
    const int T = threads_for(a.C, V, NV, most);
    const int64_t wgs = std::min<int64_t>(a.R, 256 * (2048 / std::max(T, 256)));
    a.rows_per_wg = int(ceil_div(a.R, wgs));
    const int grid = int(ceil_div(a.R, a.rows_per_wg));
    if (vec) {
        if (NV == 1) return launch_fwd<8, 1, 512>(a, T, grid, st);
        if (NV == 2) return launch_fwd<8, 2, 512>(a, T, grid, st);
        return launch_fwd<8, 4, 1024>(a, T, grid, st);
    }
    if (NV == 8) return launch_fwd<1, 8, 512>(a, T, grid, st);
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

    const int V = vec ? 8 : 1;
    const int64_t pieces = ceil_div(a.C, V);
    const int most = pieces > 512 * 4 * (vec ? 1 : 8) ? 1024 : 512;
    int NV = 1;
    if (vec) while (int64_t(most) * NV < pieces) NV *= 2;
    else NV = int64_t(most) * 8 >= pieces ? 8 : 32;
    const int T = threads_for(a.C, V, NV, most), grid = int(p.wgs);
    hipError_t e = hipSuccess;
    if (grid == 0) {
        // no rows: the sums below are empty and write zeros
    } else if (vec) {
        if (NV == 1) e = launch_bwd<8, 1, 512>(a, T, grid, st);
        else if (NV == 2) e = launch_bwd<8, 2, 512>(a, T, grid, st);
        else e = launch_bwd<8, 4, 1024>(a, T, grid, st);
    } else if (NV == 8) e = launch_bwd<1, 8, 512>(a, T, grid, st);
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
    hipLaunchKernelGGL(column_sum_kernel, dim3(unsigned(ceil_div(a.C, 64)), unsigned(outs), unsigned(n)), dim3(1024), 0,
                       st, c);
    return hipGetLastError();
}

}  // namespace ql
