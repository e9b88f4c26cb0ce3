// C ABI of the block-scaled e4m3 operators and of the ones that bring tokens into expert order and back:
// argument validation, sizes and launches.  Every check runs before anything is queued, so an error leaves
// all outputs untouched.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qlinear.h"
#include "ql_experts.hpp"
#include "ql_f8.hpp"

using namespace ql;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
ql_status from_hip(hipError_t e) { return e == hipSuccess ? QL_OK : QL_E_HIP; }
bool known(ql_dtype d) { return d == QL_BF16 || d == QL_F32; }
size_t width(ql_dtype d) { return d == QL_F32 ? 4 : 2; }

constexpr int64_t N_MAX = int64_t(1) << 20;     // rows of channels keep 32-bit offsets
constexpr int64_t E_MAX = int64_t(1) << 16;
constexpr int64_t ROWS_MAX = (int64_t(1) << 31) - 1;
constexpr int64_t D_MAX = int64_t(1) << 24;

bool inputs_ok(int64_t K) { return K > 0 && K <= I8_K_MAX && K % 32 == 0; }
ql_status check_weight(int64_t E, int64_t N, int64_t K) {
    return E > 0 && E <= E_MAX && N > 0 && N <= N_MAX && inputs_ok(K) ? QL_OK : QL_E_SHAPE;
}
ql_status check_product(int64_t M, int64_t E, int64_t N, int64_t K, int grouped) {
    if (grouped != 0 && grouped != 1) return QL_E_ARG;
    const ql_status st = check_weight(E, N, K);
    if (st != QL_OK) return st;
    return M < 0 || M > ROWS_MAX || (!grouped && E != 1) ? QL_E_SHAPE : QL_OK;
}
template <typename Plan>
bool fits(const Plan &p) {
    return p.threads <= LAUNCH_THREADS_MAX && p.mtiles * p.nblocks <= INT32_MAX - 8;
}

ql_status check_slots(int64_t T, int64_t k, int64_t D) {
    if (T < 0 || k <= 0 || k > CHOICES_MAX || D <= 0 || D > D_MAX || T > ROWS_MAX / k) return QL_E_SHAPE;
    return QL_OK;
}

}  // namespace

extern "C" {

ql_status qlinear_f8_quantize(const void *x, ql_dtype x_dtype, ql_act act, int64_t R, int64_t K, void *codes, float *scales,
                              void *stream) {
    if (!known(x_dtype) || (act != QL_ACT_NONE && act != QL_ACT_SWIGLU)) return QL_E_ARG;
    if (R < 0 || R > ROWS_MAX || !inputs_ok(K)) return QL_E_SHAPE;
    if (R == 0) return QL_OK;
    if (!x || !codes || !scales) return QL_E_ARG;
    if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(scales, 4)) return QL_E_ALIGN;
    F8Quant a{};
    a.x = x;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    a.R = R;
    a.K = int(K);
    a.f32 = x_dtype == QL_F32;
    a.swiglu = act == QL_ACT_SWIGLU;
    return from_hip(launch_f8_quantize(a, (hipStream_t)stream));
}

ql_status qlinear_f8_quantize_backward(const void *dh, const void *raw, int64_t R, int64_t K, void *draw, void *stream) {
    if (R < 0 || R > ROWS_MAX || !inputs_ok(K)) return QL_E_SHAPE;
    if (R == 0) return QL_OK;
    if (!dh || !raw || !draw) return QL_E_ARG;
    if (!aligned(dh, 16) || !aligned(raw, 16) || !aligned(draw, 16)) return QL_E_ALIGN;
    return from_hip(launch_f8_quantize_backward(static_cast<const uint16_t *>(dh), static_cast<const uint16_t *>(raw),
                                                static_cast<uint16_t *>(draw), R, int(K), (hipStream_t)stream));
}

ql_status qlinear_f8_dequantize(const void *codes, const float *scales, int64_t R, int64_t K, void *out, ql_dtype out_dtype,
                                void *stream) {
    if (!known(out_dtype)) return QL_E_ARG;
    if (R < 0 || R > ROWS_MAX || !inputs_ok(K)) return QL_E_SHAPE;
    if (R == 0) return QL_OK;
    if (!codes || !scales || !out) return QL_E_ARG;
    if (!aligned(codes, 8) || !aligned(scales, 4) || !aligned(out, width(out_dtype))) return QL_E_ALIGN;
    return from_hip(launch_f8_dequantize(static_cast<const uint8_t *>(codes), scales, out, R, int(K), out_dtype == QL_F32,
                                         (hipStream_t)stream));
}

ql_status qlinear_f8_quantize_weight(const void *w, ql_dtype w_dtype, int64_t E, int64_t N, int64_t K, void *codes,
                                     float *scales, void *stream) {
    if (!known(w_dtype)) return QL_E_ARG;
    const ql_status st = check_weight(E, N, K);
    if (st != QL_OK) return st;
    if (!w || !codes || !scales) return QL_E_ARG;
    if (!aligned(w, 16) || !aligned(codes, 8) || !aligned(scales, 4)) return QL_E_ALIGN;
    return from_hip(launch_f8_quantize_weight(make_f8_layout(E, N, K), w, w_dtype == QL_F32, static_cast<uint8_t *>(codes),
                                              scales, (hipStream_t)stream));
}

ql_status qlinear_f8_packed_bytes(int64_t E, int64_t N, int64_t K, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    const ql_status st = check_weight(E, N, K);
    if (st != QL_OK) return st;
    *bytes = size_t(E) * make_f8_layout(E, N, K).w_bytes;
    return QL_OK;
}

ql_status qlinear_f8_pack(int64_t E, int64_t N, int64_t K, const void *codes, void *packed, void *stream) {
    const ql_status st = check_weight(E, N, K);
    if (st != QL_OK) return st;
    if (!codes || !packed) return QL_E_ARG;
    if (!aligned(codes, 16) || !aligned(packed, 16)) return QL_E_ALIGN;
    return from_hip(launch_f8_pack(make_f8_layout(E, N, K), static_cast<const uint8_t *>(codes), static_cast<uint8_t *>(packed),
                                   (hipStream_t)stream));
}

ql_status qlinear_f8_unpack(int64_t E, int64_t N, int64_t K, const void *packed, void *codes, void *stream) {
    const ql_status st = check_weight(E, N, K);
    if (st != QL_OK) return st;
    if (!codes || !packed) return QL_E_ARG;
    if (!aligned(codes, 16) || !aligned(packed, 16)) return QL_E_ALIGN;
    return from_hip(launch_f8_unpack(make_f8_layout(E, N, K), static_cast<const uint8_t *>(packed), static_cast<uint8_t *>(codes),
                                     (hipStream_t)stream));
}

ql_status qlinear_f8_default_schedule(int64_t M, int64_t E, int64_t N, int64_t K, int grouped, int backward,
                                      ql_dtype out_dtype, ql_schedule *out) {
    if (!out || !known(out_dtype) || (backward != 0 && backward != 1)) return QL_E_ARG;
    const ql_status st = check_product(M, E, N, K, grouped);
    if (st != QL_OK) return st;
    if (M == 0) return QL_E_SHAPE;
    const F8Layout L = make_f8_layout(E, N, K);
    if (backward) {
        const F8BackPlan p = make_f8_back_plan(L, M, grouped != 0);
        *out = ql_schedule{p.cfg, p.ks};
    } else {
        const F8Plan p = make_f8_plan(L, M, grouped != 0, out_dtype == QL_F32);
        *out = ql_schedule{p.cfg, p.ks};
    }
    return QL_OK;
}

ql_status qlinear_f8_workspace_bytes(int64_t M, int64_t E, int64_t N, int64_t K, int grouped, ql_dtype out_dtype,
                                     size_t *bytes) {
    if (!bytes || !known(out_dtype)) return QL_E_ARG;
    const ql_status st = check_product(M, E, N, K, grouped);
    if (st != QL_OK) return st;
    *bytes = M ? make_f8_plan(make_f8_layout(E, N, K), M, grouped != 0, out_dtype == QL_F32).ws_bytes : 0;
    return QL_OK;
}

ql_status qlinear_f8_forward(const void *codes, const float *scales, int64_t M, const int32_t *tokens_per_expert, int64_t E,
                             int64_t N, int64_t K, const void *packed, const float *w_scales, const void *bias, void *out,
                             ql_dtype out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const int grouped = tokens_per_expert ? 1 : 0;
    const ql_status st = check_product(M, E, N, K, grouped);
    if (st != QL_OK) return st;
    if (!known(out_dtype) || !packed || !w_scales) return QL_E_ARG;
    if (M == 0) return QL_OK;
    if (!codes || !scales || !out) return QL_E_ARG;
    if (!aligned(codes, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(w_scales, 4) ||
        !aligned(tokens_per_expert, 4) || !aligned(bias, 2) || !aligned(out, width(out_dtype)))
        return QL_E_ALIGN;
    const F8Layout L = make_f8_layout(E, N, K);
    const F8Plan p = make_f8_plan(L, M, grouped != 0, out_dtype == QL_F32);
    if (!fits(p)) return QL_E_SHAPE;
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    F8Args a{};
    a.r = F8Rows{tokens_per_expert, int(E), int(M)};
    a.x = static_cast<const uint8_t *>(codes);
    a.xs = scales;
    a.w = static_cast<const uint8_t *>(packed);
    a.ws = w_scales;
    a.bias = static_cast<const uint16_t *>(bias);
    a.out = out;
    a.part = static_cast<float *>(workspace);
    a.out_f32 = out_dtype == QL_F32 ? 1 : 0;
    return from_hip(launch_f8_forward(L, p, a, (hipStream_t)stream));
}

ql_status qlinear_f8_backward_workspace_bytes(int64_t M, int64_t E, int64_t N, int64_t K, int grouped, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    const ql_status st = check_product(M, E, N, K, grouped);
    if (st != QL_OK) return st;
    *bytes = M ? make_f8_back_plan(make_f8_layout(E, N, K), M, grouped != 0).ws_bytes : 0;
    return QL_OK;
}

ql_status qlinear_f8_backward(const void *dy, int64_t M, const int32_t *tokens_per_expert, int64_t E, int64_t N, int64_t K,
                              const void *packed, const float *w_scales, void *dx, void *workspace, size_t workspace_bytes,
                              void *stream) {
    const int grouped = tokens_per_expert ? 1 : 0;
    const ql_status st = check_product(M, E, N, K, grouped);
    if (st != QL_OK) return st;
    if (!packed || !w_scales) return QL_E_ARG;
    if (M == 0) return QL_OK;
    if (!dy || !dx) return QL_E_ARG;
    if (!aligned(dy, 16) || !aligned(dx, 16) || !aligned(packed, 16) || !aligned(w_scales, 4) || !aligned(tokens_per_expert, 4))
        return QL_E_ALIGN;
    const F8Layout L = make_f8_layout(E, N, K);
    const F8BackPlan p = make_f8_back_plan(L, M, grouped != 0);
    if (!fits(p)) return QL_E_SHAPE;
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    F8BackArgs a{};
    a.r = F8Rows{tokens_per_expert, int(E), int(M)};
    a.dy = static_cast<const uint16_t *>(dy);
    a.w = static_cast<const uint8_t *>(packed);
    a.ws = w_scales;
    a.dx = static_cast<uint16_t *>(dx);
    return from_hip(launch_f8_backward(L, p, a, workspace, (hipStream_t)stream));
}

ql_status qlinear_expert_order_workspace_bytes(int64_t n, int64_t E, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    if (n < 0 || n > ROWS_MAX || E <= 0 || E > EXPERTS_MAX) return QL_E_SHAPE;
    *bytes = make_order_plan(n, E).ws_bytes;
    return QL_OK;
}

ql_status qlinear_expert_order(const void *ids, int id_bytes, int64_t n, int64_t E, int32_t *counts, int32_t *rows,
                               int32_t *source, void *workspace, size_t workspace_bytes, void *stream) {
    if (n < 0 || n > ROWS_MAX || E <= 0 || E > EXPERTS_MAX) return QL_E_SHAPE;
    if (id_bytes != 4 && id_bytes != 8) return QL_E_ARG;
    if (!counts || (n > 0 && (!ids || !rows || !source))) return QL_E_ARG;
    if (!aligned(ids, size_t(id_bytes)) || !aligned(counts, 4) || !aligned(rows, 4) || !aligned(source, 4)) return QL_E_ALIGN;
    const OrderPlan p = make_order_plan(n, E);
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    OrderArgs a{};
    a.ids = ids;
    a.counts = counts;
    a.rows = rows;
    a.source = source;
    a.part = static_cast<int32_t *>(workspace);
    a.n = n;
    a.E = int(E);
    a.wide = id_bytes == 8;
    return from_hip(launch_expert_order(a, p, (hipStream_t)stream));
}

ql_status qlinear_dispatch(const void *x, ql_dtype dtype, const int32_t *rows, int64_t T, int64_t k, int64_t D, void *out,
                           void *codes, float *scales, void *stream) {
    if (!known(dtype)) return QL_E_ARG;
    const ql_status st = check_slots(T, k, D);
    if (st != QL_OK) return st;
    if ((codes != nullptr) != (scales != nullptr)) return QL_E_ARG;
    if (codes && !inputs_ok(D)) return QL_E_SHAPE;
    if (T == 0) return QL_OK;
    if (!x || !rows || (out != nullptr) == (codes != nullptr)) return QL_E_ARG;
    if (!aligned(x, width(dtype)) || !aligned(out, width(dtype)) || !aligned(rows, 4) || !aligned(codes, 8) || !aligned(scales, 4))
        return QL_E_ALIGN;
    DispatchArgs a{};
    a.x = x;
    a.rows = rows;
    a.out = out;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    a.T = T;
    a.k = int(k);
    a.D = int(D);
    a.f32 = dtype == QL_F32;
    return from_hip(launch_dispatch(a, (hipStream_t)stream));
}

ql_status qlinear_combine(const void *y, ql_dtype dtype, const int32_t *rows, const float *weights, int64_t T, int64_t k,
                          int64_t D, void *out, void *stream) {
    if (!known(dtype)) return QL_E_ARG;
    const ql_status st = check_slots(T, k, D);
    if (st != QL_OK) return st;
    if (T == 0) return QL_OK;
    if (!y || !rows || !out) return QL_E_ARG;
    if (!aligned(y, width(dtype)) || !aligned(out, width(dtype)) || !aligned(rows, 4) || !aligned(weights, 4)) return QL_E_ALIGN;
    CombineArgs a{};
    a.y = y;
    a.rows = rows;
    a.w = weights;
    a.out = out;
    a.T = T;
    a.k = int(k);
    a.D = int(D);
    a.f32 = dtype == QL_F32;
    return from_hip(launch_combine(a, (hipStream_t)stream));
}

ql_status qlinear_combine_backward(const void *dout, const void *y, ql_dtype dtype, const int32_t *rows, const float *weights,
                                   int64_t T, int64_t k, int64_t D, void *dy, float *dweights, void *stream) {
    if (!known(dtype)) return QL_E_ARG;
    const ql_status st = check_slots(T, k, D);
    if (st != QL_OK) return st;
    if (T == 0) return QL_OK;
    if (!dout || !y || !rows || !weights || !dy || !dweights) return QL_E_ARG;
    if (!aligned(dout, width(dtype)) || !aligned(y, width(dtype)) || !aligned(dy, width(dtype)) || !aligned(rows, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return QL_E_ALIGN;
    CombineArgs a{};
    a.y = y;
    a.rows = rows;
    a.w = weights;
    a.dout = dout;
    a.dy = dy;
    a.dw = dweights;
    a.T = T;
    a.k = int(k);
    a.D = int(D);
    a.f32 = dtype == QL_F32;
    return from_hip(launch_combine_backward(a, (hipStream_t)stream));
}

}  // extern "C"
