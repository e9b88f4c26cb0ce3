// C ABI of the 8-bit feed-forward operators: argument validation, sizes and launches.
// Every check runs before anything is queued, so an error leaves all outputs untouched.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/qlinear.h"
#include "ql_i8.hpp"
#include "ql_norm.hpp"

using namespace ql;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
ql_status from_hip(hipError_t e) { return e == hipSuccess ? QL_OK : QL_E_HIP; }

// channels past 2^20 would pass the 31-bit row offsets of the backward product
constexpr int64_t N_MAX = int64_t(1) << 20;

ql_status check_weight(int64_t N, int64_t K, int gated) {
    if (gated != 0 && gated != 1) return QL_E_ARG;
    if (N <= 0 || N > N_MAX || K <= 0 || K > I8_K_MAX || K % 32 != 0) return QL_E_SHAPE;
    return QL_OK;
}

ql_status check_rows(int64_t M) { return M < 0 || M >= (int64_t(1) << 31) ? QL_E_SHAPE : QL_OK; }

ql_status forward(const void *codes, const float *scales, int64_t M, int64_t N, int64_t K, const void *packed_w,
                  const void *packed_s, const void *bias, int gated, int act, void *out, ql_dtype out_dtype, void *raw,
                  void *workspace, size_t workspace_bytes, void *stream) {
    ql_status st = check_weight(N, K, gated);
    if (st == QL_OK) st = check_rows(M);
    if (st != QL_OK) return st;
    if (out_dtype != QL_BF16 && out_dtype != QL_F32) return QL_E_ARG;
    if (!packed_w || !packed_s) return QL_E_ARG;
    if (M == 0) return QL_OK;
    if (!codes || !scales || !out) return QL_E_ARG;
    if (!aligned(codes, 16) || !aligned(packed_w, 16) || !aligned(packed_s, 16)) return QL_E_ALIGN;
    const size_t es = out_dtype == QL_F32 ? 4 : 2;
    if (!aligned(scales, 4) || !aligned(bias, 2) || !aligned(out, es) || !aligned(raw, 2)) return QL_E_ALIGN;
    const I8Layout L = make_i8_layout(N, K, gated != 0);
    const I8Plan p = make_i8_plan(L, M);
    if (p.threads > LAUNCH_THREADS_MAX || int64_t(p.mtiles) * p.nblocks > INT32_MAX) return QL_E_SHAPE;
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    I8Args a{};
    a.x = static_cast<const int8_t *>(codes);
    a.xs = scales;
    a.w = static_cast<const uint8_t *>(packed_w);
    a.s = static_cast<const float *>(packed_s);
    a.bias = static_cast<const uint16_t *>(bias);
    a.out = out;
    a.raw = static_cast<uint16_t *>(raw);
    a.part = static_cast<int32_t *>(workspace);
    a.M = int(M);
    a.act = act;
    a.out_f32 = out_dtype == QL_F32 ? 1 : 0;
    a.pieces = N % 8 == 0 && aligned(out, 16) && aligned(raw, 16);
    return from_hip(launch_i8_forward(L, p, a, (hipStream_t)stream));
}

ql_status backward(const void *dy, const void *raw, int64_t M, int64_t N, int64_t K, const void *packed_w,
                   const void *packed_s, int gated, int act, void *dx, void *draw, void *workspace,
                   size_t workspace_bytes, void *stream) {
    ql_status st = check_weight(N, K, gated);
    if (st == QL_OK) st = check_rows(M);
    if (st != QL_OK) return st;
    if (!packed_w || !packed_s) return QL_E_ARG;
    if (M == 0) return QL_OK;
    if (!dy || !dx || (gated && (!raw || !draw))) return QL_E_ARG;
    if (!aligned(packed_w, 16) || !aligned(packed_s, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(raw, 16) ||
        !aligned(draw, 16))
        return QL_E_ALIGN;
    const I8Layout L = make_i8_layout(N, K, gated != 0);
    const I8BackPlan p = make_i8_back_plan(L, M);
    if (p.threads > LAUNCH_THREADS_MAX || int64_t(p.mtiles) * p.nblocks > INT32_MAX) return QL_E_SHAPE;
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    return from_hip(launch_i8_backward(L, p, static_cast<const uint16_t *>(dy), static_cast<const uint16_t *>(raw), act, M,
                                       packed_w, packed_s, static_cast<uint16_t *>(dx), static_cast<uint16_t *>(draw),
                                       workspace, (hipStream_t)stream));
}

bool known_act(ql_gate_act act) { return act == QL_GATE_SILU || act == QL_GATE_GELU; }

ql_status check_norm(int64_t R, int64_t C, int64_t gates, float residual_scale, float eps, ql_dtype r_dtype,
                     ql_dtype p_dtype) {
    if (R < 0 || R >= (int64_t(1) << 31) || C <= 0 || C > NORM_C_MAX) return QL_E_SHAPE;
    if (gates < 0 || gates >= (int64_t(1) << 31) || (gates > 1 && R % gates != 0)) return QL_E_SHAPE;
    if (!isfinite(residual_scale) || !isfinite(eps) || !(eps > 0.0f)) return QL_E_ARG;
    if ((r_dtype != QL_BF16 && r_dtype != QL_F32) || (p_dtype != QL_BF16 && p_dtype != QL_F32)) return QL_E_ARG;
    return QL_OK;
}

}  // namespace

extern "C" {

ql_status qlinear_i8_packed_bytes(int64_t N, int64_t K, int gated, size_t *w_bytes, size_t *s_bytes) {
    if (!w_bytes || !s_bytes) return QL_E_ARG;
    const ql_status st = check_weight(N, K, gated);
    if (st != QL_OK) return st;
    const I8Layout L = make_i8_layout(N, K, gated != 0);
    *w_bytes = L.w_bytes;
    *s_bytes = L.s_bytes;
    return QL_OK;
}

ql_status qlinear_i8_pack(int64_t N, int64_t K, const void *codes, const float *scales, const void *gate_codes,
                          const float *gate_scales, void *packed_w, void *packed_s, void *stream) {
    const int gated = gate_codes ? 1 : 0;
    const ql_status st = check_weight(N, K, gated);
    if (st != QL_OK) return st;
    if (!codes || !scales || !packed_w || !packed_s || (gated ? !gate_scales : gate_scales != nullptr)) return QL_E_ARG;
    if (!aligned(scales, 4) || !aligned(gate_scales, 4) || !aligned(packed_w, 16) || !aligned(packed_s, 16))
        return QL_E_ALIGN;
    return from_hip(launch_i8_pack(make_i8_layout(N, K, gated != 0), static_cast<const int8_t *>(codes), scales,
                                   static_cast<const int8_t *>(gate_codes), gate_scales, packed_w, packed_s,
                                   (hipStream_t)stream));
}

ql_status qlinear_i8_unpack(int64_t N, int64_t K, const void *packed_w, const void *packed_s, void *codes, float *scales,
                            void *gate_codes, float *gate_scales, void *stream) {
    const int gated = gate_codes ? 1 : 0;
    const ql_status st = check_weight(N, K, gated);
    if (st != QL_OK) return st;
    if (!codes || !scales || !packed_w || !packed_s || (gated ? !gate_scales : gate_scales != nullptr)) return QL_E_ARG;
    if (!aligned(scales, 4) || !aligned(gate_scales, 4) || !aligned(packed_w, 16) || !aligned(packed_s, 16))
        return QL_E_ALIGN;
    return from_hip(launch_i8_unpack(make_i8_layout(N, K, gated != 0), packed_w, packed_s, static_cast<int8_t *>(codes),
                                     scales, static_cast<int8_t *>(gate_codes), gate_scales, (hipStream_t)stream));
}

ql_status qlinear_i8_default_schedule(int64_t M, int64_t N, int64_t K, int gated, int backward, ql_schedule *out) {
    if (!out || (backward != 0 && backward != 1)) return QL_E_ARG;
    ql_status st = check_weight(N, K, gated);
    if (st == QL_OK) st = check_rows(M);
    if (st != QL_OK) return st;
    if (M == 0) return QL_E_SHAPE;
    const I8Layout L = make_i8_layout(N, K, gated != 0);
    if (backward) {
        const I8BackPlan p = make_i8_back_plan(L, M);
        *out = ql_schedule{p.cfg, p.ks};
    } else {
        const I8Plan p = make_i8_plan(L, M);
        *out = ql_schedule{p.cfg, p.ks};
    }
    return QL_OK;
}

ql_status qlinear_i8_workspace_bytes(int64_t M, int64_t N, int64_t K, int gated, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    ql_status st = check_weight(N, K, gated);
    if (st == QL_OK) st = check_rows(M);
    if (st != QL_OK) return st;
    *bytes = M ? make_i8_plan(make_i8_layout(N, K, gated != 0), M).ws_bytes : 0;
    return QL_OK;
}

ql_status qlinear_i8_forward(const void *codes, const float *scales, int64_t M, int64_t N, int64_t K,
                             const void *packed_w, const void *packed_s, const void *bias, void *out, ql_dtype out_dtype,
                             void *workspace, size_t workspace_bytes, void *stream) {
    return forward(codes, scales, M, N, K, packed_w, packed_s, bias, 0, 0, out, out_dtype, nullptr, workspace,
                   workspace_bytes, stream);
}

ql_status qlinear_i8_gated_forward(const void *codes, const float *scales, int64_t M, int64_t N, int64_t K,
                                   const void *packed_w, const void *packed_s, const void *bias, ql_gate_act act,
                                   void *out, ql_dtype out_dtype, void *raw, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (!known_act(act)) return QL_E_ARG;
    return forward(codes, scales, M, N, K, packed_w, packed_s, bias, 1, int(act), out, out_dtype, raw, workspace,
                   workspace_bytes, stream);
}

ql_status qlinear_i8_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int gated, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    ql_status st = check_weight(N, K, gated);
    if (st == QL_OK) st = check_rows(M);
    if (st != QL_OK) return st;
    *bytes = M ? make_i8_back_plan(make_i8_layout(N, K, gated != 0), M).ws_bytes : 0;
    return QL_OK;
}

ql_status qlinear_i8_backward(const void *dy, int64_t M, int64_t N, int64_t K, const void *packed_w,
                              const void *packed_s, void *dx, void *workspace, size_t workspace_bytes, void *stream) {
    return backward(dy, nullptr, M, N, K, packed_w, packed_s, 0, 0, dx, nullptr, workspace, workspace_bytes, stream);
}

ql_status qlinear_i8_gated_backward(const void *dh, const void *raw, int64_t M, int64_t N, int64_t K,
                                    const void *packed_w, const void *packed_s, ql_gate_act act, void *dx, void *draw,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    if (!known_act(act)) return QL_E_ARG;
    return backward(dh, raw, M, N, K, packed_w, packed_s, 1, int(act), dx, draw, workspace, workspace_bytes, stream);
}

ql_status qlinear_block_norm(const void *residual, ql_dtype residual_dtype, const void *y, const void *post_weight,
                             const void *pre_weight, const void *gate, ql_dtype param_dtype, int64_t gates,
                             float residual_scale, float eps, int64_t R, int64_t C, void *residual_out, void *x,
                             void *codes, float *scales, void *stream) {
    const ql_status st = check_norm(R, C, gates, residual_scale, eps, residual_dtype, param_dtype);
    if (st != QL_OK) return st;
    if ((gates > 0) != (gate != nullptr)) return QL_E_ARG;
    if (R > 0 && !y && (post_weight || gate)) return QL_E_ARG;
    if (R == 0) return QL_OK;
    if ((codes != nullptr) != (scales != nullptr)) return QL_E_ARG;
    if (pre_weight ? ((x != nullptr) == (codes != nullptr)) : (x || codes)) return QL_E_ARG;
    if (!residual || !residual_out) return QL_E_ARG;
    const size_t er = residual_dtype == QL_F32 ? 4 : 2, ep = param_dtype == QL_F32 ? 4 : 2;
    if (!aligned(residual, er) || !aligned(residual_out, er) || !aligned(y, 2) || !aligned(x, 2) || !aligned(scales, 4) ||
        !aligned(post_weight, ep) || !aligned(pre_weight, ep) || !aligned(gate, ep))
        return QL_E_ALIGN;
    NormArgs a{};
    a.y = y;
    a.r = residual;
    a.r_out = residual_out;
    a.post = post_weight;
    a.pre = pre_weight;
    a.gate = gate;
    a.x = static_cast<uint16_t *>(x);
    a.codes = static_cast<int8_t *>(codes);
    a.scales = scales;
    a.alpha = residual_scale;
    a.eps = eps;
    a.R = int(R);
    a.C = int(C);
    a.gate_rows = gates > 1 ? int(R / gates) : 0;
    a.p_bf16 = param_dtype == QL_BF16;
    a.r_f32 = residual_dtype == QL_F32;
    bool vec = C % 8 == 0 && aligned(codes, 8);
    for (const void *p : {residual, static_cast<const void *>(residual_out), y, static_cast<const void *>(x), post_weight,
                          pre_weight, gate})
        vec = vec && aligned(p, 16);
    return from_hip(launch_block_norm(a, vec, (hipStream_t)stream));
}

ql_status qlinear_block_norm_backward_workspace_bytes(int64_t R, int64_t C, int64_t gates, size_t *bytes) {
    if (!bytes) return QL_E_ARG;
    const ql_status st = check_norm(R, C, gates, 1.0f, 1.0f, QL_F32, QL_F32);
    if (st != QL_OK) return st;
    *bytes = make_norm_back_plan(R, C, gates).ws_bytes;
    return QL_OK;
}

ql_status qlinear_block_norm_backward(const void *dx, const void *dresidual, const void *residual_out,
                                      ql_dtype residual_dtype, const void *y, const void *post_weight,
                                      const void *pre_weight, const void *gate, ql_dtype param_dtype, int64_t gates,
                                      float residual_scale, float eps, int64_t R, int64_t C, void *dresidual_in,
                                      void *dy, float *dpost, float *dpre, float *dgate, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    const ql_status st = check_norm(R, C, gates, residual_scale, eps, residual_dtype, param_dtype);
    if (st != QL_OK) return st;
    if ((gates > 0) != (gate != nullptr)) return QL_E_ARG;
    if (R > 0 && !y && (post_weight || gate)) return QL_E_ARG;
    if ((post_weight != nullptr) != (dpost != nullptr) || (pre_weight != nullptr) != (dpre != nullptr) ||
        (gate != nullptr) != (dgate != nullptr))
        return QL_E_ARG;
    if (R > 0) {
        if (!dresidual_in || (y != nullptr) != (dy != nullptr)) return QL_E_ARG;
        if (pre_weight ? (!dx || !residual_out) : dx != nullptr) return QL_E_ARG;
    }
    const size_t er = residual_dtype == QL_F32 ? 4 : 2, ep = param_dtype == QL_F32 ? 4 : 2;
    if (!aligned(residual_out, er) || !aligned(dresidual, er) || !aligned(dresidual_in, er) || !aligned(y, 2) ||
        !aligned(dx, 2) || !aligned(dy, 2) || !aligned(post_weight, ep) || !aligned(pre_weight, ep) ||
        !aligned(gate, ep) || !aligned(dpost, 4) || !aligned(dpre, 4) || !aligned(dgate, 4))
        return QL_E_ALIGN;
    const NormBackPlan p = make_norm_back_plan(R, C, gates);
    if (p.ws_bytes) {
        if (!workspace || workspace_bytes < p.ws_bytes) return QL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return QL_E_ALIGN;
    }
    NormBackArgs a{};
    a.dx = dx;
    a.dres = dresidual;
    a.r = residual_out;
    a.y = y;
    a.post = post_weight;
    a.pre = pre_weight;
    a.gate = gate;
    a.dr = dresidual_in;
    a.dy = static_cast<uint16_t *>(dy);
    a.alpha = residual_scale;
    a.eps = eps;
    a.R = int(R);
    a.C = int(C);
    a.p_bf16 = param_dtype == QL_BF16;
    a.r_f32 = residual_dtype == QL_F32;
    bool vec = C % 8 == 0;
    for (const void *q : {dx, dresidual, residual_out, y, post_weight, pre_weight, gate, static_cast<const void *>(dy),
                          static_cast<const void *>(dresidual_in), static_cast<const void *>(dgate)})
        vec = vec && aligned(q, 16);
    return from_hip(launch_block_norm_back(a, p, dpost, dpre, dgate, gates, workspace, vec, (hipStream_t)stream));
}

}  // extern "C"
