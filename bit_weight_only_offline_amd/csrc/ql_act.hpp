// Gated activations and small store helpers shared by the per-channel INT8 kernels.
//
// Both activations have the form  act(g) = g * p,  p = logistic(z):  z = g for SiLU, and
// z = 2 sqrt(2/pi) (g + 0.044715 g^3) for the tanh form of GELU, since (1 + tanh(z / 2)) / 2
// is the logistic function of z.  So  act'(g) = p + g p (1 - p) z'.  The argument of z is
// held to |g| <= 1e4, far past where p is 0 or 1 in float32, so that no cube overflows; a
// comparison with NaN is false, so NaN stays NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ql_decode.hpp"

namespace ql {

enum : int { GATE_SILU = 0, GATE_GELU = 1 };

constexpr float GELU_A = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float GELU_B = 0.044715f;

// 1 / (1 + exp(-z)): the hardware's exponential of two and reciprocal, each within about 1 ulp.
// The exponent z log2(e) is rounded, which for negative z is |z| 2^-24 of the result; the roundings
// of z itself, from the float32 sum and scales, come to as much and more whatever the exponential.
__device__ inline float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ inline float gate_clamp(float g) { return g > 1e4f ? 1e4f : (g < -1e4f ? -1e4f : g); }

__device__ inline float gate_act(float g, int act) {
    const float c = gate_clamp(g);
    return g * logistic(act == GATE_SILU ? c : GELU_A * (c + GELU_B * c * c * c));
}

// act(g) and act'(g)
__device__ inline void gate_act_grad(float g, int act, float &a, float &da) {
    const float c = gate_clamp(g);
    const float z = act == GATE_SILU ? c : GELU_A * (c + GELU_B * c * c * c);
    const float dz = act == GATE_SILU ? 1.0f : GELU_A * (1.0f + 3.0f * GELU_B * c * c);
    const float p = logistic(z);
    a = g * p;
    da = p + c * p * logistic(-z) * dz;
}

// two float32 rounded to bf16 (to nearest even) in one conversion
__device__ inline uint32_t pack_bf16(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Vectors at any element's address: the compute units' memory access is set up to take loads
// and stores at every alignment, and the compiler, told that these are not aligned, emits
// single instructions for them.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Four consecutive values of one row at element index i, of which the first `count` exist.
__device__ inline void store4_bf16(uint16_t *p, int64_t i, const float (&v)[4], int count) {
    if (count >= 4) {
        *reinterpret_cast<u32x2_any *>(p + i) = u32x2_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (r < count) reinterpret_cast<__bf16 *>(p)[i + r] = (__bf16)v[r];
    }
}
__device__ inline void store4_f32(float *p, int64_t i, const float (&v)[4], int count) {
    if (count >= 4) {
        *reinterpret_cast<f32x4_any *>(p + i) = f32x4_any{v[0], v[1], v[2], v[3]};
    } else {
        if (count > 0) p[i] = v[0];
        if (count > 1) p[i + 1] = v[1];
        if (count > 2) p[i + 2] = v[2];
    }
}

}  // namespace ql
