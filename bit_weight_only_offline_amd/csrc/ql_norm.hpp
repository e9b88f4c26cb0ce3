// Launch arguments of the fused block norm and of its backward pass.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ql_common.hpp"

namespace ql {

constexpr int64_t NORM_C_MAX = 32768;   // a row stays in the registers of one workgroup

struct NormArgs {
    const void *y;          // bf16 [R, C] or null
    const void *r;          // residual [R, C], bf16 or float32 (r_f32)
    void *r_out;            // same type
    const void *post, *pre, *gate;   // float32, or bf16 (p_bf16); null: absent
    uint16_t *x;            // bf16 [R, C], or null and
    int8_t *codes;          // int8 [R, C] with
    float *scales;          // float32 [R]
    float alpha, eps;
    int R, C;
    int gate_rows;          // rows of one gate vector, 0: one vector for all rows
    int p_bf16, r_f32;
};

struct NormBackArgs {
    const void *dx;         // bf16 [R, C] (with pre)
    const void *dres;       // gradient of r' or null (zero)
    const void *r;          // r' as the forward pass returned it
    const void *y;
    const void *post, *pre, *gate;
    void *dr;               // gradient of r
    uint16_t *dy;
    float *dgate;           // written directly where a workgroup owns whole gates
    float *part_post, *part_pre, *part_gate;
    float alpha, eps;
    int R, C;
    int gate_rows, cpb;     // rows of one gate, workgroups per gate
    int p_bf16, r_f32;
    int rows_per_wg;
};

struct NormBackPlan {
    int64_t gate_rows = 0, rows_per_wg = 0, cpb = 1, wgs = 0;
    size_t off_post = 0, off_pre = 0, off_gate = 0, ws_bytes = 0;
};

struct ColumnSums {
    float *out[3];
    const float *part[3];
    int count[3], outs[3];
    int C;
};

hipError_t launch_block_norm(const NormArgs &a, bool vec, hipStream_t st);
NormBackPlan make_norm_back_plan(int64_t R, int64_t C, int64_t gates);
hipError_t launch_block_norm_back(const NormBackArgs &a, const NormBackPlan &p, float *dpost, float *dpre, float *dgate,
                                  int64_t gates, void *ws, bool vec, hipStream_t st);

}  // namespace ql
