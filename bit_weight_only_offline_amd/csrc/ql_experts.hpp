// Launch arguments of the operators that bring tokens into expert order and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ql_common.hpp"

namespace ql {

constexpr int64_t EXPERTS_MAX = 1024;    // the order's counters of sixteen wavefronts lie in LDS
constexpr int64_t CHOICES_MAX = 256;

// Workgroups of the order, each with a run of `per` slots (a multiple of 1024).
struct OrderPlan {
    int64_t wgs = 1, per = 0;
    size_t ws_bytes = 0;                 // the workgroups' counts [wgs][E] where there are several
};
OrderPlan make_order_plan(int64_t n, int64_t E);

struct OrderArgs {
    const void *ids;         // [n] int32 or int64
    int32_t *counts;         // [E]
    int32_t *rows;           // [n]
    int32_t *source;         // [n]
    int32_t *part;           // [wgs][E]
    int64_t n, per;
    int E, wide;             // wide: int64 ids
};
hipError_t launch_expert_order(const OrderArgs &a, const OrderPlan &p, hipStream_t st);

struct DispatchArgs {
    const void *x;           // [T, D]
    const int32_t *rows;     // [T, k]
    void *out;               // [T k, D], or null and
    uint8_t *codes;          // [T k, D] with
    float *scales;           // [T k, ceil(D / 128)]
    int64_t T;
    int k, D;
    int f32;
};
hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t st);

struct CombineArgs {
    const void *y;           // [T k, D]
    const int32_t *rows;     // [T, k]
    const float *w;          // [T, k], or null: ones
    void *out;               // [T, D]
    const void *dout;        // backward: [T, D] and
    void *dy;                // [T k, D]
    float *dw;               // [T, k]
    int64_t T;
    int k, D;
    int f32;
};
hipError_t launch_combine(const CombineArgs &a, hipStream_t st);
hipError_t launch_combine_backward(const CombineArgs &a, hipStream_t st);

}  // namespace ql
