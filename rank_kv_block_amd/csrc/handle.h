// The predictor handle and the helpers every C entry point shares: its error
// message, size products and alignment checks (defined in pred_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pred.h"

struct pred_handle {
    pred_dims d;
    int device;
    int n_cu;          // compute units of that device
    uint16_t* p_dev;   // [D, R] bf16
    double* pf_dev;    // [D, R] float64 copy read by the projection kernels
    uint16_t* ag_dev;  // [L, N, Hk, B, R] bf16
    uint32_t* err_dev; // device error word
};

namespace pred {

// Set the thread's message and return `code`; clear it and return PRED_OK; a
// failing HIP call's code and message.
int fail(int code, const char* fmt, ...);
int ok();
int hip_fail(hipError_t e, const char* what);

// a * b into *out; false if either is negative or the product overflows.
bool mul_ok(int64_t a, int64_t b, int64_t* out);

inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

}  // namespace pred
