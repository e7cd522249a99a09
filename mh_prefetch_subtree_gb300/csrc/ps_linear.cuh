// A projection with 16-bit weights: what its kernel and its entry point share.
#pragma once

#include "ps_internal.cuh"

namespace ps {

struct LinearParams {
    ps_linear lin;              // device pointers
    const void *x;
    int64_t x_ld;
    int32_t n_rows;
    int32_t dtype;              // of out and residual
    const void *residual;       // or NULL
    int64_t residual_ld;
    void *out;
    int64_t ld;
};

// lost: ps_selftest_linear_wait.
cudaError_t launch_linear(const LinearParams &p, int sms, bool lost, cudaStream_t stream);

}  // namespace ps
