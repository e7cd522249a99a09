// The 4-bit output head: what its kernels and its entry point share.
#pragma once

#include "ps_internal.cuh"

namespace ps {

struct HeadParams {
    ps_head head;               // device pointers
    const uint16_t *hidden;     // bfloat16
    int64_t hidden_ld;
    int32_t n_rows;
    void *logits;
    int64_t ld;
    int32_t dtype;
};

cudaError_t launch_head_rows(const HeadParams &p, int sms, cudaStream_t stream);

}  // namespace ps
