// The 4-bit output head: what its kernels and its entry point share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ __half2 h2_of(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }

// A small integer put into the low bits of a float's mantissa and the power of two that
// those bits then stand on taken off again, which is an old way to convert without a
// conversion; for 4-bit weights and float16 it is in Kim, Henry, Fahim and Hassan Awadalla,
// "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale
// Production" (2022).
// The four pairs (j, j + 4) of a word less the zero, as float16.  z1 holds
// -(1024 + zero) twice, z16 -(64 + zero).
__device__ __forceinline__ void unpack(uint32_t word, uint32_t z1, uint32_t z16, uint32_t (&x)[4]) {
    const uint32_t w8 = word >> 8;
    const __half2 sixteenth = h2_of(0x2c002c00u);
    x[0] = h2_bits(__hadd2(h2_of((word & 0x000f000fu) | 0x64006400u), h2_of(z1)));
    x[1] = h2_bits(__hfma2(h2_of((word & 0x00f000f0u) | 0x64006400u), sixteenth, h2_of(z16)));
    x[2] = h2_bits(__hadd2(h2_of((w8 & 0x000f000fu) | 0x64006400u), h2_of(z1)));
    x[3] = h2_bits(__hfma2(h2_of((w8 & 0x00f000f0u) | 0x64006400u), sixteenth, h2_of(z16)));
}

// x 2^e, where 2^e alone may be out of range.
__device__ __forceinline__ float times_power(float x, int e) {
    const int a = e / 2, b = e - a;
    return x * __int_as_float((a + 127) << 23) * __int_as_float((b + 127) << 23);
}

// The exponent that brings a hidden row's largest finite element to 2^14 .. 2^15,
// found by one warp; 0 for a row of zeros.
__device__ __forceinline__ int row_power(const uint16_t *row, int32_t K, int lane) {
    uint32_t top = 0;
#pragma unroll 8
    for (int i = lane; i < K / 8; i += 32) {
        const uint4 h = __ldg(reinterpret_cast<const uint4 *>(row) + i);
        const uint32_t x[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = x[j] & 0x7fffu, hi = x[j] >> 16 & 0x7fffu;
            if (lo < 0x7f80u) top = max(top, lo);
            if (hi < 0x7f80u) top = max(top, hi);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    return top ? 14 + 127 - max(1, (int)(top >> 7)) : 0;
}

// 8 hidden elements times 2^e as float16, in the order that unpack() makes of a
// word: the pairs (0, 4), (1, 5), (2, 6), (3, 7).
// 2^e comes as two factors, as it may be out of range.
__device__ __forceinline__ uint4 hidden_pairs(uint4 h, float2 e) {
    auto pair = [&](uint32_t lo, uint32_t hi) {
        return h2_bits(__floats2half2_rn(__uint_as_float(lo) * e.x * e.y, __uint_as_float(hi) * e.x * e.y));
    };
    return make_uint4(pair(h.x << 16, h.z << 16), pair(h.x & 0xffff0000u, h.z & 0xffff0000u),
                      pair(h.y << 16, h.w << 16), pair(h.y & 0xffff0000u, h.w & 0xffff0000u));
}

#endif  // __CUDACC__

// ps_head.cu; it leaves what ps_head_tile.cu takes to that.
cudaError_t launch_head_rows(const HeadParams &p, int sms, cudaStream_t stream);
bool head_tile_takes(const HeadParams &p, int sms);
cudaError_t launch_head_tile(const HeadParams &p, int sms, cudaStream_t stream);
// ps_selftest_head_wait: 33 to 64 hidden rows of at most 2048 elements, bfloat16 scales,
// groups of 128 or more.
cudaError_t launch_head_lost(const HeadParams &p, int sms, cudaStream_t stream);

}  // namespace ps
