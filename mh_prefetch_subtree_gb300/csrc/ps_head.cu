// Logits rows from hidden states and a 4-bit output head (ps_head_rows).
//
// For few rows the weights are all that moves: V K / 2 bytes, each read once.
// A warp takes 16 vocabulary rows and multiplies them by 8 hidden rows at a time
// with m16n8k16 matrix instructions: the weights are the 16-row operand, made
// in registers from the words that the lane has just loaded, so they never pass
// through shared memory.  The order of k inside a product is free as long as
// both operands have the same one, so it follows the packing: a lane loads
// consecutive words of its row and takes elements j and j + 4 of a word as a
// pair (one AND each).  The hidden rows are laid out once a block in shared
// memory, in that order.
//
// 4-bit to bfloat16: 0x4300 | q is 128 + q exactly, and (128 + q) - (128 + zero)
// is exact too, so the products have no rounding but the float32 sums'.  The
// sums of a unit of k (a group, or 128 elements of one) are scaled in float32.
#include <cuda_bf16.h>

#include "ps_head.cuh"

namespace ps {
namespace {

constexpr int kHeadThreads = 256;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kMaxStageK = 8192;      // hidden elements laid out at a time

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Elements j and j + 4 of a word, less the zero, as two bfloat16.
__device__ __forceinline__ uint32_t weight_pair(uint32_t word, int j, uint32_t zero128) {
    const uint32_t t = ((word >> (4 * j)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&t),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&zero128));
    return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ float load_scale(const HeadParams &p, int64_t i) {
    if (p.head.scale_dtype == PS_BF16)
        return __uint_as_float(
            (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p.head.scales) + i) << 16);
    return __ldg(reinterpret_cast<const float *>(p.head.scales) + i);
}

// U: elements of k whose sums share a scale (32, 64 or 128); a lane holds U / 32
// words of each of its two rows.  wk warps of a block share a tile's k.
template <int U>
__global__ void __launch_bounds__(kHeadThreads) head_rows_kernel(const HeadParams p, int wk) {
    extern __shared__ __align__(16) uint4 smem4[];
    constexpr int W = U / 32;
    __shared__ float part[kHeadWarps][16][8];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int g = lane >> 2, tig = lane & 3;
    const int32_t V = p.head.V, K = p.head.K;
    const int64_t groups = K / p.head.group;
    const int n0 = blockIdx.y * 8;
    const int64_t n_tiles = ((int64_t)V + 15) / 16;
    const int per = kHeadWarps / wk, kw = wid % wk;
    const bool one = K <= kMaxStageK;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < n_tiles; t0 += (int64_t)gridDim.x * per) {
        const int64_t tile = t0 + wid / wk;
        const int64_t r0 = min(tile * 16 + g, (int64_t)V - 1), r1 = min(tile * 16 + g + 8, (int64_t)V - 1);
        float total[4] = {0.f, 0.f, 0.f, 0.f};
        for (int32_t ks = 0; ks < K; ks += kMaxStageK) {
            const int32_t kn = min(kMaxStageK, K - ks);
            if (!one || t0 == (int64_t)blockIdx.x * per) {
                __syncthreads();
                for (int i = threadIdx.x; i < kn; i += kHeadThreads) {     // kn / 8 * 8 rows
                    const int n = i & 7, c = i >> 3;                        // 8 elements from k = 8 c
                    const int u = c / (U / 8), in = c % (U / 8);
                    const int tg = in / W, w = in % W;
                    uint4 h = make_uint4(0, 0, 0, 0);
                    if (n0 + n < p.n_rows)
                        h = __ldg(reinterpret_cast<const uint4 *>(
                            p.hidden + (int64_t)(n0 + n) * p.hidden_ld + ks + c * 8));
                    // pairs (0, 4), (1, 5), (2, 6), (3, 7)
                    uint4 o;
                    o.x = __byte_perm(h.x, h.z, 0x5410);
                    o.y = __byte_perm(h.x, h.z, 0x7632);
                    o.z = __byte_perm(h.y, h.w, 0x5410);
                    o.w = __byte_perm(h.y, h.w, 0x7632);
                    smem4[(u * W + w) * 32 + n * 4 + tg] = o;
                }
                __syncthreads();
            }
            if (tile < n_tiles) {
                const uint8_t *q0 = p.head.q + r0 * (K / 2) + ks / 2 + tig * (U / 8);
                const uint8_t *q1 = p.head.q + r1 * (K / 2) + ks / 2 + tig * (U / 8);
                for (int u = kw; u < kn / U; u += wk) {
                    uint32_t a[W], b[W];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        a[w] = __ldg(reinterpret_cast<const uint32_t *>(q0 + (int64_t)u * (U / 2)) + w);
                        b[w] = __ldg(reinterpret_cast<const uint32_t *>(q1 + (int64_t)u * (U / 2)) + w);
                    }
                    const int64_t gr = (ks + u * U) / p.head.group;
                    const float s0 = load_scale(p, r0 * groups + gr), s1 = load_scale(p, r1 * groups + gr);
                    uint32_t z0 = 8, z1 = 8;
                    if (p.head.zeros) {
                        z0 = __ldg(p.head.zeros + r0 * groups + gr) & 15u;
                        z1 = __ldg(p.head.zeros + r1 * groups + gr) & 15u;
                    }
                    z0 = 0x43004300u | z0 * 0x10001u;
                    z1 = 0x43004300u | z1 * 0x10001u;
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint4 h = smem4[(u * W + w) * 32 + lane];
                        mma16816(c, weight_pair(a[w], 0, z0), weight_pair(b[w], 0, z1),
                                 weight_pair(a[w], 1, z0), weight_pair(b[w], 1, z1), h.x, h.y);
                        mma16816(c, weight_pair(a[w], 2, z0), weight_pair(b[w], 2, z1),
                                 weight_pair(a[w], 3, z0), weight_pair(b[w], 3, z1), h.z, h.w);
                    }
                    total[0] = fmaf(s0, c[0], total[0]);
                    total[1] = fmaf(s0, c[1], total[1]);
                    total[2] = fmaf(s1, c[2], total[2]);
                    total[3] = fmaf(s1, c[3], total[3]);
                }
            }
        }
        // join the warps of a tile in order, then store
        __syncthreads();
        part[wid][g][tig * 2] = total[0];
        part[wid][g][tig * 2 + 1] = total[1];
        part[wid][g + 8][tig * 2] = total[2];
        part[wid][g + 8][tig * 2 + 1] = total[3];
        __syncthreads();
        for (int i = threadIdx.x; i < per * 128; i += kHeadThreads) {
            const int t = i / 128, n = (i / 16) % 8, m = i % 16;
            const int64_t v = (t0 + t) * 16 + m;
            if (v >= V || n0 + n >= p.n_rows) continue;
            float x = 0.f;
            for (int j = 0; j < wk; ++j) x += part[t * wk + j][m][n];
            const int64_t at = (int64_t)(n0 + n) * p.ld + v;
            if (p.dtype == PS_BF16)
                reinterpret_cast<__nv_bfloat16 *>(p.logits)[at] = __float2bfloat16_rn(x);
            else
                reinterpret_cast<float *>(p.logits)[at] = x;
        }
    }
}

template <int U>
cudaError_t launch(const HeadParams &p, int sms, cudaStream_t stream) {
    const int smem = (p.head.K < kMaxStageK ? p.head.K : kMaxStageK) * 16;
    cudaError_t e = cudaFuncSetAttribute(head_rows_kernel<U>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((int64_t)p.head.V + 15) / 16;
    int wk = 1;
    while (wk < kHeadWarps && tiles * wk < (int64_t)sms * 16) wk *= 2;
    const int64_t per = kHeadWarps / wk, want = (tiles + per - 1) / per, most = (int64_t)sms * 2;
    const dim3 grid((unsigned)(want < most ? want : most), (unsigned)((p.n_rows + 7) / 8));
    head_rows_kernel<U><<<grid, kHeadThreads, smem, stream>>>(p, wk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_rows(const HeadParams &p, int sms, cudaStream_t stream) {
    if (p.head.group == 32) return launch<32>(p, sms, stream);
    if (p.head.group == 64) return launch<64>(p, sms, stream);
    return launch<128>(p, sms, stream);
}

}  // namespace ps
