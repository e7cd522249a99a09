// out = act(x W^T + b) + residual with bfloat16 weights and rows (ps_linear_rows).
//
// The products are tcgen05's: 128 rows of W are the first operand and N rows of x the
// second, 64 k of both a step, brought by TMA into a ring in shared memory.  A lane of
// tensor memory is then a row of W, so neighbouring lanes store neighbouring outputs of one
// row of x, and a lane's bias is one value.  One warp brings, one issues, eight take sums
// out (four took as long as the products: 2000 rows 2411 us); sums have two places, so that
// one tile's leave while the next one's are made.
//   N   16, 32, 64, 128 or 256: what the rows of x fill.  Few rows are bound by the weights'
//       bytes, for which the ring holds 200 KB under way: one row of 151936 x 4096 takes 184
//       to 189 us, 6.6 TB/s.  Many are bound by the products: 2000 rows 1560 us, 1.6 PFLOP/s;
//       small K by the way out: 1158 rows of 262144 x 256 222 to 257 us (450 before outputs
//       were converted in pairs and their addresses stepped), capped 384 to 457.
//   C   of 256 rows a tile two blocks share a product and bring half of x's rows each.
//   S   where W has too few tiles for all multiprocessors and few rows of x, the S blocks of
//       a cluster divide k, and the first adds the others' float32 sums in their order.
// Blocks take tiles in the order of W's rows and then x's, so that those that run together
// read the same weights.
//
// Every wait is bounded.  Where one runs out, nothing more is handed on, the waits after
// it run out too, and NaN is stored for what could not be made.
#include "ps_linear.cuh"

#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "ps_api.cuh"
#include "ps_tensor.cuh"

namespace ps {
namespace {

constexpr int kRows = 128, kStep = 64;                        // of W a tile; of k a step
constexpr int kBytesW = kRows * kStep * 2;
constexpr int kOutWarps = 8, kThreads = (2 + kOutWarps) * 32;
// Tensor-core sums are rounded towards zero: one of 512 products of 16 is off by 1.7e-6 of its
// size where float32 additions are by 4e-7.  After every 32, added to a float32 in registers
// rounded to nearest, it is at most 5e-7, after every 8 1e-7.
template <int N>
constexpr int kExactSteps = N == 256 ? 8 : 2;
constexpr int kMostRing = 11, kMostSplit = 8;
constexpr int kSmem = 226 * 1024;
constexpr uint64_t kTestWaitNs = 100000000ull;                // in the diagnostic variant

struct Bars {
    uint64_t full[kMostRing], empty[kMostRing];
    uint64_t made[2], taken[2];
    uint64_t drained;
    Place issued;                                             // of the last copy
    uint32_t tmem;
    int failed;
};

// One product of 16 k: of a block, or of the two of a cluster, 128 rows of W and of the sums
// in each, half of x's rows.
template <int C>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (C == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)add)
            : "memory");
}
// An arrival, in each block, when the products so far have ended.
template <int C>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (C == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
}
// The same in this block alone.
template <int C>
__device__ __forceinline__ void commit_here(uint64_t *bar) {
    if constexpr (C == 1)
        commit<1>(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A copy into this block that the first block of a pair counts, at the barrier's address there.
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// The address of `p` in the shared memory of the cluster's block `rank`.
__device__ __forceinline__ uint32_t address_at(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z, float cap, float inv_cap) {
    if constexpr (ACT == PS_ACT_CAP) return cap * tanhf(z * inv_cap);
    if constexpr (ACT == PS_ACT_SILU) return __fdividef(z, 1.f + expf(-z));
    if constexpr (ACT == PS_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678f);
    return z;
}

__device__ __forceinline__ float bias_of(const LinearParams &p, int v) {
    if (!p.lin.bias || v >= p.lin.N) return 0.f;
    return p.lin.bias_dtype == PS_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.lin.bias)[v])
                                       : reinterpret_cast<const float *>(p.lin.bias)[v];
}
// Sixteen rows' residuals at one row of W, loaded all at once; rows past the last are not used.
template <bool HALF, bool FLOAT>
__device__ __forceinline__ void residual_of(const LinearParams &p, int64_t r, int v, int n, float (&res)[16]) {
    if (n <= 0) return;
    if (HALF && (!FLOAT || p.dtype == PS_BF16)) {
        const uint16_t *from = reinterpret_cast<const uint16_t *>(p.residual) + r * p.residual_ld + v;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            res[i] = __uint_as_float((uint32_t)__ldcg(from) << 16);
            if (i + 1 < n) from += p.residual_ld;
        }
    } else {
        const float *from = reinterpret_cast<const float *>(p.residual) + r * p.residual_ld + v;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            res[i] = __ldcg(from);
            if (i + 1 < n) from += p.residual_ld;
        }
    }
}
// Sixteen rows' outputs at one row of W, from the sums with the bias; rounded once.
template <int ACT, typename OutT>
__device__ __forceinline__ void put16(const LinearParams &p, int64_t r, int v, const float (&z)[16], const float (&res)[16], int n) {
    const float cap = p.lin.cap, inv_cap = ACT == PS_ACT_CAP ? __frcp_rn(cap) : 0.f;
    OutT *out = reinterpret_cast<OutT *>(p.out) + r * p.ld + v;
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = act_of<ACT>(z[i], cap, inv_cap);
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] += res[i];
    }
    auto store = [&](int i) {
        if constexpr (sizeof(OutT) == 2) {
            // two are rounded together
            const __nv_bfloat162 two = __floats2bfloat162_rn(y[i & ~1], y[i | 1]);
            *out = i & 1 ? two.y : two.x;
        } else {
            *out = y[i];
        }
        out += p.ld;
    };
    if (n >= 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) store(i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) store(i);
    }
}
// HALF, FLOAT: the types that a kernel's outputs may have.
template <bool HALF, bool FLOAT>
__device__ __forceinline__ void put_out(const LinearParams &p, int64_t r, int v, const float (&z)[16], const float (&res)[16], int n) {
    auto as = [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        if constexpr (HALF && FLOAT) {
            if (p.dtype == PS_BF16) put16<kAct, __nv_bfloat16>(p, r, v, z, res, n);
            else put16<kAct, float>(p, r, v, z, res, n);
        } else if constexpr (HALF) {
            put16<kAct, __nv_bfloat16>(p, r, v, z, res, n);
        } else {
            put16<kAct, float>(p, r, v, z, res, n);
        }
    };
    switch (p.lin.act) {
        case PS_ACT_CAP: return as(std::integral_constant<int, PS_ACT_CAP>());
        case PS_ACT_SILU: return as(std::integral_constant<int, PS_ACT_SILU>());
        case PS_ACT_GELU: return as(std::integral_constant<int, PS_ACT_GELU>());
        default: return as(std::integral_constant<int, PS_ACT_NONE>());
    }
}

// EXACT: sums of kExact steps are added up in registers, for float32 outputs and divided k.
// LOST (the diagnostic variant): the first block brings no copies once its ring has been filled.
template <int N, int C, bool SPLIT, bool EXACT, bool LOST>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const LinearParams p, const int n_ring, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
    constexpr int kBytesX = N / C * kStep * 2, kSlot = kBytesW + kBytesX;
    static_assert(C == 1 || !SPLIT, "a cluster is a pair or divides k");
    static_assert(EXACT || !SPLIT, "a divided k's sums are in registers");
    constexpr uint32_t kCols = 2 * N < 32 ? 32 : 2 * N;
    constexpr int kExact = kExactSteps<N>;
    constexpr uint64_t kLimit = LOST ? kTestWaitNs : kTensorWaitNs;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    volatile int *failed = &bars.failed;
    uint8_t *ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    float *others = reinterpret_cast<float *>(ring + n_ring * kSlot);         // SPLIT: [S - 1][N][128]
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int V = p.lin.N;
    const uint32_t rank = SPLIT || C > 1 ? cluster_rank() : 0;
    uint32_t split = 1;
    if (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));

    if (threadIdx.x == 0) {
        for (int i = 0; i < n_ring; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.made[i], 1);
            mbar_init(&bars.taken[i], kOutWarps * C);
        }
        mbar_init(&bars.drained, 1);
        bars.failed = 0;
        bars.issued = Place{0, 0};
        fence_mbar_init();
    }
    if (wid == 1) {
        if constexpr (C == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)), "n"(kCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)), "n"(kCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
        tc_before();
    }
    __syncthreads();
    if (SPLIT || C > 1) cluster_sync();
    tc_after();
    const uint32_t tmem = bars.tmem;

    const int n_cols = (p.n_rows + N - 1) / N, n_tiles = (V + C * kRows - 1) / (C * kRows);
    const int all_steps = (p.lin.K + kStep - 1) / kStep;
    const uint32_t part = SPLIT ? rank : 0, group = SPLIT ? split : C;
    const int step0 = (int)((int64_t)all_steps * part / split), n_steps = (int)((int64_t)all_steps * (part + 1) / split) - step0;
    const int64_t units = (int64_t)n_cols * n_tiles, unit0 = blockIdx.x / group, unit_step = gridDim.x / group;
    // of a pair, its first row of W in a tile, and of x
    const int w_off = C > 1 ? (int)rank * kRows : 0, x_off = C > 1 ? (int)rank * (N / C) : 0;
    bool ok = true;

    if (wid == 0) {
        // the producer
        if (lane == 0) {
            Place copy{0, 0};
            for (int64_t unit = unit0; unit < units; unit += unit_step) {
                const int tile = (int)(unit / n_cols), col = (int)(unit % n_cols);
                for (int s = 0; s < n_steps; ++s, copy.step(1, n_ring)) {
                    const uint32_t slot = copy.at;
                    if (copy.turn > 0) ok = ok && wait(&bars.empty[slot], (copy.turn - 1) & 1, failed, kLimit);
                    if (!ok || (LOST && blockIdx.x == 0 && copy.turn > 0)) continue;
                    const int k0 = (step0 + s) * kStep, w0 = tile * C * kRows + w_off, x0 = col * N + x_off;
                    const uint32_t to = smem_addr(ring + slot * kSlot);
                    // of a pair the first block counts both blocks' bytes
                    if (C == 1 || rank == 0) mbar_arrive_expect_tx(&bars.full[slot], C * kSlot);
                    if constexpr (C == 1) {
                        tma_2d(to, &map_w, k0, w0, &bars.full[slot]);
                        tma_2d(to + kBytesW, &map_x, k0, x0, &bars.full[slot]);
                    } else {
                        const uint32_t bar = address_at(&bars.full[slot], 0);
                        tma_pair(to, &map_w, k0, w0, bar);
                        tma_pair(to + kBytesW, &map_x, k0, x0, bar);
                    }
                    bars.issued = copy;
                }
            }
        }
    } else if (wid == 1) {
        // the products: bfloat16 operands, float32 sums; rows of 128 bytes, swizzled by 128, eight of them 1 KB
        constexpr uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(N / 8) << 17 | (uint32_t)(C * kRows / 16) << 24;
        constexpr uint64_t desc0 = (uint64_t)2 << 61 | (uint64_t)1 << 46 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 16;
        Place copy{0, 0}, sums{0, 0};
        // of a pair, the first block's for both
        for (int64_t unit = C > 1 && rank > 0 ? units : unit0; unit < units; unit += unit_step) {
            for (int s = 0; s < n_steps; ++s, copy.step(1, n_ring)) {
                const bool begins = EXACT ? s % kExact == 0 : s == 0;
                const bool ends = s == n_steps - 1 || (EXACT && s % kExact == kExact - 1);
                if (begins && sums.turn > 0) ok = ok && wait(&bars.taken[sums.at], (sums.turn - 1) & 1, failed, kLimit);
                ok = ok && wait(&bars.full[copy.at], copy.turn & 1, failed, kLimit);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_after();
                if (elect()) {
                    const uint32_t at = smem_addr(ring + copy.at * kSlot);
                    const uint64_t a = desc0 | (at >> 4 & 0x3fffu), b = desc0 | ((at + kBytesW) >> 4 & 0x3fffu);
#pragma unroll
                    for (int i = 0; i < kStep / 16; ++i) mma<C>(tmem + sums.at * N, a + 2 * i, b + 2 * i, idesc, !begins || i > 0);
                    commit<C>(&bars.empty[copy.at]);
                    if (ends) commit<C>(&bars.made[sums.at]);
                }
                __syncwarp();
                if (ends) sums.step(1, 2);
            }
        }
    } else {
        // taking sums out: a lane has a row of W
        const int quarter = wid & 3, row = quarter * 32 + lane, c0 = (wid - 2) / 4 * 16;
        const uint32_t lanes = (uint32_t)quarter << 21;
        Place sums{0, 0};
        auto taken = [&] {
            tc_before();
            __syncwarp();
            if (lane == 0 && ok) {
                if (C == 1) arrive(&bars.taken[sums.at]);
                else arrive_at(&bars.taken[sums.at], 0);
            }
            sums.step(1, 2);
        };
        auto made = [&] {
            ok = ok && wait(&bars.made[sums.at], sums.turn & 1, failed, kLimit);
            ok = __all_sync(0xffffffffu, ok);
            tc_after();
        };
        for (int64_t unit = unit0; unit < units; unit += unit_step) {
            const int v = (int)(unit / n_cols) * C * kRows + w_off + row, n0 = (int)(unit % n_cols) * N;
            const float bias = bias_of(p, v);
            if (p.residual) {
                // a lane a row: the residual's pieces are in L2 when the sums are made
                const int first = v - lane, esz = p.dtype == PS_BF16 ? 2 : 4;
                for (int c = c0; c < N; c += 32)
                    if (lane < 16 && n0 + c + lane < p.n_rows && first < V)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t *>(p.residual) +
                                                                      ((int64_t)(n0 + c + lane) * p.residual_ld + first) * esz));
            }
            if constexpr (EXACT) {
                constexpr int kGroups = (N + 31) / 32;
                float total[kGroups][16];
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
#pragma unroll
                    for (int i = 0; i < 16; ++i) total[q][i] = 0.f;
                for (int s = 0; s < n_steps; s += kExact) {
                    made();
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        if (c0 + q * 32 >= N) break;
                        uint32_t x[16];
                        tmem_load16(tmem + sums.at * N + lanes + c0 + q * 32, x);
                        tmem_loaded(x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) total[q][i] += __uint_as_float(x[i]);
                    }
                    taken();
                }
                const float nan = ok ? 0.f : __int_as_float(0x7fffffff), add = bias + nan;
                if (SPLIT && rank > 0) {
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        const int c = c0 + q * 32;
                        if (c >= N) break;
                        const uint32_t to = address_at(others + ((rank - 1) * N + c) * kRows + row, 0);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * kRows * 4), "f"(total[q][i] + nan) : "memory");
                    }
                }
                if constexpr (SPLIT) {
                    // a cluster has one tile; the other warps are on their way to this
                    __syncwarp();
                    cluster_sync();
                }
                if (rank == 0 || !SPLIT) {
                    const bool more = p.residual && v < V;
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        const int c = c0 + q * 32;
                        if (c >= N || n0 + c >= p.n_rows) break;
                        float res[16];
                        if (more) residual_of<SPLIT, true>(p, n0 + c, v, p.n_rows - n0 - c, res);
                        for (uint32_t o = 0; SPLIT && o + 1 < split; ++o) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) total[q][i] += others[(o * N + c + i) * kRows + row];
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) total[q][i] += add;
                        if (v < V) put_out<SPLIT, true>(p, n0 + c, v, total[q], res, p.n_rows - n0 - c);
                    }
                }
            } else {
                float res[16], next[16];
                const bool more = p.residual && v < V;
                if (more && c0 < N) residual_of<true, false>(p, n0 + c0, v, p.n_rows - n0 - c0, res);
                made();
                const float add = ok ? bias : __int_as_float(0x7fffffff);
#pragma unroll 1
                for (int c = c0; c < N && n0 + c < p.n_rows; c += 32) {
                    __syncwarp();
                    uint32_t x[16];
                    float z[16];
                    tmem_load16(tmem + sums.at * N + lanes + c, x);
                    // the next residuals are on their way
                    if (more && c + 32 < N) residual_of<true, false>(p, n0 + c + 32, v, p.n_rows - n0 - c - 32, next);
                    tmem_loaded(x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(x[i]) + add;
                    if (v < V) put_out<true, false>(p, n0 + c, v, z, res, p.n_rows - n0 - c);
#pragma unroll
                    for (int i = 0; i < 16; ++i) res[i] = next[i];
                }
                taken();                                        // all have been in registers
            }
        }
    }
    if (SPLIT && wid < 2) {
        __syncwarp();
        cluster_sync();
    }
    __syncthreads();
    // Sums of all products have been taken out, so nothing is in flight; after a wait that
    // ran out, copies and products may be, and are waited for.
    if (__any_sync(0xffffffffu, *failed)) {
        auto drain = [&](uint64_t *bar, uint32_t parity) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kTensorWaitNs / 100) {}
        };
        if (wid == 0 && lane == 0 && (C == 1 || rank == 0))
            for (uint32_t i = 0; i < (uint32_t)n_ring; ++i) {
                // the last copy into a place: of the last copy's turn, or of the one before
                const uint32_t turns = bars.issued.turn + (i <= bars.issued.at);
                if (turns > 0) drain(&bars.full[i], (turns - 1) & 1);
            }
        // of a pair, by the thread that issues; the arrival is at its own block's barrier
        if (wid == 1 && (C == 1 || rank == 0) && elect()) {
            commit_here<C>(&bars.drained);
            drain(&bars.drained, 0);
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    if (C > 1) cluster_sync();
    if (wid == 1) {
        tc_after();
        if constexpr (C == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols));
    }
}

cudaError_t map_of(CUtensorMap *map, const void *p, int64_t rows, int32_t K, int64_t ld, int box) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t boxes[2] = {kStep, (cuuint32_t)box}, ones[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Tiles of the sums, of C blocks each.
int64_t units_of(const LinearParams &p, int N, int C) {
    return ((int64_t)p.lin.N + C * kRows - 1) / (C * kRows) * (((int64_t)p.n_rows + N - 1) / N);
}

template <int N, int C, bool SPLIT, bool EXACT, bool LOST>
cudaError_t launch(const LinearParams &p, int split, int sms, cudaStream_t stream) {
    constexpr int kSlot = kBytesW + N / C * kStep * 2;
    const int fixed = 1024 + (SPLIT ? (split - 1) * N * kRows * 4 : 0);
    const int n_ring = std::min((kSmem - (int)sizeof(Bars) - fixed) / kSlot, kMostRing);
    // First of all: in a thread that has used no CUDA before, this makes the device's
    // context current, without which the driver refuses to make a map.
    cudaError_t e = cudaFuncSetAttribute(linear_kernel<N, C, SPLIT, EXACT, LOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem - (int)sizeof(Bars));
    if (e != cudaSuccess) return e;
    CUtensorMap map_w, map_x;
    e = map_of(&map_w, p.lin.w, p.lin.N, p.lin.K, p.lin.w_ld, kRows);
    if (e == cudaSuccess) e = map_of(&map_x, p.x, p.n_rows, p.lin.K, p.x_ld, N / C);
    if (e != cudaSuccess) return e;
    const int64_t units = units_of(p, N, C);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SPLIT ? split : C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? units * split : std::min(units, (int64_t)sms / C) * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = fixed + n_ring * kSlot;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<N, C, SPLIT, EXACT, LOST>, p, n_ring, map_w, map_x);
}

// Blocks that divide k: as many as the multiprocessors have room for, with at least two
// steps each.  In a graph, divided and not: 16 rows of 4096 x 4096 9.5 / 21.8 us, 64 rows 12.5 /
// 22.9, 1 row of 8192 x 2048 9.5 / 12.7, 4 rows of 1024 x 1024 5.5 / 7.6.
int split_of(const LinearParams &p, int N, int sms) {
    const int64_t units = units_of(p, N, 1);
    const int steps = (p.lin.K + kStep - 1) / kStep;
    int s = 1;
    while (s < kMostSplit && units * s * 2 <= sms && steps >= s * 4) s *= 2;
    return s;
}

template <int N, bool LOST>
cudaError_t launch_n(const LinearParams &p, int sms, cudaStream_t stream) {
    const bool exact = p.dtype == PS_F32;
    if constexpr (N <= 64) {
        int s = split_of(p, N, sms);
        if (N == 64) s = std::min(s, 4);                       // the first block holds the others' sums
        if (s > 1) return launch<N, 1, true, true, LOST>(p, s, sms, stream);
    }
    // One block a tile and two, in us with a cold L2: 64 rows of 262144 x 2048 187 / 191, 128 of
    // 151936 x 4096 218 / 216, 256 of it 275 / 236, 2000 of it 1485 / 1404, 256 of 20000 x 4096
    // 81 / 68; so pairs for 256 rows a tile, where there are tiles for all.
    if constexpr (N == 256)
        if (units_of(p, N, 2) >= sms / 2)
            return exact ? launch<N, 2, false, true, LOST>(p, 1, sms, stream) : launch<N, 2, false, false, LOST>(p, 1, sms, stream);
    return exact ? launch<N, 1, false, true, LOST>(p, 1, sms, stream) : launch<N, 1, false, false, LOST>(p, 1, sms, stream);
}

cudaError_t launch_rows(const LinearParams &p, int sms, bool lost, cudaStream_t stream) {
    if (lost) return p.n_rows <= 64 ? launch_n<64, true>(p, sms, stream) : launch_n<256, true>(p, sms, stream);
    if (p.n_rows <= 16) return launch_n<16, false>(p, sms, stream);
    if (p.n_rows <= 32) return launch_n<32, false>(p, sms, stream);
    if (p.n_rows <= 64) return launch_n<64, false>(p, sms, stream);
    if (p.n_rows <= 128) return launch_n<128, false>(p, sms, stream);
    return launch_n<256, false>(p, sms, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearParams &params, int sms, bool lost, cudaStream_t stream) {
    // The kernel counts rows, a tile's last ones among them, in 32 bits.
    constexpr int64_t kMostRows = (int64_t)1 << 30;             // of a launch
    const int64_t esz = params.dtype == PS_BF16 ? 2 : 4;
    for (int64_t r = 0; r < params.n_rows; r += kMostRows) {
        LinearParams p = params;
        p.n_rows = (int32_t)std::min(params.n_rows - r, kMostRows);
        p.x = (const uint8_t *)params.x + r * params.x_ld * 2;
        p.out = (uint8_t *)params.out + r * params.ld * esz;
        if (params.residual) p.residual = (const uint8_t *)params.residual + r * params.residual_ld * esz;
        const cudaError_t e = launch_rows(p, sms, lost, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ps
