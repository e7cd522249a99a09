// Logits rows of more than 16 hidden states and a 4-bit output head (ps_head_rows).
//
// With that many hidden rows the products outweigh the bytes, so they go to the
// tcgen05 tensor cores.  A pipeline of a block takes 128 vocabulary rows and
// multiplies them by N hidden rows, a unit of k (a group, or 128 elements of one) at
// a time:
//   the producer   brings 128 rows x 128 bytes of weights by TMA,
//   four warps     read a row each a lane, unpack it to float16 and store it to
//                  tensor memory, where it is the product's first operand,
//   one warp       issues the products of the unit into a fresh accumulator,
//   four warps     load the accumulator, a vocabulary row a lane, and add it times
//                  the group's scale to float32 totals in registers.
// So unpacked weights never go through shared memory, a group's scale is applied to
// its float32 sum, and the sums of one unit are taken in while the next are made.
// Two pipelines share the block's hidden rows, laid out once in shared memory as the
// second operand.  Where N rows of K do not fit there, two blocks of a cluster hold
// half of the rows each and one thread issues the products of both: 256 vocabulary
// rows, 128 in each block's tensor memory.  (Dividing K instead, each block's sums
// going to the other at the end of a tile, took 227 us where this takes 188; mma.sync
// with weights unpacked once for each 32 hidden rows 254: 64 rows of 262144 x 2048,
// group 64, where the weights alone need 47 us.)
//
// The unpacking and the scaling of the hidden rows are those of ps_head.cu.
//
// What bounds it: the round of a unit.  A unit goes through three hand-overs, two of
// them between blocks where there is a cluster, and tensor memory holds two or three
// units' sums; the warps that take sums in are at work two thirds of the time, about
// 1000 cycles a unit.  64 rows of 262144 x 2048: 145 us with groups of 128, 188 with
// 64, 324 with 32; without unpacking 132, 184, 323.  The tensor pipe is active 16% of
// the time with groups of 64, the issue slots 54%.  (16 rows at a time took 116 us for
// 151936 x 4096 where ps_head.cu takes 92.)
//
// Every wait is bounded.  Where one runs out, nothing more is handed on, the waits after
// it run out too, and NaN is stored for what could not be made.
#include <cuda.h>

#include "ps_head.cuh"

namespace ps {
namespace {

constexpr int kPipes = 2;
constexpr int kTileRows = 128;
constexpr int kStepBytes = 128, kStepK = 2 * kStepBytes;      // of a row, a copy
constexpr int kRingBytes = kTileRows * kStepBytes;
constexpr int kMostRing = 8, kMostWeights = 3, kMostSums = 4;
constexpr int kTileWarps = 9 * kPipes + 1, kTileThreads = kTileWarps * 32;
constexpr int kBytesB = 128 * 1024;                           // of hidden rows, at most
constexpr int kSmemB = 227 * 1024;
constexpr int kSmemStatic = 2 * 1024;                         // what is not dynamic, at most
constexpr int kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kTestWaitNs = 100000000ull;                // in the diagnostic variant

// A place in a ring, and how often it has gone round.
struct Place {
    uint32_t at, turn;
    __device__ __forceinline__ void step(uint32_t by, uint32_t ring) {
        at += by;
        if (at >= ring) at -= ring, ++turn;
    }
};

struct TileBars {
    uint64_t full[kMostRing], empty[kMostRing];               // the ring of copies
    uint64_t made[kPipes][kMostWeights], freed[kPipes][kMostWeights];
    uint64_t done[kPipes][kMostSums], taken[kPipes][kMostSums];
    uint64_t drained[kPipes];
    Place issued;                                             // of the last copy
    uint32_t tmem;
    int failed;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives at the barrier of the cluster's block `rank`.
__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.release.cta.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar)), "r"(rank)
        : "memory");
}
// The same variable of the cluster's block `rank`.
__device__ __forceinline__ void store_at(float2 *to, uint32_t rank, float x, float y) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(smem_addr(to)), "r"(rank), "f"(x), "f"(y)
        : "memory");
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// All threads of the block, or of the cluster.
template <int C>
__device__ __forceinline__ void sync_all() {
    __syncthreads();
    if (C > 1) cluster_sync();
}

// A bounded wait; once one of the block has run out, none waits any more.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *failed,
                                     uint64_t limit_ns = kWaitNs) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; i < (1u << 28); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        // the clock is slow to read: a wait of ordinary length does without
        if ((i & 255u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (*failed || now - t0 > limit_ns) break;
        }
    }
    *failed = 1;
    return false;
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]),
        "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
        : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
          "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
        : "r"(addr));
}
// The loads before it have ended: what they loaded passes through, so that no use moves up.
__device__ __forceinline__ void tmem_loaded(uint32_t (&x)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]),
                   "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]),
                   "+r"(x[14]), "+r"(x[15])::"memory");
}

// D (tensor memory, float32) = or += A (tensor memory) B (shared memory), 16 k; of
// one block, or of the two of a cluster: 128 rows of A and D in each, half of B.
template <int C>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (C == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
            "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
            "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
// An arrival, in each block, when the products so far have ended.
template <int C>
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    if constexpr (C == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar))
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
}

// The same in this block alone.
template <int C>
__device__ __forceinline__ void tc_commit_here(uint64_t *bar) {
    if constexpr (C == 1)
        tc_commit<1>(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar))
                     : "memory");
}

// One thread of the warp.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// (a, b) += (x, y) s
__device__ __forceinline__ void fma2(uint64_t &t, uint32_t x, uint32_t y, uint64_t ss) {
    uint64_t xy;
    asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "r"(x), "r"(y));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(xy), "l"(ss));
}

// The scales of a row's next eight units, shifted down as they are taken.
template <typename ScaleT>
struct Scales;
template <>
struct Scales<uint16_t> {
    uint32_t w[4];
    __device__ __forceinline__ void vector(const uint16_t *s) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(s));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void one(int i, const uint16_t *s) { w[i / 2] |= (uint32_t)__ldg(s) << i % 2 * 16; }
    __device__ __forceinline__ float take() {
        const float x = __uint_as_float(w[0] << 16);
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        w[3] >>= 16;
        return x;
    }
};
template <>
struct Scales<float> {
    float w[8];
    __device__ __forceinline__ void vector(const float *s) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(s)), y = __ldg(reinterpret_cast<const float4 *>(s) + 1);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
    __device__ __forceinline__ void clear() {}
    __device__ __forceinline__ void one(int i, const float *s) { w[i] = __ldg(s); }
    __device__ __forceinline__ float take() {
        const float x = w[0];
#pragma unroll
        for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
        return x;
    }
};

// LOST (a diagnostic): the first block leaves out the weight copies of all its tiles but
// the first of each pipeline and soon gives up the waits for them; the others are short.
template <int U, int N, int C, typename ScaleT, bool LOST>
__global__ void __launch_bounds__(kTileThreads, 1)
    head_tile_kernel(const HeadParams p, const int n_ring, const __grid_constant__ CUtensorMap map) {
    extern __shared__ uint8_t smem_raw[];
    // A pipeline's half of tensor memory: kA units of weights, U / 2 columns each, and
    // kD of sums, N columns each; more of sums, as their way round is the longer.
    constexpr int kA = N == 64 ? 2 : U == 128 ? 2 : 3, kFit = (kTmemCols / kPipes - kA * (U / 2)) / N;
    constexpr int kD = kFit < kMostSums ? kFit : kMostSums;
    static_assert(kD >= 2, "the sums of a unit are taken in while the next are made");
    constexpr int kUnitsStep = kStepK / U;
    __shared__ TileBars bars;
    constexpr int kHere = N / C;                                // hidden rows in this block
    __shared__ float2 scale_to[kHere], scale_back[N];           // powers of two, as two factors
    volatile int *failed = &bars.failed;
    constexpr uint64_t kLimit = LOST ? kTestWaitNs : kWaitNs;
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t *ring = smem;                                       // [ring][128 rows][128 B], swizzled
    uint4 *hid = reinterpret_cast<uint4 *>(smem + n_ring * kRingBytes);       // [k / 8][N]
    const int32_t V = p.head.V, K = p.head.K;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int n_units = K / U, n_steps = (K + kStepK - 1) / kStepK;

    if (threadIdx.x == 0) {
        for (int i = 0; i < n_ring; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 4);
        }
        for (int i = 0; i < kPipes; ++i) {
            for (int j = 0; j < kA; ++j) {
                mbar_init(&bars.made[i][j], 4 * C);
                mbar_init(&bars.freed[i][j], 1);
            }
            for (int j = 0; j < kD; ++j) {
                mbar_init(&bars.done[i][j], 1);
                mbar_init(&bars.taken[i][j], 4 * C);
            }
        }
        for (int i = 0; i < kPipes; ++i) mbar_init(&bars.drained[i], 1);
        bars.failed = 0;
        bars.issued = Place{0, 0};
        fence_mbar_init();
    }
    if (wid == 8 * kPipes) {
        if constexpr (C == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                         "n"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                         "n"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
        tc_before();
    }
    sync_all<C>();
    tc_after();
    const uint32_t tmem = bars.tmem;
    auto weights_at = [&](int pipe, int slot) { return tmem + pipe * (kTmemCols / kPipes) + slot * (U / 2); };
    auto sums_at = [&](int pipe, int slot) {
        return tmem + pipe * (kTmemCols / kPipes) + kA * (U / 2) + slot * N;
    };

    auto first_row = [&](int64_t pair, int pipe) { return ((pair * kPipes + pipe) * C + rank) * kTileRows; };
    // Clusters that share hidden rows divide the pairs of tiles; neighbours take the
    // same weights for other rows.
    const int n_clusters = gridDim.x / C, id = blockIdx.x / C;
    const int n_cols = (p.n_rows + N - 1) / N, member = min(n_cols, n_clusters);
    const int64_t n_pairs = ((int64_t)V + kPipes * C * kTileRows - 1) / (kPipes * C * kTileRows);
    const int64_t pair0 = id / member, pair_step = (n_clusters - id % member + member - 1) / member;

    // where this role is: in the ring of copies, the units of weights and those of sums
    const bool unpacks = wid < 4 * kPipes;
    Place copy{unpacks ? (uint32_t)wid / 4 : 0u, 0}, weights{0, 0}, sums{0, 0};
    for (int col = id % member; col < n_cols; col += member) {
        const int n0 = col * N;
        // the powers of two of this block's rows; a cluster's blocks tell each other theirs
        for (int n = wid; n < kHere; n += kTileWarps) {
            const int row = n0 + rank * kHere + n;
            const int e = row < p.n_rows ? row_power(p.hidden + (int64_t)row * p.hidden_ld, K, lane) : 0;
            if (lane == 0) scale_to[n] = make_float2(times_power(1.f, e / 2), times_power(1.f, e - e / 2));
            if (lane < C)
                store_at(&scale_back[rank * kHere + n], lane, times_power(1.f, -(e / 2)), times_power(1.f, e / 2 - e));
        }
        __syncthreads();
        // 8 rows of 4 times 8 k a warp: whole sectors read, no bank written twice
#pragma unroll 4
        for (int i = threadIdx.x; i < K / 8 * kHere; i += kTileThreads) {
            const int n = i / 32 % (kHere / 8) * 8 + i % 8, c = i / (4 * kHere) * 4 + i / 8 % 4;
            const int row = n0 + rank * kHere + n;
            uint4 h = make_uint4(0, 0, 0, 0);
            if (row < p.n_rows) h = __ldg(reinterpret_cast<const uint4 *>(p.hidden + (int64_t)row * p.hidden_ld) + c);
            hid[c * kHere + n] = hidden_pairs(h, scale_to[n]);
        }
        asm volatile("fence.proxy.async;" ::: "memory");
        sync_all<C>();
        // Once a wait has run out its role hands nothing on any more, so that the waits that
        // depend on it run out as well, and in the end those for sums.
        bool ok = __all_sync(0xffffffffu, !*failed);

        if (wid == 9 * kPipes) {
            // the producer
            if (lane == 0) {
                for (int64_t pair = pair0; pair < n_pairs; pair += pair_step)
                    for (int s = 0; s < n_steps; ++s)
                        for (int pipe = 0; pipe < kPipes; ++pipe, copy.step(1, n_ring)) {
                            const uint32_t slot = copy.at;
                            if (copy.turn > 0) ok = ok && wait(&bars.empty[slot], (copy.turn - 1) & 1, failed, kLimit);
                            if (!ok || (LOST && blockIdx.x == 0 && pair != pair0)) continue;
                            mbar_arrive_expect_tx(&bars.full[slot], kRingBytes);
                            tma_2d(smem_addr(ring + slot * kRingBytes), &map, s * kStepBytes, (int32_t)first_row(pair, pipe),
                                   &bars.full[slot]);
                            bars.issued = copy;
                        }
            }
        } else if (wid >= 8 * kPipes) {
            // the products of a pipeline: the warp waits as one, one of its threads issues; of a cluster,
            // the first block's for both
            constexpr uint32_t idesc = 1u << 4 | (uint32_t)(N / 8) << 17 | (uint32_t)(C * kTileRows / 16) << 24;
            // 8 rows x 16 bytes together; the next 8 k kHere 16 bytes on, the next 8 rows 128
            const uint64_t desc0 = (uint64_t)1 << 46 | (uint64_t)(128 >> 4) << 32 | (uint64_t)kHere << 16;
            // 14 bits: in a cluster an address has the rank of the block above them
            const uint32_t hid_at = smem_addr(hid) >> 4 & 0x3fffu;
            const int pipe = wid - 8 * kPipes;
            for (int64_t pair = rank ? n_pairs : pair0; pair < n_pairs; pair += pair_step)
                for (int u = 0; u < n_units; ++u, weights.step(1, kA), sums.step(1, kD)) {
                    if (sums.turn > 0) ok = ok && wait(&bars.taken[pipe][sums.at], (sums.turn - 1) & 1, failed, kLimit);
                    ok = ok && wait(&bars.made[pipe][weights.at], weights.turn & 1, failed, kLimit);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                    tc_after();
                    if (elect()) {
                        const uint64_t desc = desc0 | (hid_at + u * (U / 8) * kHere);
#pragma unroll
                        for (int i = 0; i < U / 16; ++i)
                            tc_mma<C>(sums_at(pipe, sums.at), weights_at(pipe, weights.at) + i * 8,
                                      desc + i * 2 * kHere, idesc, i > 0);
                        tc_commit<C>(&bars.done[pipe][sums.at]);
                        tc_commit<C>(&bars.freed[pipe][weights.at]);
                    }
                    __syncwarp();
                }
        } else if (unpacks) {
            // unpacking: a lane has a row
            const int pipe = wid / 4, row = threadIdx.x % kTileRows;
            const uint32_t lanes = (uint32_t)(wid % 4) << 21;
            const int groups = K / p.head.group;
            const uint32_t per_group = U == 128 ? p.head.group / 128 : 1;
            const bool wide = per_group == 1 && groups % 8 == 0 && (reinterpret_cast<uintptr_t>(p.head.zeros) & 7) == 0;
            uint32_t z[2], next[2] = {0x08080808u, 0x08080808u};
            auto fetch = [&](int64_t pair, int u0) {
                if (!p.head.zeros) return;
                const uint8_t *zeros = p.head.zeros + min(first_row(pair, pipe) + row, (int64_t)V - 1) * groups;
                if (wide) {
                    const uint2 x = __ldg(reinterpret_cast<const uint2 *>(zeros + u0));
                    next[0] = x.x, next[1] = x.y;
                } else {
                    next[0] = next[1] = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (u0 + i < n_units) next[i / 4] |= (uint32_t)__ldg(zeros + (u0 + i) / per_group) << i % 4 * 8;
                }
            };
            if (pair0 < n_pairs) fetch(pair0, 0);
            for (int64_t pair = pair0; ok && pair < n_pairs; pair += pair_step) {
                for (int u0 = 0; ok && u0 < n_units; u0 += 8) {
                    z[0] = next[0], z[1] = next[1];
                    if (u0 + 8 < n_units)
                        fetch(pair, u0 + 8);
                    else if (pair + pair_step < n_pairs)
                        fetch(pair + pair_step, 0);
                    const int n_now = min(8, n_units - u0);
#pragma unroll 1
                    for (int i = 0; i < n_now; ++i) {
                        const int u = u0 + i;
                        const uint32_t at = copy.at;
                        if (LOST && blockIdx.x == 0 && pair != pair0) {
                            // all four warps at once, so that the others have had no time to see it
                            const uint64_t t0 = global_timer_ns();
                            while (global_timer_ns() - t0 < kTestWaitNs / 20) {}
                            *failed = 1, ok = false;
                        }
                        if (i % kUnitsStep == 0) ok = ok && wait(&bars.full[at], copy.turn & 1, failed, kLimit);
                        const uint32_t slot = weights.at;
                        if (weights.turn > 0) ok = ok && wait(&bars.freed[pipe][slot], (weights.turn - 1) & 1, failed, kLimit);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_after();
                        const uint32_t zero = z[0] & 15u;
                        z[0] = __funnelshift_r(z[0], z[1], 8);
                        z[1] >>= 8;
                        const uint32_t z1 = zero * 0x10001u + 0xe400e400u, z16 = zero * 0x100010u + 0xd400d400u;
                        uint4 q[U / 32];
#pragma unroll
                        for (int c = 0; c < U / 32; ++c)
                            q[c] = *reinterpret_cast<const uint4 *>(
                                ring + at * kRingBytes + row * kStepBytes +
                                ((i % kUnitsStep * (U / 32) + c) ^ (row & 7)) * 16);
#pragma unroll
                        for (int c = 0; c < U / 32; ++c) {
                            const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
                            uint32_t x[16];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t y[4];
                                unpack(w[j], z1, z16, y);
#pragma unroll
                                for (int k = 0; k < 4; ++k) x[j * 4 + k] = y[k];
                            }
                            tmem_store16(weights_at(pipe, slot) + lanes + c * 16, x);
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        tc_before();
                        __syncwarp();
                        const bool last = (i + 1) % kUnitsStep == 0 || u + 1 == n_units;
                        if (lane == 0) {
                            if (C == 1) arrive(&bars.made[pipe][slot]);
                            else arrive_at(&bars.made[pipe][slot], 0);
                            if (last) arrive(&bars.empty[at]);
                        }
                        if (last) copy.step(kPipes, n_ring);
                        weights.step(1, kA);
                    }
                }
            }
        } else {
            // taking in the sums: a lane has a row
            const int pipe = (wid - 4 * kPipes) / 4, row = threadIdx.x % kTileRows;
            const uint32_t lanes = (uint32_t)(wid % 4) << 21;
            const int groups = K / p.head.group;
            const uint32_t per_group = U == 128 ? p.head.group / 128 : 1;
            const bool wide = per_group == 1 && groups % 8 == 0 && (reinterpret_cast<uintptr_t>(p.head.scales) & 15) == 0;
            Scales<ScaleT> held, next;
            auto fetch = [&](int64_t pair, int u0) {
                const ScaleT *scales = reinterpret_cast<const ScaleT *>(p.head.scales) +
                                       min(first_row(pair, pipe) + row, (int64_t)V - 1) * groups;
                if (wide)
                    next.vector(scales + u0);
                else {
                    next.clear();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (u0 + i < n_units) next.one(i, scales + (u0 + i) / per_group);
                }
            };
            if (pair0 < n_pairs) fetch(pair0, 0);
            for (int64_t pair = pair0; pair < n_pairs; pair += pair_step) {
                const int64_t v = first_row(pair, pipe) + row;
                uint64_t total[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) total[i] = 0;
                for (int u0 = 0; u0 < n_units; u0 += 8) {
                    held = next;
                    if (u0 + 8 < n_units)
                        fetch(pair, u0 + 8);
                    else if (pair + pair_step < n_pairs)
                        fetch(pair + pair_step, 0);
                    const int n_now = min(8, n_units - u0);
#pragma unroll 1
                    for (int i = 0; i < n_now; ++i) {
                        const uint32_t slot = sums.at;
                        ok = ok && wait(&bars.done[pipe][slot], sums.turn & 1, failed, kLimit);
                        ok = __all_sync(0xffffffffu, ok);
                        tc_after();
                        const float s = held.take();
                        uint64_t ss;
                        asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
                        for (int h = 0; h < N / 32; ++h) {
                            uint32_t x[2][16];
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tmem_load16(sums_at(pipe, slot) + lanes + h * 32 + c * 16, x[c]);
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                tmem_loaded(x[c]);
                                if (h == N / 32 - 1 && c == 1) {      // all are in registers
                                    tc_before();
                                    __syncwarp();
                                    if (lane == 0 && ok) {
                                        if (C == 1) arrive(&bars.taken[pipe][slot]);
                                        else arrive_at(&bars.taken[pipe][slot], 0);
                                    }
                                }
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    fma2(total[h * 16 + c * 8 + j], x[c][2 * j], x[c][2 * j + 1], ss);
                            }
                        }
                        sums.step(1, kD);
                    }
                }
                float sum[N];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    sum[2 * i] = __uint_as_float((uint32_t)total[i]);
                    sum[2 * i + 1] = __uint_as_float((uint32_t)(total[i] >> 32));
                }
                const int n_here = v < V ? p.n_rows - n0 : 0;
                const float nan = ok ? 0.f : __int_as_float(0x7fffffff);
                auto store = [&](int n, float x) {
                    if (n >= n_here) return;
                    const int64_t at = (int64_t)(n0 + n) * p.ld + v;
                    const float2 f = scale_back[n];
                    x = x * f.x * f.y + nan;
                    if (p.dtype == PS_BF16)
                        reinterpret_cast<__nv_bfloat16 *>(p.logits)[at] = __float2bfloat16_rn(x);
                    else
                        reinterpret_cast<float *>(p.logits)[at] = x;
                };
#pragma unroll
                for (int n = 0; n < N; ++n) store(n, sum[n]);
            }
        }
        sync_all<C>();
    }
    // The sums of all products have been taken in, so nothing is in flight; after a
    // wait that ran out, copies and products may be, and are waited for.
    if (__any_sync(0xffffffffu, *failed)) {
        auto drain = [&](uint64_t *bar, uint32_t parity) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitNs / 100) {}
        };
        if (wid == 9 * kPipes && lane == 0)
            for (uint32_t i = 0; i < (uint32_t)n_ring; ++i) {
                // the last copy into a place: of the last copy's turn, or of the one before
                const uint32_t turns = bars.issued.turn + (i <= bars.issued.at);
                if (turns > 0) drain(&bars.full[i], (turns - 1) & 1);
            }
        // the products, by the thread that issues them; the arrival is at its own block's
        // barrier, as the other block may be gone by the time that one there would come
        if (wid >= 8 * kPipes && wid < 9 * kPipes && rank == 0 && elect()) {
            tc_commit_here<C>(&bars.drained[wid - 8 * kPipes]);
            drain(&bars.drained[wid - 8 * kPipes], 0);
        }
    }
    __syncwarp();
    tc_before();
    sync_all<C>();
    if (wid == 8 * kPipes) {
        tc_after();
        if constexpr (C == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) !=
                cudaSuccess || r != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// Hidden rows of a product, 32 or 64, and the blocks that hold them, 1 or 2; no rows
// where K is too long for that.
struct Shape {
    int rows, blocks;
};
Shape shape_of(const HeadParams &p) {
    for (int n = p.n_rows > 32 ? 64 : 32; n >= 32; n /= 2)
        for (int c = 1; c <= 2; ++c)
            if ((int64_t)n / c * 2 * p.head.K <= kBytesB) return Shape{n, c};
    return Shape{0, 0};
}

template <int U, int N, int C, typename ScaleT, bool LOST = false>
cudaError_t launch(const HeadParams &p, int sms, cudaStream_t stream) {
    const int K = p.head.K, fixed = N / C * 2 * K;
    // 1 KB aligns the ring
    int n_ring = (kSmemB - kSmemStatic - 1024 - fixed) / kRingBytes;
    if (n_ring > kMostRing) n_ring = kMostRing;
    const int smem = 1024 + fixed + n_ring * kRingBytes;

    // First of all: in a thread that has used no CUDA before, this makes the device's
    // context current, without which the driver refuses to make a map.  The most of any
    // call: the limit belongs to the kernel, which calls with other sizes may be launching
    // from other threads.
    cudaError_t e = cudaFuncSetAttribute(head_tile_kernel<U, N, C, ScaleT, LOST>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemB - kSmemStatic);
    if (e != cudaSuccess) return e;

    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)p.head.V}, strides[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {kStepBytes, kTileRows}, ones[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(p.head.q), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;

    const int64_t work = ((int64_t)p.head.V + kPipes * C * kTileRows - 1) / (kPipes * C * kTileRows) *
                         (((int64_t)p.n_rows + N - 1) / N);
    const int64_t clusters = sms / C;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((work < clusters ? work : clusters) * C));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, head_tile_kernel<U, N, C, ScaleT, LOST>, p, n_ring, map);
}

template <int U, typename ScaleT>
cudaError_t launch_n(const HeadParams &p, int sms, cudaStream_t stream) {
    const Shape s = shape_of(p);
    if (s.rows == 64 || U == 32)
        return s.blocks == 1 ? launch<U, 64, 1, ScaleT>(p, sms, stream) : launch<U, 64, 2, ScaleT>(p, sms, stream);
    if constexpr (U > 32)
        return s.blocks == 1 ? launch<U, 32, 1, ScaleT>(p, sms, stream) : launch<U, 32, 2, ScaleT>(p, sms, stream);
    return cudaErrorNotSupported;
}

template <int U>
cudaError_t launch_u(const HeadParams &p, int sms, cudaStream_t stream) {
    return p.head.scale_dtype == PS_BF16 ? launch_n<U, uint16_t>(p, sms, stream)
                                         : launch_n<U, float>(p, sms, stream);
}

}  // namespace

// Where both run, in us, this kernel and that of ps_head.cu:
//   33 to 64 rows, 262144 x 2048, groups of 32, 64, 128: 308 / 336, 187 / 255, 144 / 230
//                  65536 x 3968:                        266 / 412, 177 / 371, 130 / 349
//   17 to 32 rows, 262144 x 2048:                        219 / 175, 152 / 140, 115 / 126
//                  151936 x 4096:                        259 / 252, 179 / 201, 130 / 171
//                  151936 x 1024:                         73 / 113, 57 / 109, 42 / 97
// so groups of 32 are left to the other but for 64 rows at a time.  Groups of 64 and up to
// 32 rows go either way: at 65536 and 151936 vocabulary rows this one takes 0.4 to 0.9 of the
// other's time (32 rows, K from 512 to 3200), at 262144, where the other's rounds come out
// even, it takes as long up to K = 1536 and 1.09 times as long above.  That is left so: a
// rule by the other's rounds would follow single sizes.  With few vocabulary rows
// it is the longer way of a unit that counts: 64 rows of 2000 x 4096 and groups of 128 take
// 48 / 23, of 20000 x 2048 42 / 44, 32 rows of 40000 x 512, 1024, 2048 and groups of 64
// 25 / 29, 37 / 38, 56 / 48, so a vocabulary has to fill all pipelines once.
bool head_tile_takes(const HeadParams &p, int sms) {
    const Shape s = shape_of(p);
    return p.n_rows > 16 && p.head.K >= kStepK && s.rows > 0 && (p.head.group > 32 || s.rows == 64) &&
           p.head.V >= (int64_t)sms * kPipes * kTileRows;
}

cudaError_t launch_head_tile(const HeadParams &p, int sms, cudaStream_t stream) {
    if (p.head.group == 32) return launch_u<32>(p, sms, stream);
    if (p.head.group == 64) return launch_u<64>(p, sms, stream);
    return launch_u<128>(p, sms, stream);
}

cudaError_t launch_head_lost(const HeadParams &p, int sms, cudaStream_t stream) {
    return shape_of(p).blocks == 1 ? launch<128, 64, 1, uint16_t, true>(p, sms, stream)
                                   : launch<128, 64, 2, uint16_t, true>(p, sms, stream);
}

}  // namespace ps
