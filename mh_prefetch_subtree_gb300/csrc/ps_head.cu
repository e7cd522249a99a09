// Logits rows from hidden states and a 4-bit output head (ps_head_rows): few hidden
// rows, or sizes that ps_head_tile.cu does not take.
//
// For few rows the weights are all that moves: V K / 2 bytes, each read once.
// A warp takes 16 MT vocabulary rows and multiplies them by 8 NT hidden rows with
// m16n8k16 matrix instructions: the weights are the 16-row operand, made in
// registers from the words that the lane has just loaded, so they never pass
// through shared memory.  The order of k inside a product is free as long as
// both operands have the same one, so it follows the packing: a lane loads 16
// bytes of its row, 32 consecutive k, and takes elements j and j + 4 of a word as a
// pair (one AND each).  The hidden rows are laid out once a block in shared
// memory, in that order.
//
// 4-bit to float16: 0x6400 | q is 1024 + q and 0x6400 | 16 q is 1024 + 16 q, so two
// of a word's pairs need no shift, and 1024 + q - (1024 + zero) and
// (1024 + 16 q) / 16 - (64 + zero) are exact.  (In bfloat16, with 7 bits of
// mantissa, every pair but one needs a shift: 1 row of 151936 x 4096 took 80 us,
// bound by the integer pipe.)  The hidden rows become float16 as well: each is
// scaled by the power of two that brings its largest element to 2^14 .. 2^15,
// which is taken back at the end.  That is exact but for elements below 2^-29 of
// the largest, which are rounded to a multiple of 2^-39 of it or so, far below the
// float32 sums' own rounding.  The sums of a unit of k (a group, or 128 elements of
// one) are scaled in float32.  With groups of 32 or 64 a lane's 16 bytes are not
// spread over the four lanes of a quad as one product needs them, so the quad
// first exchanges words.
//
// What bounds it: memory brings a multiprocessor 1 KB of weights every 43 cycles.
// The integer pipe, which takes one instruction every other cycle, is at work 68% of the
// time (1 row of 151936 x 4096, 68 us); unpacking, 5 integer instructions of 9 for
// 8 weights, is less than half of that, and the rest is addresses (clamped for each
// load), scale and zero words, and group indices.
#include "ps_head.cuh"

namespace ps {
namespace {

constexpr int kHeadSmem = 200 * 1024;  // for hidden rows
constexpr int kMaxStageK = 8192;       // hidden elements laid out at a time, when not all fit

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The words of a quad's 128 k, 4 in each lane, regrouped so that each unit of U k
// has U / 32 words in every lane: word slot `unit U/32 + i`.
template <int U>
__device__ __forceinline__ void spread(uint32_t (&q)[4], int tig) {
    if constexpr (U == 128) return;
    const bool hi = tig & 2;
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, hi ? q[0] : q[2], 2);
    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, hi ? q[1] : q[3], 2);
    // lanes 0, 1: their units' words 0, 1, then those of lanes 2, 3; lanes 2, 3:
    // words 2, 3 of lanes 0, 1, then their own
    uint32_t a0 = hi ? r0 : q[0], a1 = hi ? r1 : q[1], b0 = hi ? q[2] : r0, b1 = hi ? q[3] : r1;
    if constexpr (U == 32) {
        // (unit 0 or 1: a, unit 2 or 3: b) of the pair's lanes: one word of each to both
        const bool odd = tig & 1;
        const uint32_t ra = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
        const uint32_t rb = __shfl_xor_sync(0xffffffffu, odd ? b0 : b1, 1);
        const uint32_t ka = odd ? a1 : a0, kb = odd ? b1 : b0;
        a0 = odd ? ra : ka;
        a1 = odd ? ka : ra;
        b0 = odd ? rb : kb;
        b1 = odd ? kb : rb;
    }
    q[0] = a0;
    q[1] = a1;
    q[2] = b0;
    q[3] = b1;
}

// Where the 8 k from 8 c on are after spread(): the lane of the quad and the slot.
template <int U>
__device__ __forceinline__ void place(int c, int &tig, int &slot) {
    const int lane = c / 4, w = c % 4;               // as loaded
    if constexpr (U == 128) {
        tig = lane;
        slot = w;
    } else if constexpr (U == 64) {
        tig = (lane & 1) | (w & 2);
        slot = (lane & 2) | (w & 1);
    } else {
        // word w of lane (its unit) goes to lane w
        tig = w;
        slot = lane;
    }
}

// A scale and its group's zero, as one or two words.
template <typename ScaleT>
struct ScaleZero;
template <>
struct ScaleZero<uint16_t> {
    uint32_t w;
    __device__ __forceinline__ void load(const uint16_t *s, const uint8_t *z) {
        w = (uint32_t)__ldg(s) << 16 | (z ? __ldg(z) & 15u : 8u);
    }
    __device__ __forceinline__ ScaleZero from(int lane) const {
        return ScaleZero{__shfl_sync(0xffffffffu, w, lane)};
    }
    __device__ __forceinline__ float scale() const { return __uint_as_float(w & 0xffff0000u); }
    __device__ __forceinline__ uint32_t zero() const { return w & 0xffffu; }
};
template <>
struct ScaleZero<float> {
    float s;
    uint32_t z;
    __device__ __forceinline__ void load(const float *sp, const uint8_t *zp) {
        s = __ldg(sp);
        z = zp ? __ldg(zp) & 15u : 8u;
    }
    __device__ __forceinline__ ScaleZero from(int lane) const {
        return ScaleZero{__shfl_sync(0xffffffffu, s, lane), __shfl_sync(0xffffffffu, z, lane)};
    }
    __device__ __forceinline__ float scale() const { return s; }
    __device__ __forceinline__ uint32_t zero() const { return z; }
};

// U: elements of k whose sums share a scale (32, 64 or 128).  wk warps of a block
// share a tile's k.  K is laid out whole, or where it does not fit (then NT is 1)
// in parts that all warps of the block work on together.
template <int U, int NT, int MT, int WARPS, typename ScaleT>
__global__ void __launch_bounds__(WARPS * 32, 1) head_rows_kernel(const HeadParams p, int wk, int stage_k) {
    extern __shared__ __align__(16) uint4 smem4[];
    constexpr int kHeadWarps = WARPS, kHeadThreads = WARPS * 32;
    constexpr int W = U / 32;                        // words of a unit in a lane
    constexpr int kUnits = 4 / W;                    // units of a 128-k step
    constexpr int kPf = MT * WARPS == 32 ? 2 : 4;     // steps in flight; divides 4
    constexpr int kRows = 16 * MT, kCols = 8 * NT;
    __shared__ int power[kCols];                     // of each hidden row
    float *part = reinterpret_cast<float *>(smem4 + (size_t)NT * stage_k);      // [warps][kCols][kRows]
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int g = lane >> 2, tig = lane & 3;
    const int32_t V = p.head.V, K = p.head.K;
    const int groups = K / p.head.group;
    // a 128-k step's group, where groups are longer: step / (group / 128)
    const uint32_t long_group = U == 128 && p.head.group > 128 ? 0xffffffffu / (p.head.group / 128) + 1 : 0;
    const int64_t n_tiles = ((int64_t)V + kRows - 1) / kRows;
    const int per = kHeadWarps / wk, kw = wid % wk;
    const int n_cols = (p.n_rows + kCols - 1) / kCols;
    const int64_t n_work = (n_tiles + per - 1) / per * n_cols;
    int laid_n0 = -1;
    for (int64_t work = blockIdx.x; work < n_work; work += gridDim.x) {
        // blocks next to each other take the same weights for other rows
        const int n0 = (int)(work % n_cols) * kCols;
        const int64_t t0 = work / n_cols * per, tile = t0 + wid / wk;
        const bool live = tile < n_tiles;
        // the tile's weights, scales and zeros, and where the lane's rows begin in them
        const int64_t v0 = min(tile * kRows, (int64_t)V - 1);
        const uint8_t *tile_q = p.head.q + v0 * (K / 2);
        const ScaleT *tile_s = reinterpret_cast<const ScaleT *>(p.head.scales) + v0 * groups;
        const uint8_t *tile_z = p.head.zeros ? p.head.zeros + v0 * groups : nullptr;
        uint32_t row_q[MT][2], row_s[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t row = min((int64_t)(i * 16 + j * 8 + g), V - 1 - v0);
                row_q[i][j] = row * (uint32_t)(K / 2);
                row_s[i][j] = row * (uint32_t)groups;
            }
        if (laid_n0 != n0) {
            // the power of two of each hidden row, from its largest finite element
            __syncthreads();
            for (int n = wid; n < kCols; n += kHeadWarps) {
                const int e = n0 + n < p.n_rows
                                  ? row_power(p.hidden + (int64_t)(n0 + n) * p.hidden_ld, K, lane) : 0;
                if (lane == 0) power[n] = e;
            }
            __syncthreads();
        }
        float total[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) total[i][n][j] = 0.f;
        for (int32_t ks = 0; ks < K; ks += stage_k) {
            const int32_t kn = min(stage_k, K - ks);
            if (stage_k < K || laid_n0 != n0) {
                laid_n0 = n0;
                __syncthreads();
                for (int i = threadIdx.x; i < NT * kn; i += kHeadThreads) {
                    const int n = i % kCols, c = i / kCols;             // 8 k from ks + 8 c on
                    uint4 h = make_uint4(0, 0, 0, 0);
                    if (n0 + n < p.n_rows)
                        h = __ldg(reinterpret_cast<const uint4 *>(
                            p.hidden + (int64_t)(n0 + n) * p.hidden_ld + ks + c * 8));
                    int tg, at;
                    if (c / 16 < kn / 128) {
                        place<U>(c % 16, tg, at);
                        at += c / 16 * 4;
                    } else {                                            // the rest: units one by one
                        const int u = c / (U / 8), in = c % (U / 8);
                        tg = in / W;
                        at = u * W + in % W;
                    }
                    smem4[(size_t)(n / 8) * kn + at * 32 + (n % 8) * 4 + tg] = hidden_pairs(h, make_float2(times_power(1.f, power[n] / 2), times_power(1.f, power[n] - power[n] / 2)));
                }
                __syncthreads();
            }
            if (!live) continue;
            // adds the sums of one unit, from the lane's words of it
            auto unit = [&](const uint32_t *(&a)[MT], const uint32_t *(&b)[MT], int at,
                            const ScaleZero<ScaleT> (&sz)[MT][2]) {
                float c[MT][NT][4];
                uint32_t z1[MT][2], z16[MT][2];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        z1[i][j] = sz[i][j].zero() * 0x10001u + 0xe400e400u;
                        z16[i][j] = sz[i][j].zero() * 0x100010u + 0xd400d400u;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) c[i][n][j] = 0.f;
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint4 h[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) h[n] = smem4[n * kn + (at + w) * 32 + lane];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t x[4], y[4];
                        unpack(a[i][w], z1[i][0], z16[i][0], x);
                        unpack(b[i][w], z1[i][1], z16[i][1], y);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(c[i][n], x[0], y[0], x[1], y[1], h[n].x, h[n].y);
                            mma16816(c[i][n], x[2], y[2], x[3], y[3], h[n].z, h[n].w);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            total[i][n][j] = fmaf(sz[i][j >> 1].scale(), c[i][n][j], total[i][n][j]);
            };
            // the scale and zero of unit u, counted from k = 0
            auto scale_zero = [&](ScaleZero<ScaleT> &sz, int i, int j, uint32_t u) {
                if (U == 128 && long_group) u = __umulhi(u, long_group);
                u += row_s[i][j];
                sz.load(tile_s + u, tile_z ? tile_z + u : nullptr);
            };
            // this warp's steps: a run, in rounds of four.  Lane `tig` of a quad holds
            // the scales of the round's step `tig`.
            const int n_step = kn / 128, s0 = n_step * kw / wk, s1 = n_step * (kw + 1) / wk;
            if (s0 < s1) {
                uint32_t buf[kPf][MT][2][4];
                ScaleZero<ScaleT> held[kUnits][MT][2], next[kUnits][MT][2];
                // past the end the last step is read again
                auto fetch = [&](int st, int f) {
                    st = min(st, s1 - 1);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                        {
                            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(
                                tile_q + (row_q[i][j] + (uint32_t)(ks / 2 + st * 64 + tig * 16))));
                            buf[f][i][j][0] = x.x;
                            buf[f][i][j][1] = x.y;
                            buf[f][i][j][2] = x.z;
                            buf[f][i][j][3] = x.w;
                        }
                };
                auto fetch_scales = [&](int st) {
                    st = ks / 128 + min(st + tig, s1 - 1);
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) scale_zero(next[u][i][j], i, j, st * kUnits + u);
                };
                fetch_scales(s0);
#pragma unroll
                for (int f = 0; f < kPf; ++f) fetch(s0 + f, f);
                for (int st = s0; st < s1; st += 4) {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) held[u][i][j] = next[u][i][j];
                    if (st + 4 < s1) fetch_scales(st + 4);
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        if (st + f >= s1) break;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            spread<U>(buf[f % kPf][i][0], tig);
                            spread<U>(buf[f % kPf][i][1], tig);
                        }
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            const uint32_t *a[MT], *b[MT];
                            ScaleZero<ScaleT> sz[MT][2];
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                a[i] = &buf[f % kPf][i][0][u * W];
                                b[i] = &buf[f % kPf][i][1][u * W];
                                sz[i][0] = held[u][i][0].from((lane & ~3) + f);
                                sz[i][1] = held[u][i][1].from((lane & ~3) + f);
                            }
                            unit(a, b, (st + f) * 4 + u * W, sz);
                        }
                        fetch(st + f + kPf, f % kPf);
                    }
                }
            }
            // what is left of k after whole steps: units, by the words of the unit
            if constexpr (U < 128) {
                for (int u = n_step * kUnits + kw; u < kn / U; u += wk) {
                    uint32_t q[MT][2][W];
                    const uint32_t *a[MT], *b[MT];
                    ScaleZero<ScaleT> sz[MT][2];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int w = 0; w < W; ++w)
                                q[i][j][w] = __ldg(reinterpret_cast<const uint32_t *>(
                                    tile_q + (row_q[i][j] + (uint32_t)(ks / 2 + u * (U / 2) + tig * (U / 8)))) + w);
                            scale_zero(sz[i][j], i, j, ks / U + u);
                        }
                        a[i] = q[i][0];
                        b[i] = q[i][1];
                    }
                    unit(a, b, u * W, sz);
                }
            }
        }
        auto store = [&](int n, int64_t v, float x) {
            if (v >= V || n0 + n >= p.n_rows) return;
            const int64_t at = (int64_t)(n0 + n) * p.ld + v;
            x = times_power(x, -power[n]);
            if (p.dtype == PS_BF16)
                reinterpret_cast<__nv_bfloat16 *>(p.logits)[at] = __float2bfloat16_rn(x);
            else
                reinterpret_cast<float *>(p.logits)[at] = x;
        };
        if (wk == 1) {
            if (live)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            store(n * 8 + tig * 2 + (j & 1), tile * kRows + i * 16 + g + (j >> 1) * 8,
                                  total[i][n][j]);
        } else {
            // join the warps of a tile in order
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        part[(wid * kCols + n * 8 + tig * 2 + (j & 1)) * kRows + i * 16 + g + (j >> 1) * 8] =
                            total[i][n][j];
            __syncthreads();
            for (int i = threadIdx.x; i < per * kCols * kRows; i += kHeadThreads) {
                const int t = i / (kCols * kRows), n = i / kRows % kCols, m = i % kRows;
                float x = 0.f;
                for (int j = 0; j < wk; ++j) x += part[((t * wk + j) * kCols + n) * kRows + m];
                store(n, (t0 + t) * kRows + m, x);
            }
        }
    }
}

// Warps that share a tile's k: as few as give every warp work, and of those the
// number that leaves the least of it over in the last round.
int split_k(int64_t tiles, int64_t cols, int sms, int steps, int warps) {
    int best = 1;
    double least = 1e30;
    for (int wk = 1; wk <= warps && warps % wk == 0 && (wk == 1 || wk <= steps); wk *= 2) {
        const int64_t per = warps / wk, work = (tiles + per - 1) / per * cols;
        const double rounds = (double)((work + sms - 1) / sms) / wk;
        if (rounds < 0.9 * least) {
            least = rounds;
            best = wk;
        }
    }
    return best;
}

template <int U, int NT, int MT, int WARPS, typename ScaleT>
cudaError_t launch(const HeadParams &p, int sms, cudaStream_t stream) {
    const int K = p.head.K;
    const int stage_k = (int64_t)NT * K * 16 <= kHeadSmem ? K : kMaxStageK;
    const int64_t tiles = ((int64_t)p.head.V + 16 * MT - 1) / (16 * MT);
    const int64_t cols = ((int64_t)p.n_rows + 8 * NT - 1) / (8 * NT);
    const int wk = split_k(tiles, cols, sms, K / 128, WARPS);
    constexpr int kJoin = WARPS * 16 * MT * 8 * NT * 4;
    static_assert(kHeadSmem + kJoin <= 226 * 1024, "and 1 KB for what is static");
    const int smem = NT * stage_k * 16 + (wk > 1 ? kJoin : 0);
    // The most of any call: the limit belongs to the kernel, which calls with other sizes
    // may be launching from other threads.
    cudaError_t e = cudaFuncSetAttribute(head_rows_kernel<U, NT, MT, WARPS, ScaleT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kHeadSmem + kJoin);
    if (e != cudaSuccess) return e;
    const int64_t per = WARPS / wk, work = (tiles + per - 1) / per * cols;
    head_rows_kernel<U, NT, MT, WARPS, ScaleT>
        <<<(unsigned)(work < sms ? work : sms), WARPS * 32, smem, stream>>>(p, wk, stage_k);
    return cudaGetLastError();
}

// Hidden rows of a block: 8, 16 or 32, as many as there are and as fit.  With 8, a
// warp takes 32 vocabulary rows (1 row of 151936 x 4096: 68 us, with 16: 96), but 16 with
// groups of 32 (119 us, with 32: 124; 262144 x 2048: 105, 128); with more
// there are not the registers (16 rows: 105 us with 32, 92 with 16).  12 warps instead of
// 16 pay with 32 hidden rows only (64 rows of 262144 x 2048: 254 and 279 us; 8 warps 274).
template <int U, typename ScaleT>
cudaError_t launch_n(const HeadParams &p, int sms, cudaStream_t stream) {
    const int64_t fits = kHeadSmem / ((int64_t)p.head.K * 16);
    if (p.n_rows > 16 && fits >= 4) return launch<U, 4, 1, 12, ScaleT>(p, sms, stream);
    if (p.n_rows > 8 && fits >= 2) return launch<U, 2, 1, 16, ScaleT>(p, sms, stream);
    return launch<U, 1, U >= 64 ? 2 : 1, 16, ScaleT>(p, sms, stream);
}

template <int U>
cudaError_t launch_u(const HeadParams &p, int sms, cudaStream_t stream) {
    return p.head.scale_dtype == PS_BF16 ? launch_n<U, uint16_t>(p, sms, stream)
                                         : launch_n<U, float>(p, sms, stream);
}

}  // namespace

cudaError_t launch_head_rows(const HeadParams &p, int sms, cudaStream_t stream) {
    if (head_tile_takes(p, sms)) return launch_head_tile(p, sms, stream);
    if (p.head.group == 32) return launch_u<32>(p, sms, stream);
    if (p.head.group == 64) return launch_u<64>(p, sms, stream);
    return launch_u<128>(p, sms, stream);
}

}  // namespace ps
