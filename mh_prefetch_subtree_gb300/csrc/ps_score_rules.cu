// log p0, log q_tau and entropy of each row's token under rules
// (ps_score_rows_rules), without writing the processed rows.
//
// The formulation is ps_score_rows.cu's: sums relative to a reference, the token
// left out.  ps_rule_rows.cuh brings the rows to the block.  Its patchers take the
// token and the ids that penalties or biases touch out of the stage (their places
// become -inf) and hand their processed float32 values on apart, so nothing is
// rounded to the rows' type.  (Summed by the patchers themselves, those values cost
// the blocks with the most touched ids 30%.)  Each of the other 12 warps sums 64
// (float32: 32) ids and one such value a lane, with the mask applied: lane l of warp
// w has blocks of 32 ids 12 (32 h + l) + (w + l) % 12, where the skew puts the
// lanes' vectors in different banks.  What is left are 16 partial sums for each slice of a
// row, which a second kernel joins in their order.
//
// Where a mask leaves a lane at most kFewIds of its 64 (32 for float32) ids, the
// warp steps through the allowed ones instead of exponentiating all (events around one
// pass: 8000 rows of 151936 bf16 under 24 masks 543 us, never 662, up to 20 542; 1500 rows
// of 262144 with entropy 237, 296, 237; under masks that leave 0.1% of the ids 426, 625, 425
// and 190, 285, 191).
//
// The reference only has to keep the exponentials in range, so without entropy
// the warp keeps the one of the row before and looks for its ids' maximum only when
// the sums leave [2^-60, 2^64].  With entropy the sum of 2^y y cancels the more the
// further the reference is from the maximum, so each row takes its own.
#include "ps_rule_rows.cuh"

namespace ps {
namespace {

constexpr int kRing = 3;
constexpr int kFewIds = 10;
static_assert(kHeld == kSumWarps / kPatchWarps, "what a patcher holds fits the summing lanes");
constexpr int kTouched = kHeld * 32;   // one for each lane of the summing warps
constexpr float kLeast = 8.673617379884035e-19f;     // 2^-60

template <int DT>
struct ScoreSmem : RuleSmem<DT, DT == PS_BF16 ? 2 : 1, kRing> {
    uint4 off[8];                                    // a block that does not count
    // processed logits of the first touched ids of each patcher, and how many
    float touched[kRing][kPatchWarps][kTouched];
    int32_t n_touched[kRing][kPatchWarps];
};

static_assert(sizeof(ScoreSmem<PS_BF16>) <= 232448 && sizeof(ScoreSmem<PS_F32>) <= 232448,
              "the shared memory of a block");

__device__ __forceinline__ float warp_max_nan(float m) {
    float d;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(m));
    return d;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 2^(g y) from y and e = 2^y.
template <int NP>
__device__ __forceinline__ float tau_term(float y, float e, float g) {
    if constexpr (NP == 0) return ex2(g * y);
    else if constexpr (NP == 1) return e;
    else if constexpr (NP == 2) return e * e;
    else if constexpr (NP == 4) return (e * e) * (e * e);
    else return ((e * e) * (e * e)) * ((e * e) * (e * e));
}

// Sums relative to a reference, by lane.
struct Sums {
    float s1, st, y1;
};

template <int NP, bool ENT>
__device__ __forceinline__ void add_term(Sums &a, float y, float g) {
    const float e = ex2(y);
    a.s1 += e;
    if constexpr (NP != 1) a.st += tau_term<NP>(y, e, g);
    if constexpr (ENT) a.y1 = fmaf(e, y, a.y1);
}

template <int DT>
__device__ __forceinline__ void pairs_of(uint4 q, float2 *v) {
    if constexpr (DT == PS_BF16) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    } else {
        v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
    }
}

// A lane's ids in a stage: two runs of four vectors (for bfloat16 its two blocks,
// for float32 the halves of its block), read in an order that spreads the lanes
// over the banks, and the bits of the ids that count, in the same order.
struct LaneIds {
    const uint4 *a, *b;
    int first;                  // vector to begin with
    uint32_t ma, mb;            // its bits at the bottom
};

// Calls f(vector, vector) for the lane's pairs of vectors, those of b after those
// of a.  A rolled loop: the eight vectors in one run of code would not fit the
// instruction caches that three kinds of warps share.
template <int DT, bool MASKED, typename F>
__device__ __forceinline__ void each_pair(const LaneIds &l, uint32_t off, F f) {
    constexpr int kBits = DT == PS_BF16 ? 8 : 4;
    int k = l.first;
    uint4 qa = l.a[k], qb = l.b[k];
    uint32_t ma = l.ma, mb = l.mb;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        k = (k + 1) & 3;
        const uint4 na = l.a[k], nb = l.b[k];            // the next ones
        if constexpr (MASKED) {
            qa = masked_by<DT>(qa, ma, off);
            qb = masked_by<DT>(qb, mb, off);
            ma >>= kBits;
            mb >>= kBits;
        }
        f(qa, qb);
        qa = na;
        qb = nb;
    }
}

template <int DT, bool MASKED>
__device__ __forceinline__ float max_of(const LaneIds &l, uint32_t off) {
    if constexpr (DT == PS_BF16) {
        uint32_t m = 0xff80ff80u;
        each_pair<DT, MASKED>(l, off, [&](uint4 a, uint4 b) {
            a.x = max_nan_bf16x2(max_nan_bf16x2(a.x, a.y), max_nan_bf16x2(a.z, a.w));
            b.x = max_nan_bf16x2(max_nan_bf16x2(b.x, b.y), max_nan_bf16x2(b.z, b.w));
            m = max_nan_bf16x2(m, max_nan_bf16x2(a.x, b.x));
        });
        return max_nan_f32(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        float m = -INFINITY;
        each_pair<DT, MASKED>(l, off, [&](uint4 a, uint4 b) {
            const auto top = [](uint4 q) {
                return max_nan_f32(max_nan_f32(__uint_as_float(q.x), __uint_as_float(q.y)),
                                   max_nan_f32(__uint_as_float(q.z), __uint_as_float(q.w)));
            };
            m = max_nan_f32(m, max_nan_f32(top(a), top(b)));
        });
        return m;
    }
}

// Raises -inf to the floor, which keeps 2^y y finite.
template <int DT>
__device__ __forceinline__ uint32_t raised(uint32_t w) {
    if constexpr (DT == PS_BF16) return max_nan_bf16x2(w, kFloorBf16x2);
    else return __float_as_uint(max_nan_f32(__uint_as_float(w), kFloorF32));
}

// The lane's sums.
template <int DT, int NP, bool ENT, bool MASKED>
__device__ __forceinline__ Sums sum_dense(const LaneIds &l, uint32_t off, float ref,
                                          float g, bool raise) {
    constexpr int kPairs = DT == PS_BF16 ? 4 : 2;
    const float2 L2 = make_float2(kLog2e, kLog2e), nR2 = make_float2(-ref, -ref);
    const float2 GL2 = make_float2(g * kLog2e, g * kLog2e), nGR2 = make_float2(-g * ref, -g * ref);
    float2 a1[4], at[4], ay[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a1[j] = at[j] = ay[j] = make_float2(0.f, 0.f);
    each_pair<DT, MASKED>(l, off, [&](uint4 qa, uint4 qb) {
        if (ENT && raise) {
            qa = make_uint4(raised<DT>(qa.x), raised<DT>(qa.y), raised<DT>(qa.z), raised<DT>(qa.w));
            qb = make_uint4(raised<DT>(qb.x), raised<DT>(qb.y), raised<DT>(qb.z), raised<DT>(qb.w));
        }
        float2 v[2 * kPairs];
        pairs_of<DT>(qa, v);
        pairs_of<DT>(qb, v + kPairs);
#pragma unroll
        for (int j = 0; j < 2 * kPairs; ++j) {
            const int c = j & 3;
            const float2 x = __ffma2_rn(v[j], L2, nR2);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            a1[c] = __fadd2_rn(a1[c], e);
            if constexpr (ENT) ay[c] = __ffma2_rn(e, x, ay[c]);
            if constexpr (NP == 0) {
                const float2 z = __ffma2_rn(v[j], GL2, nGR2);
                at[c] = __fadd2_rn(at[c], make_float2(ex2(z.x), ex2(z.y)));
            } else if constexpr (NP != 1) {
                float2 f = e;
                if constexpr (NP >= 4) f = __fmul2_rn(f, f);
                if constexpr (NP >= 8) f = __fmul2_rn(f, f);
                at[c] = __ffma2_rn(f, f, at[c]);
            }
        }
    });
    Sums s;
    s.s1 = hsum4(a1);
    s.st = NP == 1 ? s.s1 : hsum4(at);
    s.y1 = ENT ? hsum4(ay) : 0.f;
    return s;
}

// The patchers' rows: takes the token and the touched ids out of each stage and
// leaves their sums as partial sums of their own.
template <int DT, int NP, bool ENT, typename Smem>
__device__ __forceinline__ void patch_rows(Smem &sm, const ScoreRulesParams &p) {
    constexpr uint32_t kOff = ENT ? Elem<DT>::kFloorWord : Elem<DT>::kNegInfWord;
    const int lane = threadIdx.x & 31;
    const float g = p.rows.g;
    const RuleSpan span(p.r.n_rows, p.cut.n_slices);
    int64_t r = span.t0 % span.rows;
    RuleWalk<Smem> walk(sm, p.r, SliceMap(p.cut, p.r.V, (int32_t)(span.t0 / span.rows)));
    ChunkPart *at = p.parts + (r * p.cut.n_slices + walk.map.slice) * kScoreParts + kSumWarps + walk.wid;
    int s = 0;
    uint32_t lap = 0;
    for (int64_t t = span.t0; t < span.t1; ++t) {
        if (!mbar_wait_bounded(&sm.full[s], lap & 1u, kRuleWaitNs)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        uint8_t *buf = sm.stage[s];
        const int4 dh = *reinterpret_cast<const int4 *>(&sm.desc[s]);       // tok, bad, flags, len
        if ((dh.z & ~kDescMask) && !walk.enter_row(s, dh.z, dh.w)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        const int32_t bad = dh.y | walk.bad;
        const int32_t tok = dh.x;
        const uint32_t *mw = dh.z & kDescMask ? sm.mask[s] : nullptr;
        if (walk.map.slice == 0 && walk.wid == 0 && lane == 0) {
            if (bad) set_status(p.r.status, bad);
            p.row_bad[r] = bad;
        }
        Acc more = acc_empty();                       // ids that find no place in `touched`
        auto put_off = [&](uint32_t d) {
            if constexpr (DT == PS_BF16) reinterpret_cast<uint16_t *>(buf)[d] = (uint16_t)kOff;
            else reinterpret_cast<uint32_t *>(buf)[d] = kOff;
        };
        auto allowed = [&](uint32_t d) { return mw == nullptr || ((mw[d >> 5] >> (d & 31)) & 1u); };
        if (!bad) {
            if (walk.n_list > kListCap)               // then a lane's share may be less than its places
#pragma unroll
                for (int j = 0; j < kHeld; ++j) sm.touched[s][walk.wid][j * 32 + lane] = -INFINITY;
            walk.for_touched([&](int j, uint32_t d, float pos, float neg, float add) {
                float l = load_elem<DT>(buf, d);
                put_off(d);
                l = fmaf(l, l > 0.f ? pos : neg, add);
                if (!allowed(d)) l = -INFINITY;
                if ((int32_t)d == tok) {
                    p.tok_logit[r] = l;
                    l = -INFINITY;
                }
                if (j < kHeld) {
                    sm.touched[s][walk.wid][j * 32 + lane] = l;
                } else if (!(l <= kAbsentBelow)) {
                    const float x = l * kLog2e;
                    if (!(x <= more.R)) more = rebase<NP, ENT>(more, x, g);       // keeps a NaN
                    const float y = x - more.R, e = ex2(y);
                    more.s1 += e;
                    more.st[0] += tau_term<NP>(y, e, g);
                    more.y1 = fmaf(e, y, more.y1);
                }
            });
            if (tok >= 0 && lane == 0 && owner_of(tok) == (uint32_t)walk.wid && !walk.is_seen(tok) &&
                !walk.is_biased(tok)) {
                p.tok_logit[r] = allowed(tok) ? load_elem<DT>(buf, tok) : -INFINITY;
                put_off(tok);
            }
        }
        // ids past the vocabulary in the last block
        if ((walk.map.nid & 31) && walk.wid == 0 && lane >= (walk.map.nid & 31))
            put_off((uint32_t)(walk.map.nid & ~31) + lane);
        const int32_t n_list = bad ? 0 : walk.n_list;
        __syncwarp();
        if (lane == 0) {
            sm.n_touched[s][walk.wid] = n_list <= kListCap ? n_list : -1;
            mbar_arrive(&sm.patched[s]);
        }

        ChunkPart part{-INFINITY, 0.f, 0.f, 0.f};
        if (n_list > kTouched) {
            more = warp_merge<NP, ENT>(more, g);
            part = ChunkPart{more.R, more.s1, more.st[0], more.y1};
            if constexpr (NP == 1) part.st = part.s1;
        }
        if (lane == 0) *at = part;
        at += p.cut.n_slices * kScoreParts;
        if (++s == kRing) {
            s = 0;
            ++lap;
        }
        if (++r == span.rows) {
            r = 0;
            walk.map = SliceMap(p.cut, p.r.V, walk.map.slice + 1);
            at = p.parts + walk.map.slice * kScoreParts + kSumWarps + walk.wid;
        }
    }
}

template <int DT, int NP, bool ENT>
__global__ void __launch_bounds__(rule_threads<kRing>(), 1) score_rules_kernel(
    const __grid_constant__ ScoreRulesParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Smem = ScoreSmem<DT>;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr int kNb = DT == PS_BF16 ? 2 : 1;
    constexpr int kVec = 16 / Smem::kEsz;            // ids of a 16-byte vector
    constexpr int kBv = kBlockIds / kVec;            // vectors of a block: 4 or 8
    // the places of ids that do not count: -inf, or with entropy a large negative
    // value, which keeps 2^y y finite
    constexpr uint32_t kOff = ENT ? Elem<DT>::kFloorWord : Elem<DT>::kNegInfWord;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const float g = p.rows.g;

    if (threadIdx.x < kBv) sm.off[threadIdx.x] = make_uint4(kOff, kOff, kOff, kOff);
    rule_smem_init<Smem, kRing>(sm);
    __syncthreads();

    if (wid >= kFirstProducer) {
        rule_producer<DT, kNb, kRing, false>(sm, p.r, p.cut, p.rows.logits, p.rows.ld_bytes,
                                            p.rows.row_index, p.rows.n_logit_rows,
                                            p.rows.tokens, [](int, int64_t, int32_t) {});
        return;
    }
    if (wid >= kSumWarps) {
        patch_rows<DT, NP, ENT>(sm, p);
        return;
    }

    const RuleSpan span(p.r.n_rows, p.cut.n_slices);
    int64_t r = span.t0 % span.rows;
    int32_t slice = (int32_t)(span.t0 / span.rows);
    int32_t nid = SliceMap(p.cut, p.r.V, slice).nid;
    float ref = 0.f;                                  // the warp's reference
    int s = 0;
    uint32_t lap = 0;
    ChunkPart *part = p.parts + (r * p.cut.n_slices + slice) * kScoreParts + wid;
    const uint32_t first = block_of(wid, lane, 0);
    uint32_t fills = 0;
    for (int64_t t = span.t0; t < span.t1; ++t) {
        bool ok = mbar_wait_bounded(&sm.full[s], lap & 1u, kRuleWaitNs);
        if (ok && (sm.desc[s].flags & kDescRebuild))
            ok = rule_tables(sm, SliceMap(p.cut, p.r.V, slice), sm.rules[s], fills++) != nullptr;
        if (!ok || !mbar_wait_bounded(&sm.patched[s], lap & 1u, kRuleWaitNs)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        const uint8_t *buf = sm.stage[s];
        const bool masked = sm.desc[s].flags & kDescMask;
        uint32_t m[kNb];
        int few = kFewIds + 1;
#pragma unroll
        for (int h = 0; h < kNb; ++h) m[h] = (first + h * 32 * kSumWarps) * kBlockIds < (uint32_t)nid ? 0xffffffffu : 0u;
        if (masked) {
            few = 0;
#pragma unroll
            for (int h = 0; h < kNb; ++h) {
                if (m[h]) m[h] = sm.mask[s][first + h * 32 * kSumWarps];
                few += __popc(m[h]);
            }
            few = __reduce_max_sync(0xffffffffu, few);
        }
        // a touched id's processed logit for this lane (n: -1 means all places are written)
        float px = -INFINITY;
        if ((uint32_t)(wid / kPatchWarps * 32 + lane) < (uint32_t)sm.n_touched[s][wid % kPatchWarps])
            px = sm.touched[s][wid % kPatchWarps][wid / kPatchWarps * 32 + lane];
        // Without mass, as the stage's ids this low are: times log2 e it may leave float32's
        // range, and 2^y y would be 0 * -inf.  Keeps a NaN.
        if (px <= kAbsentBelow) px = -INFINITY;
        Sums sum{0.f, 0.f, 0.f};
        auto join_lanes = [&](Sums a) {
            if (px != -INFINITY) add_term<NP, ENT>(a, fmaf(px, kLog2e, -ref), g);
            if constexpr (NP == 1) a.st = a.s1;
            sum.s1 = warp_sum(a.s1);
            sum.st = NP == 1 ? sum.s1 : warp_sum(a.st);
            if constexpr (ENT) sum.y1 = warp_sum(a.y1);
        };
        auto in_range = [&]() {
            return sum.s1 >= kLeast && sum.s1 <= kLimit && sum.st >= kLeast && sum.st <= kLimit;
        };
        if (few <= kFewIds) {
            // step through the allowed ids of the lane
            auto each = [&](auto f) {
#pragma unroll
                for (int h = 0; h < kNb; ++h)
                    for (uint32_t x = m[h]; x != 0; x &= x - 1)
                        f(load_elem<DT>(buf, (first + h * 32 * kSumWarps) * kBlockIds + __ffs(x) - 1));
            };
            for (bool look = ENT; few > 0 || __any_sync(0xffffffffu, px != -INFINITY);) {
                if (look) {
                    float x = -INFINITY;
                    each([&](float l) { x = max_nan_f32(x, l); });
                    if (x <= kAbsentBelow) x = -INFINITY;
                    x = warp_max_nan(max_nan_f32(x, px));
                    if (x == -INFINITY) {
                        sum = Sums{0.f, 0.f, 0.f};
                        break;
                    }
                    ref = x * kLog2e;
                }
                Sums a{0.f, 0.f, 0.f};
                each([&](float l) {
                    if (!(l <= kAbsentBelow)) add_term<NP, ENT>(a, fmaf(l, kLog2e, -ref), g);
                });
                join_lanes(a);
                if (look || in_range()) break;
                look = true;
            }
        } else {
            LaneIds l;
            const uint4 *v = reinterpret_cast<const uint4 *>(buf);
            l.first = (kNb == 2 ? lane >> 1 : lane) & 3;
            l.a = m[0] ? v + first * kBv : sm.off;
            if constexpr (kNb == 2) {
                l.b = m[1] ? v + (first + 32 * kSumWarps) * kBv : sm.off;
                l.ma = __funnelshift_r(m[0], m[0], 8 * l.first);
                l.mb = __funnelshift_r(m[1], m[1], 8 * l.first);
            } else {
                // a: the half of the block that puts the eight lanes of a bank sweep apart
                const int half = (lane >> 2) & 1;
                l.b = l.a + 4 * (half ^ 1);
                l.a += 4 * half;
                const uint32_t lo = m[0] & 0xffffu, hi = m[0] >> 16;
                const uint32_t x = half ? hi : lo, y = half ? lo : hi;
                l.ma = (x * 0x10001u) >> (4 * l.first);
                l.mb = (y * 0x10001u) >> (4 * l.first);
            }
            // 0: with the reference at hand; 1: with the maximum; 2: with the maximum,
            // and -inf raised (among the logits it makes 2^y y NaN)
            for (int look = ENT;; ++look) {
                if (look == 1) {
                    float x = masked ? max_of<DT, true>(l, kOff) : max_of<DT, false>(l, kOff);
                    if (x <= kAbsentBelow) x = -INFINITY;
                    x = warp_max_nan(max_nan_f32(x, px));
                    if (x == -INFINITY) {             // nothing here
                        sum = Sums{0.f, 0.f, 0.f};
                        break;
                    }
                    ref = x * kLog2e;
                }
                join_lanes(masked ? sum_dense<DT, NP, ENT, true>(l, kOff, ref, g, look == 2)
                                  : sum_dense<DT, NP, ENT, false>(l, kOff, ref, g, look == 2));
                if (ENT ? look == 2 || sum.y1 == sum.y1 || sum.s1 != sum.s1 : look || in_range()) break;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[s]);
        if (lane == 0) *part = ChunkPart{sum.s1 == 0.f ? -INFINITY : ref, sum.s1, sum.st, sum.y1};
        part += p.cut.n_slices * kScoreParts;
        if (++s == kRing) {
            s = 0;
            ++lap;
        }
        if (++r == span.rows) {
            r = 0;
            ++slice;
            if (slice < p.cut.n_slices) nid = SliceMap(p.cut, p.r.V, slice).nid;
            part = p.parts + slice * kScoreParts + wid;
        }
    }
}

// Part `a` relative to reference M >= a.R, and two parts as one.  References of parts with
// like mass can be 124 / g apart, so a factor 2^(g d) alone may be below float32's range
// where the sum times it is not (up to a fourth of a row's mass was lost so): it is applied
// in two halves.
template <int NP, bool ENT>
__device__ __forceinline__ Acc moved(Acc a, float M, float g) {
    if (a.R != -INFINITY) {
        const float d = a.R - M, f = ex2(0.5f * d);
        if constexpr (ENT) a.y1 = fmaf(d, a.s1, a.y1) * f * f;
        a.s1 = a.s1 * f * f;
        if constexpr (NP != 1) {
            const float t = ex2(0.5f * d * (NP == 0 ? g : (float)NP));
            a.st[0] = a.st[0] * t * t;
        }
    }
    a.R = M;
    return a;
}
template <int NP, bool ENT>
__device__ __forceinline__ Acc joined(Acc a, Acc b, float g) {
    const float M = fmaxf(a.R, b.R);
    if (M != -INFINITY) {
        a = moved<NP, ENT>(a, M, g);
        b = moved<NP, ENT>(b, M, g);
    }
    a.s1 += b.s1;
    if constexpr (NP != 1) a.st[0] += b.st[0];
    if constexpr (ENT) a.y1 += b.y1;
    return a;
}

// A row's parts, joined in their order by one warp; the result is in all lanes.
// FAR: parts whose exponentials are 0 next to those of the row's largest logit, under tau
// as well, are left out.
template <int NP, bool ENT, bool FAR>
__device__ __forceinline__ Acc join_parts(const ChunkPart *parts, int n, float tok, float g) {
    const int lane = threadIdx.x & 31;
    float least = -INFINITY;
    if constexpr (FAR) {
        float top = tok * kLog2e;                     // the sums leave the token out
        for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(&parts[i].R));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        least = top - 2048.f / fminf(g, 1.f);
    }
    Acc a = acc_empty();
    for (int i = lane; i < n; i += 32) {
        const float4 s = __ldcg(reinterpret_cast<const float4 *>(parts + i));
        if (FAR && s.x < least) continue;
        a = joined<NP, ENT>(a, Acc{s.x, s.y, {s.z, 0.f, 0.f}, s.w}, g);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Acc b = acc_empty();
        b.R = __shfl_xor_sync(0xffffffffu, a.R, o);
        b.s1 = __shfl_xor_sync(0xffffffffu, a.s1, o);
        if constexpr (NP != 1) b.st[0] = __shfl_xor_sync(0xffffffffu, a.st[0], o);
        if constexpr (ENT) b.y1 = __shfl_xor_sync(0xffffffffu, a.y1, o);
        a = joined<NP, ENT>(a, b, g);
    }
    return a;
}

// One warp a row: its partial sums joined, then the results.  A part of logits like -1e12
// has sums of no meaning (a product's rounding is 2^16 there): they may be infinite, and
// infinity times the 0 that it counts for next to others is NaN.  So sums that are not
// finite are formed again without such parts.
template <int NP, bool ENT>
__global__ void __launch_bounds__(256) score_rules_join_kernel(
    const __grid_constant__ ScoreRulesParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= p.r.n_rows) return;
    pdl_wait_prerequisites();                         // launched while the sums are made
    const bool bad = p.row_bad[r] != 0;
    const float g = p.rows.g, tok = bad ? 0.f : p.tok_logit[r];
    const int n = bad ? 0 : p.cut.n_slices * kScoreParts;
    const ChunkPart *parts = p.parts + r * p.cut.n_slices * kScoreParts;
    Acc a = join_parts<NP, ENT, false>(parts, n, tok, g);
    const bool finite = finite_f(a.s1) && (NP == 1 || finite_f(a.st[0])) && (!ENT || finite_f(a.y1));
    if (__any_sync(0xffffffffu, !finite)) a = join_parts<NP, ENT, true>(parts, n, tok, g);
    if (lane == 0) finalize_row<NP, ENT>(p.rows, r, a, tok, bad);
}

template <int DT, int NP, bool ENT>
cudaError_t launch(const ScoreRulesParams &p, int sms, cudaStream_t stream) {
    const int smem = (int)sizeof(ScoreSmem<DT>);
    cudaError_t e = cudaFuncSetAttribute(score_rules_kernel<DT, NP, ENT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t tasks = p.r.n_rows * p.cut.n_slices;
    score_rules_kernel<DT, NP, ENT>
        <<<(int)(tasks < sms ? tasks : sms), rule_threads<kRing>(), smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.r.n_rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, score_rules_join_kernel<NP, ENT>, p);
}

template <int DT, bool ENT>
cudaError_t launch_np(const ScoreRulesParams &p, int sms, cudaStream_t stream) {
    switch (p.rows.npow) {
        case 1: return launch<DT, 1, ENT>(p, sms, stream);
        case 2: return launch<DT, 2, ENT>(p, sms, stream);
        case 4: return launch<DT, 4, ENT>(p, sms, stream);
        case 8: return launch<DT, 8, ENT>(p, sms, stream);
        default: return launch<DT, 0, ENT>(p, sms, stream);
    }
}

}  // namespace

// As few slices as hold the vocabulary, or where there are few rows as many as
// give every SM a block (of 1024 ids at least).  Segments of a slice (8000 rows of 151936
// bf16 scored without masks and under 24, 150 rows of 50021 float32 with long histories
// processed): none 775, 535 and 115 us, 2: 637, 533 and 86, 9: 608, 546 and 78, all: 614,
// 607 and 76.
// The blocks to cut for are a constant, and not the device's own multiprocessors (152 on a
// GB300), so that a workspace's size depends on V, dtype and n_rows alone.
constexpr int64_t kBlocks = 152;
RuleCut rule_cut(int32_t V, int32_t most, int64_t n_rows) {
    constexpr int64_t kHead = 9;
    int64_t n = kBlocks / (n_rows > 0 ? n_rows : 1);
    if (n > V / 1024) n = V / 1024;
    if (n < 1) n = 1;
    for (;; ++n) {
        RuleCut c;
        const int64_t head = V > kSegIds ? (V / kSegIds - 1) / n : 0;
        c.head = (int32_t)(head < kHead ? head : kHead);
        const int64_t rest = V - n * c.head * kSegIds;           // > 0
        const int64_t run = ((rest + n - 1) / n + 127) / 128 * 128;
        if (c.head * kSegIds + run > most) continue;
        c.run = (int32_t)run;
        // without segments the last slices may hold nothing
        c.n_slices = (int32_t)(c.head ? n : (rest + run - 1) / run);
        return c;
    }
}

static int32_t score_most(int32_t dtype) {
    return dtype == PS_BF16 ? ScoreSmem<PS_BF16>::kIds : ScoreSmem<PS_F32>::kIds;
}

RuleCut score_cut(int32_t V, int32_t dtype, int64_t n_rows) {
    return rule_cut(V, score_most(dtype), n_rows);
}

// A row has as few slices as hold the vocabulary, or so many that all rows together
// have at most kBlocks; the latter would fall as rows are added, the bound rises.
int64_t score_slices(int32_t V, int32_t dtype, int64_t n_rows) {
    const int64_t few = n_rows * (((int64_t)V + score_most(dtype) - 1) / score_most(dtype));
    const int64_t cut = n_rows * (V / 1024);
    const int64_t many = cut < kBlocks ? cut : kBlocks;
    return few > many ? few : many;
}

cudaError_t launch_score_rules(const ScoreRulesParams &p, int sms, cudaStream_t stream) {
    if (p.rows.dtype == PS_BF16)
        return p.rows.entropy ? launch_np<PS_BF16, true>(p, sms, stream)
                              : launch_np<PS_BF16, false>(p, sms, stream);
    return p.rows.entropy ? launch_np<PS_F32, true>(p, sms, stream)
                          : launch_np<PS_F32, false>(p, sms, stream);
}

}  // namespace ps
