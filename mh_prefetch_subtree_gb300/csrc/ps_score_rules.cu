// log p0, log q_tau and entropy of each row's token under rules
// (ps_score_rows_rules), without writing the processed rows.
//
// A block takes one slice of one row: it masks the slice on its way into shared
// memory, takes the token and the ids that penalties or biases touch out of it
// (their places become -inf, their processed float32 values are added on their
// own, so nothing is rounded to the rows' type), and sums the rest.  A second
// kernel joins the slices' sums of each row.
#include "ps_row_sums.cuh"
#include "ps_rules.cuh"

namespace ps {
namespace {

// Adds one processed logit to the running sums.
template <int NP, bool ENT>
__device__ __forceinline__ void add_value(Acc &a, float l, float g) {
    if (l == -INFINITY) return;
    const float x = l * kLog2e;
    if (!(x <= a.R)) a = rebase<NP, ENT>(a, x, g);     // a NaN goes in here and stays
    const float y = x - a.R, e = ex2(y);
    a.s1 += e;
    if constexpr (NP == 0) a.st[0] += ex2(g * y);
    else if constexpr (NP != 1) a.st[0] += ex2((float)NP * y);
    if constexpr (ENT) a.y1 = fmaf(e, y, a.y1);
}

template <int DT, int VPT>
__device__ __forceinline__ float max_of(const uint4 (&q)[VPT]) {
    if constexpr (DT == PS_BF16) {
        uint32_t m = 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            m = max_nan_bf16x2(max_nan_bf16x2(max_nan_bf16x2(m, q[i].x), max_nan_bf16x2(q[i].y, q[i].z)),
                               q[i].w);
        return max_nan_f32(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            m = max_nan_f32(max_nan_f32(max_nan_f32(m, __uint_as_float(q[i].x)),
                                        max_nan_f32(__uint_as_float(q[i].y), __uint_as_float(q[i].z))),
                            __uint_as_float(q[i].w));
        return m;
    }
}

template <int DT, int NP, bool ENT>
__global__ void __launch_bounds__(kRuleThreads) score_rules_kernel(const ScoreRulesParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kEsz = DT == PS_BF16 ? 2 : 4;
    constexpr int kVec = 16 / kEsz;
    constexpr int kVpt = kSliceIds / kVec / kRuleThreads;
    uint4 *stage = reinterpret_cast<uint4 *>(smem);
    uint8_t *stage_b = smem;
    SliceTable &t = *reinterpret_cast<SliceTable *>(smem + kSliceIds * kEsz);
    __shared__ Acc warp_acc[kRuleThreads / 32];
    __shared__ float tok_logit;
    const int tid = threadIdx.x;
    const int32_t V = p.r.V;
    const float g = p.rows.g;
    const int64_t n_tasks = p.r.n_rows * p.n_slices;
    for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
        const int64_t r = task / p.n_slices;
        const int32_t v0 = (int32_t)(task - r * p.n_slices) * kSliceIds;
        const int32_t n = min(kSliceIds, V - v0);
        const int32_t tok = __ldg(p.rows.tokens + r);
        int64_t src_row = p.rows.row_index ? __ldg(p.rows.row_index + r) : r;
        RowRules w = row_rules(p.r, r);
        if (tok < 0 || tok >= V) w.bad |= PS_DEV_BAD_TOKEN;
        if (src_row < 0 || src_row >= p.rows.n_logit_rows) w.bad |= PS_DEV_BAD_ROW_INDEX;
        if (tid == 0) tok_logit = __uint_as_float(kAbsent);
        w.bad |= build_table(t, w, V, v0);
        SlicePart part{};
        if (w.bad) {
            if (tid == 0) {
                if (v0 == 0) set_status(p.r.status, w.bad);
                part.bad = 1;
                p.parts[task] = part;
            }
            __syncthreads();
            continue;
        }
        const uint8_t *src = p.rows.logits + src_row * p.rows.ld_bytes;
        for (int i = tid; i < kSliceIds / kVec; i += blockDim.x) {
            const int32_t v = v0 + i * kVec;
            uint4 q = make_uint4(0, 0, 0, 0);
            uint32_t m = 0;
            if (i * kVec < n) {
                m = mask_bits<kVec>(w.mask, v, V);
                q = *reinterpret_cast<const uint4 *>(src + (int64_t)v * kEsz);
            }
            stage[i] = masked_vec<DT>(q, m);
        }
        __syncthreads();
        Acc acc = acc_empty();
        auto take = [&](uint32_t o, uint32_t count, float bias) {
            const float l = penalised(load_elem<DT>(stage_b, o), count, w) + bias;
            store_elem<DT>(stage_b, o, -INFINITY);
            if (v0 + (int32_t)o == tok) tok_logit = l;
            else add_value<NP, ENT>(acc, l, g);
        };
        for_seen(t, [&](uint32_t o) {
            if (!is_biased(t, o)) take(o, t.count[o], 0.f);
        });
        for (int i = tid; i < w.n_bias; i += blockDim.x) {
            const uint32_t o = (uint32_t)(__ldg(w.bias_ids + i) - v0);
            if (o >= (uint32_t)kSliceIds) continue;
            // a masked id stays -inf whatever its bias
            if (mask_allows(w.mask, v0 + (int32_t)o)) take(o, t.count[o], __ldg(w.bias_values + i));
            else take(o, 0, 0.f);
        }
        const uint32_t to = (uint32_t)(tok - v0);
        if (tid == 0 && to < (uint32_t)kSliceIds && t.count[to] == 0 && !is_biased(t, to)) take(to, 0, 0.f);
        __syncthreads();
        uint4 q[kVpt];
#pragma unroll
        for (int i = 0; i < kVpt; ++i) q[i] = stage[tid + i * kRuleThreads];
        const float m = max_of<DT, kVpt>(q);
        if (m != -INFINITY) {
            Acc b = acc_empty();
            b.R = m * kLog2e;
            float cy;
            sum_vecs<DT, NP, ENT, kVpt>(q, b.R, g, b.s1, b.st, cy);
            b.y1 = cy;
            acc = merge_part<NP, ENT>(acc, b, g);
        }
        acc = warp_merge<NP, ENT>(acc, g);
        if ((tid & 31) == 0) warp_acc[tid >> 5] = acc;
        __syncthreads();
        if (tid < 32) {
            acc = tid < kRuleThreads / 32 ? warp_acc[tid] : acc_empty();
            acc = warp_merge<NP, ENT>(acc, g);
            if (tid == 0) {
                part.R = acc.R;
                part.s1 = acc.s1;
                part.st = acc.st[0];
                part.y1 = acc.y1;
                part.ltok = tok_logit;
                p.parts[task] = part;
            }
        }
        __syncthreads();
    }
}

// One warp a row: its slices' sums joined in slice order, then the results.
template <int NP, bool ENT>
__global__ void __launch_bounds__(kRuleThreads) score_rules_join_kernel(const ScoreRulesParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * (kRuleThreads / 32) + (threadIdx.x >> 5);
    if (r >= p.r.n_rows) return;
    Acc a = acc_empty();
    float lt = __uint_as_float(kAbsent);
    bool bad = false;
    for (int i = lane; i < p.n_slices; i += 32) {
        const SlicePart s = p.parts[r * p.n_slices + i];
        bad |= s.bad != 0;
        if (bad) continue;
        a = merge_part<NP, ENT>(a, Acc{s.R, s.s1, {s.st, 0.f, 0.f}, s.y1}, p.rows.g);
        if (__float_as_uint(s.ltok) != kAbsent) lt = s.ltok;
    }
    bad = __any_sync(0xffffffffu, bad);
    a = warp_merge<NP, ENT>(a, p.rows.g);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, lt, o);
        if (__float_as_uint(lt) == kAbsent) lt = other;
    }
    if (lane == 0) finalize_row<NP, ENT>(p.rows, r, a, lt, bad);
}

template <int DT, int NP, bool ENT>
cudaError_t launch(const ScoreRulesParams &p, int sms, cudaStream_t stream) {
    const int smem = (int)sizeof(SliceTable) + kSliceIds * (DT == PS_BF16 ? 2 : 4);
    cudaError_t e = cudaFuncSetAttribute(score_rules_kernel<DT, NP, ENT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t tasks = p.r.n_rows * p.n_slices, most = (int64_t)sms * 3;
    score_rules_kernel<DT, NP, ENT>
        <<<(int)(tasks < most ? tasks : most), kRuleThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t per = kRuleThreads / 32;
    score_rules_join_kernel<NP, ENT>
        <<<(int)((p.r.n_rows + per - 1) / per), kRuleThreads, 0, stream>>>(p);
    return cudaGetLastError();
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

cudaError_t launch_score_rules(const ScoreRulesParams &p, int sms, cudaStream_t stream) {
    if (p.rows.dtype == PS_BF16)
        return p.rows.entropy ? launch_np<PS_BF16, true>(p, sms, stream)
                              : launch_np<PS_BF16, false>(p, sms, stream);
    return p.rows.entropy ? launch_np<PS_F32, true>(p, sms, stream)
                          : launch_np<PS_F32, false>(p, sms, stream);
}

}  // namespace ps
