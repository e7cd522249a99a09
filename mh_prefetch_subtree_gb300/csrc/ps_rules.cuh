// Rules on logits rows (penalties, biases, masks): what the kernels that apply
// them share.  include/ps.h states the rules.
#pragma once

#include "ps_internal.cuh"

namespace ps {

struct RulesParams {
    ps_logit_rules rules;       // device pointers
    int64_t n_rows;
    int32_t V;
    int32_t *status;
};

struct ProcessParams {
    RulesParams r;
    const uint8_t *logits;
    uint8_t *out;               // may be logits itself
    int64_t ld_bytes;
    int64_t out_ld_bytes;
};

// How the vocabulary is cut for the kernels that stream rows.  A slice has `head`
// segments of kSegIds ids, which are dealt to the slices in turn from the first id on,
// and a run of the ids after those.
constexpr int32_t kSegIds = 1024;
struct RuleCut {
    int32_t n_slices;
    int32_t head;               // segments of a slice
    int32_t run;                // ids of a run, a multiple of 128
};
// most: ids of a slice at most (a multiple of kSegIds).
RuleCut rule_cut(int32_t V, int32_t most, int64_t n_rows);
RuleCut score_cut(int32_t V, int32_t dtype, int64_t n_rows);
// The slices of all rows together, of any batch of up to n_rows rows.
int64_t score_slices(int32_t V, int32_t dtype, int64_t n_rows);
constexpr int kScoreParts = 16;     // partial sums of a slice of a row: one a warp

// Sums of one warp's ids of a slice (ps_row_sums.cuh has their meaning).
struct __align__(16) ChunkPart {
    float R, s1, st, y1;
};

struct ScoreRulesParams {
    RulesParams r;
    RowsParams rows;            // logits, tokens, row_index, outputs, tau
    RuleCut cut;
    ChunkPart *parts;           // [n_rows][n_slices][kScoreParts]
    float *tok_logit;           // [n_rows] the token's processed logit
    int32_t *row_bad;           // [n_rows] status bits
};

cudaError_t launch_process_rows(const ProcessParams &p, int32_t dtype, int sms,
                                cudaStream_t stream);
cudaError_t launch_score_rules(const ScoreRulesParams &p, int sms, cudaStream_t stream);

#ifdef __CUDACC__
namespace {

constexpr int kSliceIds = 8192;
constexpr uint32_t kSeen = 0x80000000u;      // count word: the id was seen
constexpr int kTableThreads = 256;

// What row r's rules are, read and checked.
struct RowRules {
    const int32_t *hist;        // its history
    const int32_t *bias_ids;
    const float *bias_values;
    const uint32_t *mask;       // its mask row, or nullptr
    int32_t len;                // tokens of history
    int32_t len_all;            // tokens of its sequence
    int32_t prompt;             // the first of them that were not generated
    int32_t n_bias;
    float rho, freq, pres;
    int32_t bad;                // status bits; the row gets NaN when they are not 0
};

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) < INFINITY; }

__device__ __forceinline__ RowRules row_rules(const RulesParams &p, int64_t r) {
    const ps_logit_rules &u = p.rules;
    RowRules o{};
    o.rho = 1.f;
    const bool per_seq = u.seq_begin != nullptr || u.bias_begin != nullptr;
    if (per_seq) {
        const int64_t s = u.row_seq ? (int64_t)__ldg(u.row_seq + r) : r;
        if (s < 0 || s >= u.n_seqs) {
            o.bad |= PS_DEV_BAD_RULES;
        } else {
            if (u.seq_begin) {
                const int64_t b = __ldg(u.seq_begin + s), e = __ldg(u.seq_begin + s + 1);
                const int64_t n = u.row_len ? (int64_t)__ldg(u.row_len + r) : e - b;
                if (b < 0 || e < b || e > u.n_tokens || n < 0 || n > e - b || e - b > 0x7fffffff) {
                    o.bad |= PS_DEV_BAD_RULES;
                } else {
                    o.hist = u.seq_tokens + b;
                    o.len = (int32_t)n;
                    o.len_all = (int32_t)(e - b);
                    o.prompt = u.seq_prompt ? __ldg(u.seq_prompt + s) : 0;
                }
                if (u.repetition) o.rho = __ldg(u.repetition + s);
                if (u.frequency) o.freq = __ldg(u.frequency + s);
                if (u.presence) o.pres = __ldg(u.presence + s);
                if (!(o.rho > 0.f) || !finite_f(o.rho) || !finite_f(o.freq) || !finite_f(o.pres))
                    o.bad |= PS_DEV_BAD_RULES;
            }
            if (u.bias_begin) {
                const int64_t b = __ldg(u.bias_begin + s), e = __ldg(u.bias_begin + s + 1);
                if (b < 0 || e < b || e > u.n_bias || e - b > 0x7fffffff) {
                    o.bad |= PS_DEV_BAD_RULES;
                } else {
                    o.bias_ids = u.bias_ids + b;
                    o.bias_values = u.bias_values + b;
                    o.n_bias = (int32_t)(e - b);
                }
            }
        }
    }
    if (u.mask) {
        const int64_t m = u.row_mask ? (int64_t)__ldg(u.row_mask + r) : r;
        if (m < (u.row_mask ? -1 : 0) || m >= u.n_masks) o.bad |= PS_DEV_BAD_RULES;
        else if (m >= 0) o.mask = u.mask + m * u.mask_ld;
    }
    return o;
}

// The ids of slice [v0, v0 + kSliceIds) that penalties or biases touch.
struct SliceTable {
    uint32_t count[kSliceIds];         // times generated, and kSeen
    uint32_t biased[kSliceIds / 32];   // bit: in the sequence's bias list
    // Bit b of word w: id v0 + w + kTableThreads b was seen.  Thread w takes word
    // w's ids, so which thread takes an id does not depend on timing (a list in
    // order of arrival would change the order of float sums), and neighbouring
    // ids, which common tokens often are, go to different threads.
    uint32_t seen[kTableThreads];
};
static_assert(kSliceIds == 32 * kTableThreads, "one word of seen ids per thread");

// Fills `t` for one row; ends with a barrier.  Returns the status bits of the
// whole history and bias list (the same in every thread).
__device__ int32_t build_table(SliceTable &t, const RowRules &w, int32_t V, int32_t v0) {
    const int tid = threadIdx.x;
    for (int i = tid; i < kSliceIds / 4; i += blockDim.x)
        reinterpret_cast<uint4 *>(t.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kSliceIds / 32; i += blockDim.x) t.biased[i] = 0;
    t.seen[tid] = 0;
    __syncthreads();
    int bad_tok = 0, bad_bias = 0;
    // unsigned: a step past the last of 2^31 - 1 tokens has to end the loop
    for (uint32_t i = tid; i < (uint32_t)w.len; i += blockDim.x) {
        const int32_t id = __ldg(w.hist + i);
        if (id < 0 || id >= V) {
            bad_tok = 1;
            continue;
        }
        const uint32_t o = (uint32_t)(id - v0);
        if (o >= (uint32_t)kSliceIds) continue;
        atomicOr(&t.count[o], kSeen);
        atomicOr(&t.seen[o % kTableThreads], 1u << (o / kTableThreads));
        if ((int32_t)i >= w.prompt) atomicAdd(&t.count[o], 1u);
    }
    for (uint32_t i = tid; i < (uint32_t)w.n_bias; i += blockDim.x) {
        const int32_t id = __ldg(w.bias_ids + i);
        if (id < 0 || id >= V || (i > 0 && id <= __ldg(w.bias_ids + i - 1))) {
            bad_bias = 1;
            continue;
        }
        const uint32_t o = (uint32_t)(id - v0);
        if (o < (uint32_t)kSliceIds) atomicOr(&t.biased[o >> 5], 1u << (o & 31));
    }
    bad_tok = __syncthreads_or(bad_tok);
    bad_bias = __syncthreads_or(bad_bias);
    return (bad_tok ? PS_DEV_BAD_TOKEN : 0) | (bad_bias ? PS_DEV_BAD_RULES : 0);
}

// Calls f(o) for the seen ids v0 + o that are this thread's.
template <typename F>
__device__ __forceinline__ void for_seen(const SliceTable &t, F f) {
    for (uint32_t w = t.seen[threadIdx.x]; w != 0; w &= w - 1)
        f(threadIdx.x + kTableThreads * (uint32_t)(__ffs(w) - 1));
}

__device__ __forceinline__ bool is_biased(const SliceTable &t, uint32_t o) {
    return (t.biased[o >> 5] >> (o & 31)) & 1u;
}

// The processed logit of an id with count word c, in the order of operations of
// the kernels that stream rows: a factor by sign, then one summand.
__device__ __forceinline__ float penalised(float l, uint32_t c, const RowRules &w, float bias) {
    const uint32_t n = c & ~kSeen;
    float f = 1.f;
    if (c & kSeen) f = l > 0.f ? 1.f / w.rho : w.rho;
    return fmaf(l, f, bias - (w.freq * (float)n + (n ? w.pres : 0.f)));
}

__device__ __forceinline__ bool mask_allows(const uint32_t *mask, int32_t v) {
    return mask == nullptr || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u);
}

// Mask bits of the n ids from v on (n = 8 or 4, v a multiple of n), those from
// V on off.
template <int N>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *mask, int32_t v, int32_t V) {
    uint32_t m = (1u << N) - 1u;
    if (mask) m &= __ldg(mask + (v >> 5)) >> (v & 31);
    if (v + N > V) m &= (1u << (V - v)) - 1u;
    return m;
}

// One 16-byte vector of logits with the ids whose bit is 0 set to -inf.
__device__ __forceinline__ uint4 masked_bf16(uint4 q, uint32_t m) {
    if (m == 0xffu) return q;
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (!((m >> (2 * j)) & 1u)) w[j] = (w[j] & 0xffff0000u) | 0xff80u;
        if (!((m >> (2 * j + 1)) & 1u)) w[j] = (w[j] & 0xffffu) | 0xff800000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 masked_f32(uint4 q, uint32_t m) {
    if (!(m & 1u)) q.x = 0xff800000u;
    if (!(m & 2u)) q.y = 0xff800000u;
    if (!(m & 4u)) q.z = 0xff800000u;
    if (!(m & 8u)) q.w = 0xff800000u;
    return q;
}

template <int DT>
__device__ __forceinline__ uint4 masked_vec(uint4 q, uint32_t m) {
    if constexpr (DT == PS_BF16) return masked_bf16(q, m);
    else return masked_f32(q, m);
}

template <int DT>
__device__ __forceinline__ float load_elem(const uint8_t *row, int64_t i) {
    if constexpr (DT == PS_BF16)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[i] << 16);
    else
        return reinterpret_cast<const float *>(row)[i];
}

template <int DT>
__device__ __forceinline__ void store_elem(uint8_t *row, int64_t i, float x) {
    if constexpr (DT == PS_BF16) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
        reinterpret_cast<uint16_t *>(row)[i] = h;
    } else {
        reinterpret_cast<float *>(row)[i] = x;
    }
}

}  // namespace
#endif  // __CUDACC__
}  // namespace ps
