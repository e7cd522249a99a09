// Streaming rows under rules: the part that ps_process.cu and ps_score_rules.cu
// share.
//
// A block owns a slice of the vocabulary and walks down the rows, so that
// consecutive positions of a sequence, which differ by one token of history,
// reuse what is known about the row before.  One producer warp reads the rows'
// entries ahead, says in a descriptor what changes from row to row, and fills a
// ring of stages: the slice of the row's logits (bulk copies) and of its mask.
// 16 consumer warps work on the stage.
//
// Which warp takes which ids.  The slice is cut into blocks of 32 ids (one mask
// word), dealt to the warps in turn: ids of common tokens lie close together, so
// a warp that owned a long run of ids could hold most of a history (measured: 4.9
// ms instead of 1.1 for 8000 rows of 151936 with such histories).  Lane l of warp
// w owns blocks h 512 + 16 l + (w + l) % 16 (h = 0, 1, ...); the skew puts the
// lanes' vectors in different banks.
//
// What a warp knows of its ids is in shared memory: how often each was generated
// (16 bits), bit sets of the seen and the biased ones, and a list of both while it
// is short.  A new token costs a few instructions in the one warp that owns it.
// Where the sequence changes, the consumers read the whole history together.
#pragma once

#include "ps_row_sums.cuh"
#include "ps_rules.cuh"

namespace ps {
namespace {

constexpr int kRuleWarps = 16;                       // consumers
constexpr int kListCap = 128;                        // touched ids of a warp kept as a list
constexpr uint32_t kCountFull = 0xffffu;             // a count that no longer fits
constexpr int64_t kNoSeq = INT64_MIN;
constexpr int kMaxNew = 6;                           // new tokens of a row handed on one by one
constexpr uint64_t kRuleWaitNs = 4000000000ull;      // 4 s: a copy, or the other warps
constexpr uint64_t kRuleDrainNs = 1000000000ull;
constexpr int kBlockIds = 32;

// What the producer tells about one row.
struct __align__(16) RowDesc {
    int32_t tok;                // the scored token, from the slice's start (or < 0, or past it)
    int32_t bad;                // status bits so far
    int32_t flags;              // kDesc*
    int32_t n_new;
    int32_t fresh[kMaxNew];     // new tokens from the slice's start, or -1; kMade set: generated
    int32_t pad[2];
};
constexpr int32_t kDescRebuild = 1, kDescMask = 2, kDescSparse = 4;
constexpr int32_t kMade = 0x40000000;

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared memory of a block.  NB: blocks of 32 ids per lane; RING: stages.
template <int DT, int NB, int RING>
struct RuleSmem {
    static constexpr int kEsz = DT == PS_BF16 ? 2 : 4;
    static constexpr int kIds = kRuleWarps * 32 * NB * kBlockIds;     // of a slice, at most
    static constexpr int kWarpIds = kIds / kRuleWarps;
    uint8_t stage[RING][kIds * kEsz];
    uint32_t mask[RING][kIds / 32];
    uint16_t count[kRuleWarps][kWarpIds];
    uint32_t seen[kRuleWarps][kWarpIds / 32];
    uint32_t biased[kRuleWarps][kWarpIds / 32];
    uint16_t list[kRuleWarps][kListCap];             // ids from the slice's start
    float list_bias[kRuleWarps][kListCap];
    RowDesc desc[RING];
    RowRules rules[RING];
    uint64_t full[RING], empty[RING], free[RING];
    uint64_t sync;                                   // the consumers' own barrier
    int32_t bad[2];                                  // of a rebuild, by its parity
};

// Where id d of the slice belongs.
__device__ __forceinline__ uint32_t owner_of(uint32_t d) {
    const uint32_t b = d / kBlockIds, rem = b % 512;
    return (rem - rem / 16) & 15u;
}
__device__ __forceinline__ uint32_t place_of(uint32_t d) {            // among the owner's ids
    const uint32_t b = d / kBlockIds;
    return ((b / 512) * 32 + (b % 512) / 16) * kBlockIds + d % kBlockIds;
}
// The lane's block h in the slice.
__device__ __forceinline__ uint32_t block_of(int wid, int lane, int h) {
    return h * 512 + lane * 16 + ((wid + lane) & 15);
}

// Times that id is among tokens b .. e - 1.
__device__ __noinline__ uint32_t recount(const int32_t *hist, int32_t b, int32_t e, int32_t id) {
    uint32_t c = 0;
    for (int32_t i = b; i < e; ++i) c += __ldg(hist + i) == id;
    return c;
}

// The bias of id in a rising list; 0 if it is not there.
__device__ __noinline__ float bias_of(const int32_t *ids, const float *values, int32_t n, int32_t id) {
    int32_t lo = 0, hi = n;
    while (lo < hi) {
        const int32_t m = (lo + hi) / 2;
        if (__ldg(ids + m) < id) lo = m + 1;
        else hi = m;
    }
    return lo < n && __ldg(ids + lo) == id ? __ldg(values + lo) : 0.f;
}

// The order of a block's work: slice by slice, in each all rows.
struct RuleSpan {
    int64_t t0, t1, rows;
    __device__ RuleSpan(int64_t n_rows, int32_t n_slices) : rows(n_rows) {
        const int64_t total = n_rows * n_slices;
        t0 = total * blockIdx.x / gridDim.x;
        t1 = total * (blockIdx.x + 1) / gridDim.x;
    }
};

// The producer warp.  Sink: issues the copies of one row.
// SPARSE: where a row's mask leaves few of the slice's ids, only the 16-byte
// vectors that hold one are copied.
template <int DT, int NB, int RING, bool SPARSE>
__device__ __forceinline__ void rule_producer(RuleSmem<DT, NB, RING> &sm, const RulesParams &p,
                                              const RuleCut &cut, const uint8_t *logits,
                                              int64_t ld_bytes, int64_t row_bytes,
                                              const int64_t *row_index, int64_t n_logit_rows,
                                              const int32_t *tokens, uint64_t *free_bars) {
    using Smem = RuleSmem<DT, NB, RING>;
    constexpr int kEsz = Smem::kEsz;
    constexpr int kWords = Smem::kIds / 32;                // mask words of a slice
    constexpr int kWpl = kWords / 32;                      // and of a lane
    const ps_logit_rules &u = p.rules;
    const int lane = threadIdx.x & 31;
    const RuleSpan span(p.n_rows, cut.n_slices);
    const uint64_t policy = l2_evict_first_policy();
    const bool per_seq = u.seq_begin != nullptr || u.bias_begin != nullptr;
    const bool mask16 = u.mask && u.mask_ld % 4 == 0 && (reinterpret_cast<uintptr_t>(u.mask) & 15) == 0;

    // entries of 32 rows, one a lane
    int64_t base = -1;
    int32_t c_seq = 0, c_len = 0, c_mask = -1, c_tok = 0;
    int64_t c_src = 0;
    // the sequence that the consumers know
    int64_t seq = kNoSeq;
    int32_t len = 0, win = 0, win_tok = 0, bad_hist = 0;
    RowRules w{};

    int64_t r = span.t0 % span.rows;
    int32_t slice = (int32_t)(span.t0 / span.rows);
    uint32_t m[kWpl];                                      // the row's mask words, by lane
    int s = 0;
    uint32_t lap = 0;
    int64_t t = span.t0;
    for (; t < span.t1; ++t) {
        if (base < 0 || r < base || r >= base + 32) {
            base = r;
            const int64_t i = r + lane;
            const bool in = i < p.n_rows;
            c_seq = (in && per_seq && u.row_seq) ? __ldg(u.row_seq + i) : 0;
            c_len = (in && u.seq_begin && u.row_len) ? __ldg(u.row_len + i) : 0;
            c_mask = (in && u.mask && u.row_mask) ? __ldg(u.row_mask + i) : -1;
            c_tok = (in && tokens) ? __ldg(tokens + i) : 0;
            c_src = (in && row_index) ? __ldg(row_index + i) : i;
        }
        const int k = (int)(r - base);
        const int32_t s0 = slice * cut.ids;
        const int32_t nid = min(cut.ids, p.V - s0);        // ids of the slice
        int32_t bad = 0, flags = 0;
        const int64_t rm = u.row_mask ? (int64_t)__shfl_sync(0xffffffffu, c_mask, k) : r;
        if (u.mask) {
            if (rm < (u.row_mask ? -1 : 0) || rm >= u.n_masks) bad |= PS_DEV_BAD_RULES;
            else if (rm >= 0) flags |= kDescMask;
        }
        int64_t src = __shfl_sync(0xffffffffu, c_src, k);
        if (row_index && (src < 0 || src >= n_logit_rows)) {
            bad |= PS_DEV_BAD_ROW_INDEX;
            src = 0;
        }
        const int32_t tok = __shfl_sync(0xffffffffu, c_tok, k);
        if (tokens && (tok < 0 || tok >= p.V)) bad |= PS_DEV_BAD_TOKEN;

        if (lap > 0 && !mbar_wait_bounded(&free_bars[s], (lap - 1) & 1u, kRuleWaitNs)) {
            if (lane == 0) set_status(p.status, PS_DEV_TIMEOUT);
            break;
        }
        // logits and mask
        const int64_t off = (int64_t)s0 * kEsz;
        const uint32_t bytes = (uint32_t)min(((int64_t)nid * kEsz + 15) / 16 * 16, row_bytes - off);
        const uint8_t *from = logits + src * ld_bytes + off;
        int32_t left = 0;                                  // vectors that hold an allowed id
        if (flags & kDescMask) {
            const uint32_t *mrow = u.mask + rm * u.mask_ld + s0 / 32;
            const int32_t nw = (nid + 31) / 32;
            if (mask16) {
#pragma unroll
                for (int i = 0; i < kWpl; i += 4) {
                    const int at = i * 32 + lane * 4;
                    uint4 q = make_uint4(0, 0, 0, 0);
                    if (at < nw) q = __ldg(reinterpret_cast<const uint4 *>(mrow + at));
                    m[i] = q.x;
                    m[i + 1] = q.y;
                    m[i + 2] = q.z;
                    m[i + 3] = q.w;
                    reinterpret_cast<uint4 *>(sm.mask[s])[at / 4] = q;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kWpl; ++i) {
                    const int at = (i & ~3) * 32 + lane * 4 + (i & 3);
                    m[i] = at < nw ? __ldg(mrow + at) : 0u;
                    sm.mask[s][at] = m[i];
                }
            }
            if constexpr (SPARSE) {
#pragma unroll
                for (int i = 0; i < kWpl; ++i) {
                    const int at = (i & ~3) * 32 + lane * 4 + (i & 3);
                    uint32_t x = m[i];
                    if (at * 32 + 32 > nid) x &= at * 32 < nid ? (1u << (nid - at * 32)) - 1u : 0u;
                    // one bit for each vector
                    if constexpr (DT == PS_BF16) {
                        x |= x >> 4;
                        x |= x >> 2;
                        x |= x >> 1;
                        x &= 0x01010101u;
                    } else {
                        x |= x >> 2;
                        x |= x >> 1;
                        x &= 0x11111111u;
                    }
                    m[i] = x;
                    left += __popc(x);
                }
                left = __reduce_add_sync(0xffffffffu, left);
                if (left * 16 * 8 <= (int32_t)bytes) flags |= kDescSparse;
            }
        }
        if (lane == 0) {
            fence_proxy_async_smem();
            if (flags & kDescSparse) {
                if (left) asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                                           smem_addr(&sm.full[s])), "r"(left * 16) : "memory");
            } else {
                asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                                 smem_addr(&sm.full[s])), "r"(bytes) : "memory");
                bulk_g2s(sm.stage[s], from, bytes, &sm.full[s], policy);
            }
        }
        __syncwarp();
        if (SPARSE && (flags & kDescSparse)) {
            fence_proxy_async_smem();
#pragma unroll
            for (int i = 0; i < kWpl; ++i) {
                const int at = (i & ~3) * 32 + lane * 4 + (i & 3);
                for (uint32_t x = m[i]; x; x &= x - 1) {
                    const uint32_t o = (uint32_t)(at * 32 + (__ffs(x) - 1)) * kEsz;   // of the vector
                    bulk_g2s(sm.stage[s] + o, from + o, 16, &sm.full[s], policy);
                }
            }
        }
        // what changed since the row before
        const int64_t q = per_seq && !u.row_seq ? r : (int64_t)__shfl_sync(0xffffffffu, c_seq, k);
        int32_t n = __shfl_sync(0xffffffffu, c_len, k), n_new = 0;
        bool again = true;
        if (q == seq) {
            if (!u.row_len || !u.seq_begin) n = len;
            if (n > w.len_all) {                           // only this row is wrong
                bad |= PS_DEV_BAD_RULES;
                again = false;
            } else if (n >= len && n - len <= kMaxNew) {
                again = false;
                n_new = n - len;
                for (int j = 0; j < n_new; ++j, ++len) {
                    if (len < win || len >= win + 32) {
                        win = len;
                        win_tok = win + lane < w.len_all ? __ldg(w.hist + win + lane) : 0;
                    }
                    const int32_t id = __shfl_sync(0xffffffffu, win_tok, len - win);
                    int32_t d = -1;
                    if (id < 0 || id >= p.V) bad_hist |= PS_DEV_BAD_TOKEN;
                    else if (id >= s0 && id - s0 < nid) d = (id - s0) | (len >= w.prompt ? kMade : 0);
                    if (lane == 0) sm.desc[s].fresh[j] = d;
                }
            }
        }
        if (again) {
            w = row_rules(p, r);
            // a row that fails a check says nothing about the next one
            seq = w.bad ? kNoSeq : q;
            len = w.len;
            win = -64;
            bad_hist = 0;
            flags |= kDescRebuild;
            if (lane == 0) sm.rules[s] = w;
        }
        if (lane == 0) {
            RowDesc &d = sm.desc[s];
            d.tok = tok - s0;
            d.bad = bad | bad_hist | w.bad;
            d.flags = flags;
            d.n_new = n_new;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
        if (++s == RING) {
            s = 0;
            ++lap;
        }
        if (++r == span.rows) {
            r = 0;
            ++slice;
            seq = kNoSeq;
            base = -1;
        }
    }
    // copies in flight land before the block's memory goes
    const int64_t issued = t - span.t0;
    for (int64_t j = max(issued - RING, (int64_t)0); j < issued; ++j)
        mbar_wait_bounded(&sm.full[j % RING], (uint32_t)(j / RING) & 1u, kRuleDrainNs);
}

// A consumer warp's view of the rules.  The same in all lanes unless said
// otherwise.
template <typename Smem>
struct RuleWalk {
    Smem &sm;
    const RulesParams &p;
    const int lane, wid;
    int32_t s0 = 0;             // first id of the slice
    int32_t nid = 0;            // ids of the slice
    int32_t len = 0;            // tokens of history that are counted
    int32_t n_list = 0;         // touched ids; the first n_bias of the list are biased
    int32_t n_bias = 0;
    int32_t bad = 0;            // status bits of the history and the biases
    uint32_t lap = 0;           // of the consumers' own barrier: two a rebuild
    RowRules w{};
    float inv_rho = 1.f;
    // by lane: entry `lane` of the list, -1 if there is none
    int32_t e_id = -1;
    float e_pos = 1.f, e_neg = 1.f, e_add = 0.f;

    __device__ RuleWalk(Smem &sm_, const RulesParams &p_)
        : sm(sm_), p(p_), lane(threadIdx.x & 31), wid(threadIdx.x >> 5) {}

    __device__ __forceinline__ void enter_slice(int32_t slice, const RuleCut &cut) {
        s0 = slice * cut.ids;
        nid = min(cut.ids, p.V - s0);
    }
    __device__ __forceinline__ bool is_seen(uint32_t d) const {
        const uint32_t o = place_of(d);
        return (sm.seen[wid][o >> 5] >> (o & 31)) & 1u;
    }
    __device__ __forceinline__ bool is_biased(uint32_t d) const {
        const uint32_t o = place_of(d);
        return (sm.biased[wid][o >> 5] >> (o & 31)) & 1u;
    }
    // Waits for the other consumers; false when they do not come.
    __device__ __forceinline__ bool meet() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sync);
        const bool ok = mbar_wait_bounded(&sm.sync, lap & 1u, kRuleWaitNs);
        ++lap;
        return ok;
    }

    // How often id d was generated.  A count that does not fit 16 bits is taken
    // again from the history: slow, and as rare as a token that one sequence holds
    // 65535 times.
    __device__ __forceinline__ uint32_t times(uint32_t d) const {
        const uint32_t c = sm.count[wid][place_of(d)];
        return c == kCountFull ? recount(w.hist, max(0, w.prompt), len, s0 + (int32_t)d) : c;
    }

    // The processed logit of id d from its logit: a factor by sign, then a sum that
    // does not depend on the logit.
    __device__ __forceinline__ float summand(uint32_t d, float bias) const {
        const uint32_t n = times(d);
        return bias - (w.freq * (float)n + (n ? w.pres : 0.f));
    }

    __device__ __forceinline__ void load_entry() {
        e_id = -1;
        if (n_list <= kListCap && lane < n_list) {
            e_id = sm.list[wid][lane];
            const bool seen = is_seen(e_id);
            e_pos = seen ? inv_rho : 1.f;
            e_neg = seen ? w.rho : 1.f;
            e_add = summand(e_id, lane < n_bias ? sm.list_bias[wid][lane] : 0.f);
        }
    }

    __device__ __forceinline__ void count_shared(int32_t i, int32_t id, bool fits) {
        if (id < 0 || id >= p.V) {
            atomicOr(&sm.bad[(lap >> 1) & 1], PS_DEV_BAD_TOKEN);
            return;
        }
        const uint32_t d = (uint32_t)(id - s0);
        if (d >= (uint32_t)nid) return;
        const uint32_t q = owner_of(d), o = place_of(d);
        atomicOr(&sm.seen[q][o >> 5], 1u << (o & 31));
        if (i < w.prompt) return;
        uint32_t *word = reinterpret_cast<uint32_t *>(&sm.count[q][o & ~1u]);
        const int sh = (o & 1) * 16;
        if (fits) {
            atomicAdd(word, 1u << sh);
        } else {
            uint32_t old = *reinterpret_cast<volatile uint32_t *>(word), was;
            do {
                was = old;
                if (((was >> sh) & 0xffffu) == kCountFull) break;
                old = atomicCAS(word, was, was + (1u << sh));
            } while (old != was);
        }
    }

    // Takes up a row's sequence with its history so far.  False on a timeout.
    __device__ __forceinline__ bool rebuild(const RowRules &from) {
        w = from;
        inv_rho = 1.f / w.rho;
        len = w.len;
        // the warp's own ids (blocks past the slice are never touched)
        const int32_t blocks = (nid + kBlockIds - 1) / kBlockIds;
        for (int h = 0; h * 512 < blocks; ++h) {
            const int nl = min(32, (blocks - h * 512 + 15) / 16);      // lanes that own one
            for (int i = lane; i < nl * kBlockIds / 8; i += 32)
                reinterpret_cast<uint4 *>(sm.count[wid])[h * 128 + i] = make_uint4(0, 0, 0, 0);
            sm.seen[wid][h * 32 + lane] = sm.biased[wid][h * 32 + lane] = 0;
        }
        // a warp may still read the word of the rebuild before
        int32_t *bad_word = &sm.bad[(lap >> 1) & 1];
        if (threadIdx.x == 0) *bad_word = 0;
        if (!meet()) return false;
        const bool fits = w.len - max(0, min(w.prompt, w.len)) < (int32_t)kCountFull;
        for (int i = threadIdx.x; i < w.len; i += kRuleWarps * 32) count_shared(i, __ldg(w.hist + i), fits);
        for (int i = threadIdx.x; i < w.n_bias; i += kRuleWarps * 32) {
            const int32_t id = __ldg(w.bias_ids + i);
            if (id < 0 || id >= p.V || (i > 0 && id <= __ldg(w.bias_ids + i - 1))) {
                atomicOr(&sm.bad[(lap >> 1) & 1], PS_DEV_BAD_RULES);
                continue;
            }
            const uint32_t d = (uint32_t)(id - s0);
            if (d >= (uint32_t)nid) continue;
            const uint32_t o = place_of(d);
            atomicOr(&sm.biased[owner_of(d)][o >> 5], 1u << (o & 31));
        }
        if (!meet()) return false;
        bad = *reinterpret_cast<volatile int32_t *>(bad_word);
        // the list: the biased ids in the order of their list, then the others seen
        n_list = 0;
        for (int b = 0; bad == 0 && b < w.n_bias; b += 32) {
            const int32_t id = b + lane < w.n_bias ? __ldg(w.bias_ids + b + lane) : -1;
            const uint32_t d = (uint32_t)(id - s0);
            const bool mine = id >= 0 && d < (uint32_t)nid && owner_of(d) == (uint32_t)wid;
            const uint32_t all = __ballot_sync(0xffffffffu, mine);
            const int32_t at = n_list + __popc(all & ((1u << lane) - 1u));
            if (mine && at < kListCap) {
                sm.list[wid][at] = (uint16_t)d;
                sm.list_bias[wid][at] = __ldg(w.bias_values + b + lane);
            }
            n_list += __popc(all);
        }
        n_bias = n_list;
        for (int h = 0; h * 512 < blocks; ++h) {
            uint32_t m = sm.seen[wid][h * 32 + lane] & ~sm.biased[wid][h * 32 + lane];
            int32_t at = __popc(m);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            const int32_t total = __shfl_sync(0xffffffffu, at, 31);
            at += n_list - __popc(m);
            for (; m != 0; m &= m - 1, ++at)
                if (at < kListCap)
                    sm.list[wid][at] = (uint16_t)(block_of(wid, lane, h) * kBlockIds + __ffs(m) - 1);
            n_list += total;
        }
        __syncwarp();
        load_entry();
        return true;
    }

    // One more token, of the warp's own ids.
    __device__ __forceinline__ void insert(uint32_t d, bool made) {
        const uint32_t o = place_of(d), c = sm.count[wid][o];
        const bool seen = is_seen(d), listed = !seen && !is_biased(d);
        __syncwarp();
        if (lane == 0) {
            if (made && c != kCountFull) sm.count[wid][o] = (uint16_t)(c + 1);
            if (!seen) sm.seen[wid][o >> 5] |= 1u << (o & 31);
            if (listed && n_list < kListCap) sm.list[wid][n_list] = (uint16_t)d;
        }
        if (listed) ++n_list;
        __syncwarp();
    }

    // Moves to the row of the stage.  False on a timeout.
    __device__ __forceinline__ bool enter_row(int s, const RowDesc &d) {
        if (d.flags & kDescRebuild) return rebuild(sm.rules[s]);
        bool own = false;
        for (int j = 0; j < d.n_new; ++j) {
            const int32_t x = sm.desc[s].fresh[j];
            ++len;
            if (x < 0) continue;
            const uint32_t id = (uint32_t)(x & ~kMade);
            if (owner_of(id) != (uint32_t)wid) continue;
            insert(id, (x & kMade) != 0);
            own = true;
        }
        if (own) load_entry();
        return true;
    }

    // Calls f(d, factor of a positive logit, of another one, summand) for the lane's
    // share of the warp's touched ids: each of them once in the warp.
    template <typename F>
    __device__ __forceinline__ void for_touched(F f) const {
        if (n_list <= kListCap) {
            if (e_id >= 0) f((uint32_t)e_id, e_pos, e_neg, e_add);
            for (int i = lane + 32; i < n_list; i += 32) {
                const uint32_t d = sm.list[wid][i];
                const bool seen = is_seen(d);
                f(d, seen ? inv_rho : 1.f, seen ? w.rho : 1.f,
                  summand(d, i < n_bias ? sm.list_bias[wid][i] : 0.f));
            }
        } else {
            for (int h = 0; h * 512 * kBlockIds < nid; ++h) {
                const uint32_t sw = sm.seen[wid][h * 32 + lane], bw = sm.biased[wid][h * 32 + lane];
                for (uint32_t m = sw | bw; m != 0; m &= m - 1) {
                    const int b = __ffs(m) - 1;
                    const uint32_t d = block_of(wid, lane, h) * kBlockIds + b;
                    const bool seen = (sw >> b) & 1u;
                    const float bias = (bw >> b) & 1u ? bias_of(w.bias_ids, w.bias_values, w.n_bias,
                                                                s0 + (int32_t)d) : 0.f;
                    f(d, seen ? inv_rho : 1.f, seen ? w.rho : 1.f, summand(d, bias));
                }
            }
        }
    }
};

template <typename Smem, int RING>
__device__ __forceinline__ void rule_smem_init(Smem &sm, int free_count) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kRuleWarps);
            mbar_init(&sm.free[s], free_count);
        }
        mbar_init(&sm.sync, kRuleWarps);
        fence_mbar_init();
    }
}

}  // namespace
}  // namespace ps
