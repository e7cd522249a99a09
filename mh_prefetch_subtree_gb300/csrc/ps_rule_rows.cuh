// Streaming rows under rules: the part that ps_process.cu and ps_score_rules.cu
// share.
//
// A block owns a slice of the vocabulary and walks down the rows, so that
// consecutive positions of a sequence, which differ by one token of history,
// reuse what is known about the row before.  The ids that a history touches lie close
// together (common tokens have low ids), and with slices of neighbouring ids the blocks
// of the first slice took 1.8 times as long as the others; so the first ids are dealt
// to the slices in segments of 1024, some for each, and only the rest is cut into runs.
// (All in segments: 22 bulk copies for each row of a slice and as many for its mask, one
// after another.)  The block's warps have three jobs.  The
// producers, one a stage, take the rows in turn (one alone spent 3200 cycles on a
// row, and a row of 48 KB has about 1900), say in a descriptor what changed since the row before,
// and fill a ring of stages: the slice of the row's logits (bulk copies) and of its
// mask.  The patchers know which ids penalties and biases touch
// and treat those in the stage.  The others work on all that is left, without a
// thought for the rules but the mask.  (Spread over the warps that also sum, the
// touched ids cost nearly as many instructions as the sums: 620 for 64 ids a lane,
// against 340 alone.)
//
// What the patchers know is in shared memory: how often each id of the slice was
// generated (16 bits), bit sets of the seen and the biased ones, and a list of both
// while it is short.  Blocks of 32 ids (one mask word) are dealt to them in turn:
// ids of common tokens lie close together, so a warp that owned a long run of ids
// could hold most of a history.  A new token costs a few instructions in the one
// warp that owns it.  Where the sequence changes, all warps but the producers read
// the whole history together.
#pragma once

#include "ps_row_sums.cuh"
#include "ps_rules.cuh"

namespace ps {
namespace {

constexpr int kSumWarps = 12;                        // work on all ids
constexpr int kPatchWarps = 4;
constexpr int kPatchThreads = kPatchWarps * 32;
constexpr int kCountThreads = (kSumWarps + kPatchWarps) * 32;
constexpr int kFirstProducer = kSumWarps + kPatchWarps;
// One producer a stage: a stage's phases then are one warp's to wait for, in
// order.  (With more producers than stages one could wait two phases ahead, which
// a parity cannot tell from the phase before.)
template <int RING>
constexpr int rule_threads() { return (kFirstProducer + RING) * 32; }
constexpr int kHeld = 3;                             // of them in each lane's registers
constexpr int kListCap = 896;                        // touched ids of a warp kept as a list
constexpr int kBiasCap = 64;                         // biased ones among them
constexpr uint32_t kCountFull = 0xffffu;             // a count that no longer fits
constexpr int64_t kNoSeq = INT64_MIN;
constexpr int kMaxNew = 6;                           // new tokens of a row handed on one by one
constexpr uint64_t kRuleWaitNs = 4000000000ull;      // 4 s: a copy, or the other warps
constexpr uint64_t kRuleDrainNs = 1000000000ull;
constexpr int kBlockIds = 32;
constexpr int kMaskCache = 256;                      // masks whose size is remembered

// What the producer tells about one row.
struct __align__(16) RowDesc {
    int32_t tok;                // the scored token's local number, or -1
    int32_t bad;                // status bits so far
    int32_t flags;              // kDesc*, and from bit 8 on the number of new tokens
    int32_t len;                // tokens of history
    int32_t fresh[kMaxNew];     // new tokens' local numbers, -1 or kFreshBad; kMade set: generated
    int32_t pad[2];
};
constexpr int32_t kDescRebuild = 1, kDescMask = 2, kDescSparse = 4, kDescNew = 256;
// Narrow masks: copied by vectors while they would take at most this part of the
// slice.  (A copy of 16 bytes takes a memory sector of its own, and time to issue;
// bulk copies of 16 bytes would take more, as a warp issues them one by one.)  1000 rows
// of 151936 bf16 processed under masks that leave half of the ids and more, 2%, 0.1%, 32
// ids: 125, 126, 118, 113 us up to a sixteenth, the same up to a sixty-fourth; 123, 152,
// 119, 112 up to a fourth; 123, 123, 123, 122 if never.  Only ps_process_rows copies so: a row to
// be scored is sooner in whole (8000 rows of 151936 under 24 masks of these kinds 530 us
// and 735 with such copies, with 0.1% 425 and 725; 1500 rows of 262144 with entropy 228
// and 269).
constexpr int32_t kSparseShare = 16;
constexpr int32_t kMade = 0x40000000;
constexpr int32_t kFreshBad = 0x20000000;            // not an id of the vocabulary

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes) : "memory");
}

// 16 bytes by the calling thread, asynchronously; and an arrival once its copies
// so far have landed.
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared memory of a block.  NB: blocks of 32 ids per lane of the summing warps;
// RING: stages.
template <int DT, int NB, int RING>
struct RuleSmem {
    static constexpr int kEsz = DT == PS_BF16 ? 2 : 4;
    static constexpr int kIds = kSumWarps * 32 * NB * kBlockIds;      // of a slice, at most
    static constexpr int kBlocks = kIds / kBlockIds;
    uint8_t stage[RING][kIds * kEsz];
    alignas(128) uint32_t mask[RING][kBlocks];
    uint16_t count[kIds];
    uint32_t seen[kBlocks];
    uint32_t biased[kBlocks];
    uint16_t list[kPatchWarps][kListCap];            // local numbers
    float list_bias[kPatchWarps][kBiasCap];
    RowDesc desc[RING];
    RowRules rules[RING];
    uint64_t mask_ids[kMaskCache];                   // a mask and slice, and its ids there
    // a stage is full (producer and copies), patched, and finished with
    uint64_t full[RING], patched[RING], empty[RING];
    uint64_t sync;                                   // all warps but the producers
    int32_t bad[2];                                  // of a rebuild, by its parity
};

__device__ __forceinline__ uint32_t owner_of(uint32_t d) { return (d / kBlockIds) % kPatchWarps; }

// A slice of the vocabulary: its ids are numbered from 0 ("local").
struct SliceMap {
    int32_t V, n_slices, slice;
    int32_t head;               // ids of the slice in segments
    int32_t from;               // first id of its run
    int32_t nid;                // ids of the slice
    uint32_t inv;               // 2^32 / n_slices, rounded down

    __device__ SliceMap(const RuleCut &cut, int32_t V_, int32_t slice_)
        : V(V_), n_slices(cut.n_slices), slice(slice_), head(cut.head * kSegIds),
          inv(0xffffffffu / (uint32_t)cut.n_slices) {
        from = head * n_slices + slice * cut.run;
        nid = head + max(0, min(cut.run, V - from));
    }
    // The local number of id v in [0, V); -1 if it is another slice's.  (A quotient
    // below 2^20 by the reciprocal is one too small at most.)
    __device__ __forceinline__ int32_t local(int32_t v) const {
        if (v >= head * n_slices) {
            const int32_t d = v - from;
            return d >= 0 && d < nid - head ? head + d : -1;
        }
        const uint32_t j = (uint32_t)v / kSegIds;
        uint32_t q = __umulhi(j, inv), rem = j - q * n_slices;
        if (rem >= (uint32_t)n_slices) rem -= n_slices, ++q;
        return rem == (uint32_t)slice ? (int32_t)(q * kSegIds + (uint32_t)v % kSegIds) : -1;
    }
    __device__ __forceinline__ int32_t global(int32_t d) const {
        if (d >= head) return from + (d - head);
        return ((d / kSegIds) * n_slices + slice) * kSegIds + d % kSegIds;
    }
    // The slice is copied in pieces: segments, then the run.  Piece i begins at local
    // id piece_at(i) and has piece_ids(i) ids.
    __device__ __forceinline__ int pieces() const { return head / kSegIds + (nid > head); }
    __device__ __forceinline__ int32_t piece_at(int i) const { return min(i * kSegIds, head); }
    __device__ __forceinline__ int32_t piece_ids(int i) const {
        return i * kSegIds < head ? kSegIds : nid - head;
    }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// A 16-byte vector with `off` in the places whose bit of `bits` (the lowest 8 or 4) is
// 0.  A product spreads the bits over the sign bits of a word's bytes, and byte
// permutes with sign replication make masks of them.  (A table of masks in shared
// memory takes two instructions less a word, but its reads collide in the banks: 8000
// rows of 151936 with masks read whole took 1060 us.)
template <int DT>
__device__ __forceinline__ uint4 masked_by(uint4 q, uint32_t bits, uint32_t off) {
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (DT == PS_BF16) {
        // bits 0, 2, 4, 6 to 7, 15, 23, 31 (what else the sums hold reaches none of
        // these), and 1, 3, 5, 7 likewise
        const uint32_t even = (bits & 0x55u) * 0x02082080u, odd = (bits & 0xaau) * 0x01041040u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t k = prmt(even, odd, 0xcc88u + j * 0x1111u);
            w[j] = (w[j] & k) | (off & ~k);
        }
    } else {
        const uint32_t t = (bits & 15u) * 0x10204080u;            // bits 0 .. 3 likewise
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t k = prmt(t, t, 0x8888u + j * 0x1111u);
            w[j] = (w[j] & k) | (off & ~k);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The block h of 32 ids that a lane of a warp that works on all ids takes.
__device__ __forceinline__ uint32_t block_of(int wid, int lane, int h) {
    return (h * 32 + lane) * kSumWarps + (wid + lane) % kSumWarps;
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

// A producer warp: fills stage `me` with every RING-th row.
// SPARSE: where a row's mask leaves few of the slice's ids, only the 16-byte vectors that
// hold one are copied.
// done(row, slice): called once the consumers have finished the stage's row, before
// the stage is filled again.
template <int DT, int NB, int RING, bool SPARSE, typename Done>
__device__ __forceinline__ void rule_producer(RuleSmem<DT, NB, RING> &sm, const RulesParams &p,
                                              const RuleCut &cut, const uint8_t *logits,
                                              int64_t ld_bytes,
                                              const int64_t *row_index, int64_t n_logit_rows,
                                              const int32_t *tokens, Done done) {
    using Smem = RuleSmem<DT, NB, RING>;
    constexpr int kEsz = Smem::kEsz;
    constexpr int kWpl = Smem::kBlocks / 32;               // mask words of a lane
    constexpr int kVec = 16 / kEsz;                        // ids of a vector
    const ps_logit_rules &u = p.rules;
    const int lane = threadIdx.x & 31, me = (threadIdx.x >> 5) - kFirstProducer;
    const RuleSpan span(p.n_rows, cut.n_slices);
    const uint64_t policy = l2_evict_first_policy();
    const bool per_seq = u.seq_begin != nullptr || u.bias_begin != nullptr;
    const bool mask16 = u.mask && u.mask_ld % 4 == 0 && (reinterpret_cast<uintptr_t>(u.mask) & 15) == 0;

    // entries of rows base .. base + 31, one a lane
    int64_t base = -1;
    int32_t c_seq = 0, c_len = 0, c_mask = -1, c_tok = 0;
    int64_t c_src = 0;
    RowRules w{};                                          // of sequence w_seq
    int64_t w_seq = kNoSeq;
    int32_t win = -64, win_tok = 0;                        // 32 tokens of its history

    int64_t t = span.t0 + me;
    int64_t r = t % span.rows, r_before = 0;
    int32_t slice_before = 0;
    SliceMap map(cut, p.V, (int32_t)(t / span.rows));
    for (; t < span.t1; t += RING) {
        // the window holds r and the row before
        if (base < 0 || r <= base || r >= base + 32) {
            base = r > 0 ? r - 1 : 0;
            const int64_t i = base + lane;
            const bool in = i < p.n_rows;
            c_seq = (in && per_seq && u.row_seq) ? __ldg(u.row_seq + i) : 0;
            c_len = (in && u.seq_begin && u.row_len) ? __ldg(u.row_len + i) : 0;
            c_mask = (in && u.mask && u.row_mask) ? __ldg(u.row_mask + i) : -1;
            c_tok = (in && tokens) ? __ldg(tokens + i) : 0;
            c_src = (in && row_index) ? __ldg(row_index + i) : i;
        }
        const int k = (int)(r - base), k0 = k > 0 ? k - 1 : 0;
        int32_t bad = 0, flags = 0;
        int64_t rm = -1;
        if (u.mask) {
            rm = u.row_mask ? (int64_t)__shfl_sync(0xffffffffu, c_mask, k) : r;
            if (rm < (u.row_mask ? -1 : 0) || rm >= u.n_masks) bad |= PS_DEV_BAD_RULES;
            else if (rm >= 0) flags |= kDescMask;
        }
        int64_t src = __shfl_sync(0xffffffffu, c_src, k);
        if (row_index && (src < 0 || src >= n_logit_rows)) {
            bad |= PS_DEV_BAD_ROW_INDEX;
            src = 0;
        }
        const int32_t tok = __shfl_sync(0xffffffffu, c_tok, k);
        int32_t tok_d = -1;
        if (tokens) {
            if (tok < 0 || tok >= p.V) bad |= PS_DEV_BAD_TOKEN;
            else tok_d = map.local(tok);
        }

        const int64_t step = t - span.t0;
        const int s = me;
        const uint32_t lap = (uint32_t)(step / RING);
        if (lap > 0) {
            if (!mbar_wait_bounded(&sm.empty[s], (lap - 1) & 1u, kRuleWaitNs)) {
                if (lane == 0) set_status(p.status, PS_DEV_TIMEOUT);
                break;
            }
            done(s, r_before, slice_before);
        }
        r_before = r;
        slice_before = map.slice;
        // Logits and mask.  With SPARSE a mask that is not known yet is read word by word,
        // behind the copy of all logits; the next time its size says how to copy.
        const uint32_t bytes = (uint32_t)(map.nid * kEsz + 15) / 16 * 16;
        const uint8_t *from = logits + src * ld_bytes;
        const bool masked = flags & kDescMask;
        const uint32_t *mrow = u.mask + (masked ? rm * u.mask_ld : 0);
        const uint64_t key = (uint64_t)(rm * cut.n_slices + map.slice) + 1;
        bool known = false;
        if (SPARSE && masked) {
            const uint64_t x = *(volatile uint64_t *)&sm.mask_ids[rm % kMaskCache];
            known = x >> 16 == key;
            if (known && (int32_t)(x & 0xffffu) * 16 * kSparseShare <= (int32_t)bytes) flags |= kDescSparse;
        }
        const bool sparse = flags & kDescSparse;
        const bool copy_mask = masked && mask16 && !sparse && (known || !SPARSE);   // in bulk too
        if (!sparse) {
            if (lane == 0) {
                fence_proxy_async_smem();
                mbar_expect_tx(&sm.full[s], bytes + (copy_mask ? (map.nid + 127) / 128 * 16 : 0));
            }
            __syncwarp();
            if (lane < map.pieces()) {
                const int32_t d = map.piece_at(lane), ids = map.piece_ids(lane), v = map.global(d);
                bulk_g2s(sm.stage[s] + d * kEsz, from + (int64_t)v * kEsz,
                         (uint32_t)(ids * kEsz + 15) / 16 * 16, &sm.full[s], policy);
                if (copy_mask)
                    bulk_g2s(&sm.mask[s][d / 32], mrow + v / 32, (uint32_t)(ids + 127) / 128 * 16,
                             &sm.full[s], policy);
            }
        }
        if (masked && !copy_mask) {
            uint32_t m[kWpl];                              // the slice's words, by lane
            const int32_t nw = (map.nid + 31) / 32;
#pragma unroll
            for (int i = 0; i < kWpl; i += 4) {
                const int at = i * 32 + lane * 4;
                const uint32_t *word = mrow + map.global(at * 32) / 32;
                if (mask16) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (at < nw) x = __ldg(reinterpret_cast<const uint4 *>(word));
                    m[i] = x.x;
                    m[i + 1] = x.y;
                    m[i + 2] = x.z;
                    m[i + 3] = x.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) m[i + j] = at + j < nw ? __ldg(word + j) : 0u;
                }
            }
            int32_t ids = 0;
#pragma unroll
            for (int i = 0; i < kWpl; i += 4) {
                reinterpret_cast<uint4 *>(sm.mask[s])[i * 8 + lane] =
                    make_uint4(m[i], m[i + 1], m[i + 2], m[i + 3]);
                ids += __popc(m[i]) + __popc(m[i + 1]) + __popc(m[i + 2]) + __popc(m[i + 3]);
            }
            if (SPARSE && !known) {
                ids = __reduce_add_sync(0xffffffffu, ids);
                if (lane == 0) *(volatile uint64_t *)&sm.mask_ids[rm % kMaskCache] = key << 16 | ids;
            }
            if (SPARSE && sparse) {
                fence_proxy_async_smem();
#pragma unroll
                for (int i = 0; i < kWpl; ++i) {
                    const int at = ((i & ~3) * 32 + lane * 4 + (i & 3)) * 32;
                    uint32_t x = m[i];
                    while (x) {
                        // the vector that holds the lowest id left
                        const int v = (__ffs(x) - 1) / kVec * kVec;
                        const int32_t d = at + v;
                        if (d < map.nid)
                            copy16(sm.stage[s] + d * kEsz, from + (int64_t)map.global(d) * kEsz);
                        x &= ~(((1u << kVec) - 1u) << v);
                    }
                }
            }
        }
        // In the copies' shadow: what changed since the row before.  Its sequence and
        // length have to be in order, or the patchers do not know its history.
        const bool by_row = per_seq && !u.row_seq;
        const int64_t q = by_row ? r : (int64_t)__shfl_sync(0xffffffffu, c_seq, k);
        const int64_t q0 = by_row ? r - 1 : (int64_t)__shfl_sync(0xffffffffu, c_seq, k0);
        int32_t n = __shfl_sync(0xffffffffu, c_len, k), n0 = __shfl_sync(0xffffffffu, c_len, k0);
        int32_t n_new = 0, fresh = -1;                     // fresh: by lane
        if (q != w_seq) {
            w = row_rules(p, r);
            w_seq = w.bad ? kNoSeq : q;
            win = -64;
        }
        if (!u.row_len || !u.seq_begin) n = n0 = w.len_all;
        if (w_seq == q && q0 == q && t != span.t0 && r != 0 && n0 >= 0 && n0 <= w.len_all &&
            n >= n0 && n <= w.len_all && n - n0 <= kMaxNew) {
            n_new = n - n0;
            if (n_new) {
                if (n0 < win || n - 32 > win) {
                    win = n0;
                    win_tok = lane < w.len_all - win ? __ldg(w.hist + win + lane) : 0;
                }
                const int32_t id = __shfl_sync(0xffffffffu, win_tok, (n0 - win + lane) & 31);
                if (lane < n_new) {
                    if (id < 0 || id >= p.V) fresh = kFreshBad;
                    else fresh = map.local(id);
                    if (fresh >= 0 && fresh != kFreshBad && n0 + lane >= w.prompt) fresh |= kMade;
                }
                // tokens of other slices are no news
                if (!__any_sync(0xffffffffu, fresh != -1)) n_new = 0;
            }
        } else {
            w = row_rules(p, r);
            w_seq = w.bad ? kNoSeq : q;
            flags |= kDescRebuild;
            bad |= w.bad;
        }

        RowDesc &d = sm.desc[s];
        if (lane < n_new) d.fresh[lane] = fresh;
        if (lane == 0) {
            *reinterpret_cast<int4 *>(&d) = make_int4(tok_d, bad, flags | n_new * kDescNew, n);
            if (flags & kDescRebuild) sm.rules[s] = w;
        }
        // each lane's own copies (if any), then what the warp has written
        arrive_after_copies(&sm.full[s]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
        for (r += RING; r >= span.rows; r -= span.rows) {
            map = SliceMap(cut, p.V, map.slice + 1);
            base = -1;
        }
    }
    // the last row that was filled: its copies land before the block's memory goes
    t -= RING;
    if (t >= span.t0 && t < span.t1) {
        const uint32_t odd = (uint32_t)((t - span.t0) / RING) & 1u;
        if (mbar_wait_bounded(&sm.full[me], odd, kRuleDrainNs) &&
            mbar_wait_bounded(&sm.empty[me], odd, kRuleWaitNs))
            done(me, r_before, slice_before);
        else if (lane == 0)
            set_status(p.status, PS_DEV_TIMEOUT);              // the row is not stored
    }
}

// Waits for all warps but the producers, for the n-th time; false when they do not
// come.
template <typename Smem>
__device__ __forceinline__ bool rule_meet(Smem &sm, uint32_t n) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.sync);
    return mbar_wait_bounded(&sm.sync, n & 1u, kRuleWaitNs);
}

template <typename Smem>
__device__ __forceinline__ void count_token(Smem &sm, const SliceMap &map, int32_t id, bool made, bool fits,
                                            int32_t *bad_word) {
    if (id < 0 || id >= map.V) {
        atomicOr(bad_word, PS_DEV_BAD_TOKEN);
        return;
    }
    const int32_t d = map.local(id);
    if (d < 0) return;
    // most tokens of a history have come before
    if (!((*(volatile uint32_t *)&sm.seen[d >> 5] >> (d & 31)) & 1u))
        atomicOr(&sm.seen[d >> 5], 1u << (d & 31));
    if (!made) return;
    uint32_t *word = reinterpret_cast<uint32_t *>(&sm.count[d & ~1]);
    const int sh = (d & 1) * 16;
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

// Counts and bit sets of a history, made by all warps but the producers together,
// for the k-th time in this block.  Where the status bits of the history and the
// biases are; nullptr on a timeout.
template <typename Smem>
__device__ __noinline__ const int32_t *rule_tables(Smem &sm, SliceMap map, const RowRules &w, uint32_t k) {
    const int tid = threadIdx.x;
    const int32_t blocks = (map.nid + kBlockIds - 1) / kBlockIds, len = w.len, prompt = w.prompt;
    const int32_t *hist = w.hist;
    // a warp may still read the word of the time before
    int32_t *bad_word = &sm.bad[k & 1];
    if (tid == 0) *bad_word = 0;
    if (!rule_meet(sm, 3 * k)) return nullptr;      // the patchers are done with the tables
    for (int i = tid; i < blocks * kBlockIds / 8; i += kCountThreads)
        reinterpret_cast<uint4 *>(sm.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < blocks; i += kCountThreads) sm.seen[i] = sm.biased[i] = 0;
    if (!rule_meet(sm, 3 * k + 1)) return nullptr;
    const bool fits = len - max(0, min(prompt, len)) < (int32_t)kCountFull;
    constexpr int kAhead = 8;                       // tokens that a thread asks for at once
    // unsigned: a step past the last of 2^31 - 1 tokens has to end the loops
    for (uint32_t b = 0; b < (uint32_t)len; b += kCountThreads * kAhead) {
        int32_t id[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t i = b + j * kCountThreads + tid;
            id[j] = i < (uint32_t)len ? __ldg(hist + i) : 0;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t i = b + j * kCountThreads + tid;
            if (i < (uint32_t)len) count_token(sm, map, id[j], (int32_t)i >= prompt, fits, bad_word);
        }
    }
    for (uint32_t i = tid; i < (uint32_t)w.n_bias; i += kCountThreads) {
        const int32_t id = __ldg(w.bias_ids + i);
        if (id < 0 || id >= map.V || (i > 0 && id <= __ldg(w.bias_ids + i - 1))) {
            atomicOr(bad_word, PS_DEV_BAD_RULES);
            continue;
        }
        const int32_t d = map.local(id);
        if (d >= 0) atomicOr(&sm.biased[d >> 5], 1u << (d & 31));
    }
    return rule_meet(sm, 3 * k + 2) ? bad_word : nullptr;
}

// A patching warp's view of the rules.  The same in all lanes unless said
// otherwise.
template <typename Smem>
struct RuleWalk {
    Smem &sm;
    const RulesParams &p;
    const int lane, wid;        // wid: among the patchers
    SliceMap map;
    int32_t len = 0;            // tokens of history that are counted
    int32_t n_list = 0;         // touched ids; the first n_bias of the list are biased
    int32_t n_bias = 0;
    int32_t bad = 0;            // status bits of the history and the biases
    uint32_t fills = 0;         // of the tables
    RowRules w{};
    float inv_rho = 1.f;
    // by lane: entries lane, lane + 32, ... of the list (local number, kMade set:
    // seen; -1 if there is none) and what is added to their logits
    int32_t e_id[kHeld];
    float e_add[kHeld];

    __device__ RuleWalk(Smem &sm_, const RulesParams &p_, const SliceMap &map_)
        : sm(sm_), p(p_), lane(threadIdx.x & 31), wid((threadIdx.x >> 5) - kSumWarps), map(map_) {}

    __device__ __forceinline__ bool is_seen(uint32_t d) const { return (sm.seen[d >> 5] >> (d & 31)) & 1u; }
    __device__ __forceinline__ bool is_biased(uint32_t d) const {
        return (sm.biased[d >> 5] >> (d & 31)) & 1u;
    }
    // How often id d was generated.  A count that does not fit 16 bits is taken
    // again from the history: slow, and as rare as a token that one sequence holds
    // 65535 times.
    __device__ __forceinline__ uint32_t times(uint32_t d) const {
        const uint32_t c = sm.count[d];
        return c == kCountFull ? recount(w.hist, max(0, w.prompt), len, map.global((int32_t)d)) : c;
    }

    // The processed logit of id d from its logit: a factor by sign, then a sum that
    // does not depend on the logit.
    __device__ __forceinline__ float summand(uint32_t d, float bias) const {
        const uint32_t n = times(d);
        return bias - (w.freq * (float)n + (n ? w.pres : 0.f));
    }

    __device__ __forceinline__ void load_entries() {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = lane + 32 * j;
            e_id[j] = -1;
            if (n_list <= kListCap && i < n_list) {
                const uint32_t d = sm.list[wid][i];
                e_id[j] = (int32_t)d | (is_seen(d) ? kMade : 0);
                e_add[j] = summand(d, i < n_bias ? sm.list_bias[wid][i] : 0.f);
            }
        }
    }

    // Takes up a row's sequence with its history so far.  False on a timeout.
    __device__ __forceinline__ bool rebuild(const RowRules &from) {
        w = from;
        inv_rho = 1.f / w.rho;
        len = w.len;
        const int32_t *bad_word = rule_tables(sm, map, from, fills++);
        if (bad_word == nullptr) return false;
        bad = *reinterpret_cast<const volatile int32_t *>(bad_word);
        const int32_t blocks = (map.nid + kBlockIds - 1) / kBlockIds;
        // the list: the biased ids in the order of their list, then the others seen
        n_list = 0;
        for (int b = 0; bad == 0 && b < w.n_bias; b += 32) {
            const int32_t id = b + lane < w.n_bias ? __ldg(w.bias_ids + b + lane) : -1;
            const int32_t d = id >= 0 ? map.local(id) : -1;
            const bool mine = d >= 0 && owner_of(d) == (uint32_t)wid;
            const uint32_t all = __ballot_sync(0xffffffffu, mine);
            const int32_t at = n_list + __popc(all & ((1u << lane) - 1u));
            if (mine && at < kBiasCap) {
                sm.list[wid][at] = (uint16_t)d;
                sm.list_bias[wid][at] = __ldg(w.bias_values + b + lane);
            }
            n_list += __popc(all);
        }
        n_bias = n_list;
        if (n_bias > kBiasCap) n_list = kListCap + 1;       // no list
        for (int b0 = 0; b0 < blocks; b0 += kPatchThreads) {
            const int b = b0 + lane * kPatchWarps + wid;
            uint32_t m = b < blocks ? sm.seen[b] & ~sm.biased[b] : 0u;
            int32_t at = __popc(m);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            const int32_t total = __shfl_sync(0xffffffffu, at, 31);
            at += n_list - __popc(m);
            for (; m != 0; m &= m - 1, ++at)
                if (at < kListCap) sm.list[wid][at] = (uint16_t)(b * kBlockIds + __ffs(m) - 1);
            n_list += total;
        }
        __syncwarp();
        load_entries();
        return true;
    }

    // One more token, of the warp's own ids.
    __device__ __forceinline__ void insert(uint32_t d, bool made) {
        const uint32_t c = sm.count[d];
        const bool seen = is_seen(d), listed = !seen && !is_biased(d);
        __syncwarp();
        if (lane == 0) {
            if (made && c != kCountFull) sm.count[d] = (uint16_t)(c + 1);
            if (!seen) sm.seen[d >> 5] |= 1u << (d & 31);
            if (listed && n_list < kListCap) sm.list[wid][n_list] = (uint16_t)d;
        }
        if (listed) ++n_list;
        __syncwarp();
    }

    // Moves to the row of the stage.  False on a timeout.
    __device__ __forceinline__ bool enter_row(int s, int32_t flags, int32_t n) {
        if (flags & kDescRebuild) return rebuild(sm.rules[s]);
        len = n;
        bool own = false;
        for (int j = 0; j < flags / kDescNew; ++j) {
            const int32_t x = sm.desc[s].fresh[j];
            if (x == kFreshBad) bad |= PS_DEV_BAD_TOKEN;
            if (x < 0 || x == kFreshBad) continue;
            const uint32_t id = (uint32_t)(x & ~kMade);
            if (owner_of(id) != (uint32_t)wid) continue;
            insert(id, (x & kMade) != 0);
            own = true;
        }
        if (own) load_entries();
        return true;
    }

    // Calls f(j, d, factor of a positive logit, of another one, summand) for the lane's
    // share of the warp's touched ids, each of them once in the warp: its j-th.
    template <typename F>
    __device__ __forceinline__ void for_touched(F f) const {
        if (n_list <= kListCap) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (n_list <= 32 * j) return;
                const bool seen = e_id[j] & kMade;
                if (e_id[j] >= 0)
                    f(j, (uint32_t)(e_id[j] & ~kMade), seen ? inv_rho : 1.f, seen ? w.rho : 1.f, e_add[j]);
            }
            for (int i = lane + 32 * kHeld; i < n_list; i += 32) {
                const uint32_t d = sm.list[wid][i];
                const bool seen = is_seen(d);
                f(i / 32, d, seen ? inv_rho : 1.f, seen ? w.rho : 1.f,
                  summand(d, i < n_bias ? sm.list_bias[wid][i] : 0.f));
            }
        } else {
            // too many for a list: block by block, one id a lane
            int j = 0;
            for (int b = wid; b * kBlockIds < map.nid; b += kPatchWarps) {
                const uint32_t sw = sm.seen[b], bw = sm.biased[b];
                if (((sw | bw) >> lane) & 1u) {
                    const uint32_t d = b * kBlockIds + lane;
                    const bool seen = (sw >> lane) & 1u;
                    const float bias = (bw >> lane) & 1u ? bias_of(w.bias_ids, w.bias_values, w.n_bias,
                                                                   map.global((int32_t)d)) : 0.f;
                    f(j++, d, seen ? inv_rho : 1.f, seen ? w.rho : 1.f, summand(d, bias));
                }
            }
        }
    }
};

template <typename Smem, int RING>
__device__ __forceinline__ void rule_smem_init(Smem &sm) {
    for (int i = threadIdx.x; i < kMaskCache; i += blockDim.x) sm.mask_ids[i] = 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(&sm.full[s], 33);               // the producer's lanes, and once more
            mbar_init(&sm.patched[s], kPatchWarps);
            mbar_init(&sm.empty[s], kSumWarps);
        }
        mbar_init(&sm.sync, kSumWarps + kPatchWarps);
        fence_mbar_init();
    }
}

}  // namespace
}  // namespace ps
