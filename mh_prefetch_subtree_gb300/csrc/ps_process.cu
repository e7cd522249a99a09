// Rules applied to logits rows, written out (ps_process_rows).
//
// A row is nearly all copy: its history and bias list touch some hundreds of
// V ids, the mask needs one bit each.
//
// Apart from the input, the rows stream through shared memory (ps_rule_rows.cuh):
// bulk copies bring a slice of a row in, the patchers rewrite its touched ids, the
// other warps write -inf where the mask says so (only into vectors that it
// touches), and the stage's producer sends it out with bulk copies before it fills
// the stage again.  What bounds it is memory: every byte is read once and written
// once.
//
// In place nothing has to move but what the rules change, so a kernel of its own
// writes masked vectors and touched ids only; it reads each slice's part of the
// history anew for every row, into a table of counts in shared memory.
#include "ps_rule_rows.cuh"

namespace ps {
namespace {

constexpr int kRing = 3;

template <int DT>
struct ProcessSmem : RuleSmem<DT, DT == PS_BF16 ? 2 : 1, kRing> {
    int32_t row_bad[kRing];
};
static_assert(sizeof(ProcessSmem<PS_BF16>) <= 232448 && sizeof(ProcessSmem<PS_F32>) <= 232448,
              "the shared memory of a block");

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}
// The calling thread's bulk stores so far have read their source / are done.
__device__ __forceinline__ void bulk_stores_read() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_stores_done() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The patchers' rows: the touched ids rewritten in the stage.
template <int DT, typename Smem>
__device__ __forceinline__ void patch_rows(Smem &sm, const ProcessParams &p, const RuleCut &cut) {
    const int lane = threadIdx.x & 31;
    const RuleSpan span(p.r.n_rows, cut.n_slices);
    int64_t r = span.t0 % span.rows;
    RuleWalk<Smem> walk(sm, p.r, SliceMap(cut, p.r.V, (int32_t)(span.t0 / span.rows)));
    int s = 0;
    uint32_t lap = 0;
    for (int64_t t = span.t0; t < span.t1; ++t) {
        if (!mbar_wait_bounded(&sm.full[s], lap & 1u, kRuleWaitNs)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        uint8_t *buf = sm.stage[s];
        const int4 dh = *reinterpret_cast<const int4 *>(&sm.desc[s]);       // -, bad, flags, len
        if ((dh.z & ~(kDescMask | kDescSparse)) && !walk.enter_row(s, dh.z, dh.w)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        const int32_t bad = dh.y | walk.bad;
        if (walk.wid == 0 && lane == 0) {
            if (bad && walk.map.slice == 0) set_status(p.r.status, bad);
            sm.row_bad[s] = bad;
        }
        // a masked id may hold anything now: the mask comes after
        if (!bad)
            walk.for_touched([&](int, uint32_t d, float pos, float neg, float add) {
                const float l = load_elem<DT>(buf, d);
                store_elem<DT>(buf, d, fmaf(l, l > 0.f ? pos : neg, add));
            });
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.patched[s]);
        if (++s == kRing) {
            s = 0;
            ++lap;
        }
        if (++r == span.rows) {
            r = 0;
            walk.map = SliceMap(cut, p.r.V, walk.map.slice + 1);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(rule_threads<kRing>(), 1) process_rows_kernel(
    const __grid_constant__ ProcessParams p, const __grid_constant__ RuleCut cut) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Smem = ProcessSmem<DT>;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    constexpr int kNb = DT == PS_BF16 ? 2 : 1;
    constexpr int kEsz = Smem::kEsz;
    constexpr int kVec = 16 / kEsz;
    constexpr int kBv = kBlockIds / kVec;
    constexpr uint32_t kOff = Elem<DT>::kNegInfWord;
    constexpr uint32_t kNan = DT == PS_BF16 ? 0x7fc07fc0u : 0x7fc00000u;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    rule_smem_init<Smem, kRing>(sm);
    __syncthreads();

    if (wid >= kFirstProducer) {
        rule_producer<DT, kNb, kRing, true>(
            sm, p.r, cut, p.logits, p.ld_bytes, nullptr, p.r.n_rows, nullptr,
            [&](int s, int64_t r, int32_t slice) {
                // out with the stage: whole vectors in bulk, ids after the last one by hand
                const SliceMap map(cut, p.r.V, slice);
                uint8_t *to = p.out + r * p.out_ld_bytes;
                if (lane < map.pieces()) {
                    const int32_t d = map.piece_at(lane), ids = map.piece_ids(lane);
                    const int64_t v = map.global(d);
                    const int32_t whole = ids / kVec * kVec;
                    const uint8_t *from = sm.stage[s] + d * kEsz;
                    if (whole) bulk_s2g(to + v * kEsz, from, whole * kEsz);
                    for (int32_t i = whole; i < ids; ++i) {
                        if constexpr (DT == PS_BF16)
                            reinterpret_cast<uint16_t *>(to)[v + i] = reinterpret_cast<const uint16_t *>(from)[i];
                        else
                            reinterpret_cast<float *>(to)[v + i] = reinterpret_cast<const float *>(from)[i];
                    }
                }
                bulk_stores_read();
                __syncwarp();
            });
        bulk_stores_done();
        return;
    }
    if (wid >= kSumWarps) {
        patch_rows<DT>(sm, p, cut);
        return;
    }

    const RuleSpan span(p.r.n_rows, cut.n_slices);
    int64_t r = span.t0 % span.rows;
    int32_t slice = (int32_t)(span.t0 / span.rows);
    int32_t nid = SliceMap(cut, p.r.V, slice).nid;
    int s = 0;
    uint32_t lap = 0;
    const uint32_t first = block_of(wid, lane, 0);
    uint32_t fills = 0;
    for (int64_t t = span.t0; t < span.t1; ++t) {
        bool ok = mbar_wait_bounded(&sm.full[s], lap & 1u, kRuleWaitNs);
        if (ok && (sm.desc[s].flags & kDescRebuild))
            ok = rule_tables(sm, SliceMap(cut, p.r.V, slice), sm.rules[s], fills++) != nullptr;
        if (!ok || !mbar_wait_bounded(&sm.patched[s], lap & 1u, kRuleWaitNs)) {
            if (lane == 0) set_status(p.r.status, PS_DEV_TIMEOUT);
            return;
        }
        const bool bad = sm.row_bad[s] != 0;
        if (bad || (sm.desc[s].flags & kDescMask)) {
#pragma unroll
            for (int h = 0; h < kNb; ++h) {
                const uint32_t b = first + h * 32 * kSumWarps;
                if (b * kBlockIds >= (uint32_t)nid) continue;
                const uint32_t m = bad ? 0u : sm.mask[s][b];
                if (m == 0xffffffffu) continue;
                uint4 *v = reinterpret_cast<uint4 *>(sm.stage[s]) + b * kBv;
#pragma unroll
                for (int i = 0; i < kBv; ++i) {
                    // the lanes' vectors in an order that spreads them over the banks
                    const int k = kBv == 4 ? ((i + (lane >> 1)) & 3) : ((i + lane) & 7);
                    const uint32_t x = m >> (k * kVec);
                    v[k] = masked_by<DT>(v[k], x, bad ? kNan : kOff);
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[s]);
        if (++s == kRing) {
            s = 0;
            ++lap;
        }
        if (++r == span.rows) {
            r = 0;
            ++slice;
            if (slice < cut.n_slices) nid = SliceMap(cut, p.r.V, slice).nid;
        }
    }
}

// In place: a block takes a run of ids of one row.
template <int DT>
__global__ void __launch_bounds__(kTableThreads) process_in_place_kernel(const ProcessParams p,
                                                                         int32_t n_runs) {
    extern __shared__ __align__(16) uint8_t smem[];
    SliceTable &t = *reinterpret_cast<SliceTable *>(smem);
    constexpr int kEsz = DT == PS_BF16 ? 2 : 4;
    constexpr int kVec = 16 / kEsz;
    const int tid = threadIdx.x;
    const int32_t V = p.r.V;
    const int64_t n_tasks = p.r.n_rows * n_runs;
    for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
        const int64_t r = task / n_runs;
        const int32_t v0 = (int32_t)(task - r * n_runs) * kSliceIds;
        const int32_t n = min(kSliceIds, V - v0);
        RowRules w = row_rules(p.r, r);
        w.bad |= build_table(t, w, V, v0);
        uint8_t *row = p.out + r * p.out_ld_bytes;
        if (w.bad) {
            if (tid == 0 && v0 == 0) set_status(p.r.status, w.bad);
            for (int i = tid; i < n; i += blockDim.x)
                store_elem<DT>(row, v0 + i, __int_as_float(0x7fc00000));
            __syncthreads();
            continue;
        }
        if (w.mask)
            for (int i = tid * kVec; i < n; i += blockDim.x * kVec) {
                const int32_t v = v0 + i;
                const uint32_t m = mask_bits<kVec>(w.mask, v, V);
                if (v + kVec <= V) {
                    if (m == (1u << kVec) - 1u) continue;
                    uint4 *q = reinterpret_cast<uint4 *>(row + (int64_t)v * kEsz);
                    *q = masked_vec<DT>(m ? *q : make_uint4(0, 0, 0, 0), m);
                } else {
                    for (int j = 0; v + j < V; ++j)
                        if (!((m >> j) & 1u)) store_elem<DT>(row, v + j, -INFINITY);
                }
            }
        // an allowed id still holds its logit here
        __syncthreads();
        for_seen(t, [&](uint32_t o) {
            const int32_t v = v0 + (int32_t)o;
            if (is_biased(t, o) || !mask_allows(w.mask, v)) return;
            store_elem<DT>(row, v, penalised(load_elem<DT>(row, v), t.count[o], w, 0.f));
        });
        for (int i = tid; i < w.n_bias; i += blockDim.x) {
            const int32_t v = __ldg(w.bias_ids + i);
            const uint32_t o = (uint32_t)(v - v0);
            if (o >= (uint32_t)kSliceIds || !mask_allows(w.mask, v)) continue;
            store_elem<DT>(row, v, penalised(load_elem<DT>(row, v), t.count[o], w,
                                             __ldg(w.bias_values + i)));
        }
        __syncthreads();
    }
}

template <int DT>
cudaError_t launch(const ProcessParams &p, int sms, cudaStream_t stream) {
    if (p.out == p.logits) {
        const int smem = (int)sizeof(SliceTable);
        cudaError_t e = cudaFuncSetAttribute(process_in_place_kernel<DT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int32_t runs = (int32_t)(((int64_t)p.r.V + kSliceIds - 1) / kSliceIds);
        const int64_t tasks = p.r.n_rows * runs, most = (int64_t)sms * 4;
        process_in_place_kernel<DT>
            <<<(int)(tasks < most ? tasks : most), kTableThreads, smem, stream>>>(p, runs);
        return cudaGetLastError();
    }
    const int smem = (int)sizeof(ProcessSmem<DT>);
    cudaError_t e = cudaFuncSetAttribute(process_rows_kernel<DT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const RuleCut cut = rule_cut(p.r.V, ProcessSmem<DT>::kIds, p.r.n_rows);
    const int64_t tasks = p.r.n_rows * cut.n_slices;
    process_rows_kernel<DT>
        <<<(int)(tasks < sms ? tasks : sms), rule_threads<kRing>(), smem, stream>>>(p, cut);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_process_rows(const ProcessParams &p, int32_t dtype, int sms,
                                cudaStream_t stream) {
    return dtype == PS_BF16 ? launch<PS_BF16>(p, sms, stream) : launch<PS_F32>(p, sms, stream);
}

}  // namespace ps
