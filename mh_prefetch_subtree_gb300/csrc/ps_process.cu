// Rules applied to logits rows, written out (ps_process_rows).
//
// A row is nearly all copy: its history and bias list touch some hundreds of
// V ids, the mask needs one bit each.  So a block takes one slice of one row,
// copies it with the mask applied, and then rewrites the touched ids of the
// slice, which it has collected in a table of counts in shared memory.
#include "ps_rules.cuh"

namespace ps {
namespace {

template <int DT>
__global__ void __launch_bounds__(kTableThreads) process_rows_kernel(const ProcessParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    SliceTable &t = *reinterpret_cast<SliceTable *>(smem);
    constexpr int kEsz = DT == PS_BF16 ? 2 : 4;
    constexpr int kVec = 16 / kEsz;
    const int tid = threadIdx.x;
    const int32_t V = p.r.V;
    const int64_t n_tasks = p.r.n_rows * p.n_slices;
    for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
        const int64_t r = task / p.n_slices;
        const int32_t v0 = (int32_t)(task - r * p.n_slices) * kSliceIds;
        const int32_t n = min(kSliceIds, V - v0);
        RowRules w = row_rules(p.r, r);
        w.bad |= build_table(t, w, V, v0);
        const uint8_t *src = p.logits + r * p.ld_bytes;
        uint8_t *dst = p.out + r * p.out_ld_bytes;
        if (w.bad) {
            if (tid == 0 && v0 == 0) set_status(p.r.status, w.bad);
            for (int i = tid; i < n; i += blockDim.x)
                store_elem<DT>(dst, v0 + i, __int_as_float(0x7fc00000));
            __syncthreads();
            continue;
        }
        for (int i = tid * kVec; i < n; i += blockDim.x * kVec) {
            const int32_t v = v0 + i;
            const uint32_t m = mask_bits<kVec>(w.mask, v, V);
            if (v + kVec <= V) {
                const uint4 q = *reinterpret_cast<const uint4 *>(src + (int64_t)v * kEsz);
                *reinterpret_cast<uint4 *>(dst + (int64_t)v * kEsz) = masked_vec<DT>(q, m);
            } else {
                for (int j = 0; v + j < V; ++j)
                    store_elem<DT>(dst, v + j, (m >> j) & 1u ? load_elem<DT>(src, v + j) : -INFINITY);
            }
        }
        // in place, an allowed id still holds its logit here
        __syncthreads();
        for_seen(t, [&](uint32_t o) {
            const int32_t v = v0 + (int32_t)o;
            if (is_biased(t, o) || !mask_allows(w.mask, v)) return;
            store_elem<DT>(dst, v, penalised(load_elem<DT>(src, v), t.count[o], w));
        });
        for (int i = tid; i < w.n_bias; i += blockDim.x) {
            const int32_t v = __ldg(w.bias_ids + i);
            const uint32_t o = (uint32_t)(v - v0);
            if (o >= (uint32_t)kSliceIds || !mask_allows(w.mask, v)) continue;
            store_elem<DT>(dst, v, penalised(load_elem<DT>(src, v), t.count[o], w) +
                                       __ldg(w.bias_values + i));
        }
        __syncthreads();
    }
}

template <int DT>
cudaError_t launch(const ProcessParams &p, int sms, cudaStream_t stream) {
    const int smem = (int)sizeof(SliceTable);
    cudaError_t e = cudaFuncSetAttribute(process_rows_kernel<DT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t tasks = p.r.n_rows * p.n_slices, most = (int64_t)sms * 4;
    process_rows_kernel<DT><<<(int)(tasks < most ? tasks : most), kTableThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

int32_t rules_slice_ids(int32_t) { return kSliceIds; }

cudaError_t launch_process_rows(const ProcessParams &p, int32_t dtype, int sms,
                                cudaStream_t stream) {
    return dtype == PS_BF16 ? launch<PS_BF16>(p, sms, stream) : launch<PS_F32>(p, sms, stream);
}

}  // namespace ps
