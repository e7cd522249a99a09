// Host side of the entry points around proposals: projections of hidden rows, and drawing
// and scoring tokens under truncation.  See include/ps.h for the contract.
#include <algorithm>
#include <initializer_list>

#include "ps_api.cuh"
#include "ps_linear.cuh"
#include "ps_sample.cuh"

using namespace ps;

namespace {

// What the host can see of the sampling.
ps_status check_sampling_host(const ps_sampling *s, int32_t V, int64_t n_rows) {
    if (!s || s->n_sets < 1 || !s->tau || V > kSampleMostV) return PS_ERR_INVALID_ARG;
    if (!s->row_set && s->n_sets != 1 && s->n_sets < n_rows) return PS_ERR_INVALID_ARG;
    for (const void *p : {(const void *)s->tau, (const void *)s->top_k, (const void *)s->top_p,
                          (const void *)s->min_p, (const void *)s->row_set})
        if (!aligned(p, 4)) return PS_ERR_INVALID_ARG;
    return PS_OK;
}

// That what a kernel will read or write is the device's, where it is given.
bool all_on_device(std::initializer_list<const void *> pointers) {
    for (const void *p : pointers)
        if (p && !on_device(p)) return false;
    return true;
}
bool sampling_on_device(const ps_sampling *s) {
    return all_on_device({s->tau, s->top_k, s->top_p, s->min_p, s->row_set});
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uint8_t *x = (const uint8_t *)a, *y = (const uint8_t *)b;
    return x < y + nb && y < x + na;
}

// Checks a projection's arguments and launches it.
ps_status linear_rows(const ps_linear *h, const void *x, int64_t x_ld, int32_t n_rows, const void *residual,
                      int64_t residual_ld, void *out, int64_t ld, int32_t dtype, bool lost, void *cuda_stream) {
    // Elements that an array may span: more is no memory, and fewer are counted in bytes below.  A
    // copied tile's rows are at most 2^39 bytes apart.
    constexpr int64_t kMostSpan = int64_t(1) << 40, kMostStride = int64_t(1) << 38;
    // A block waits for a whole tile's sums, up to 2^18 steps of its copies: a tenth of a second, far from a wait's 2.
    constexpr int32_t kMostK = 1 << 24;
    if (!h || n_rows < 0 || h->N < 1 || h->K < 1 || h->K > kMostK || h->K % 8 != 0) return PS_ERR_INVALID_ARG;
    const int esz = elem_size(dtype);
    if (esz == 0 || (h->bias && elem_size(h->bias_dtype) == 0)) return PS_ERR_UNSUPPORTED;
    if (h->act < PS_ACT_NONE || h->act > PS_ACT_GELU) return PS_ERR_UNSUPPORTED;
    // the kernel multiplies by 1 / cap, which is to be far from what float32 cannot hold
    if (h->act == PS_ACT_CAP && !(h->cap >= 0x1p-60f && h->cap <= 0x1p60f)) return PS_ERR_INVALID_ARG;
    if (!h->w || !aligned(h->w, 16) || h->w_ld < h->K || h->w_ld % 8 != 0 || h->w_ld > std::min(kMostSpan / h->N, kMostStride) ||
        (h->bias && !aligned(h->bias, (size_t)elem_size(h->bias_dtype))))
        return PS_ERR_INVALID_ARG;
    if (n_rows == 0) return PS_OK;
    if (!x || !aligned(x, 16) || x_ld < h->K || x_ld % 8 != 0 || x_ld > std::min(kMostSpan / n_rows, kMostStride)) return PS_ERR_INVALID_ARG;
    ps_status st = check_rows_layout(out, h->N, dtype, ld);
    if (st != PS_OK) return st;
    if (residual) {
        st = check_rows_layout(residual, h->N, dtype, residual_ld);
        if (st != PS_OK) return st;
    }
    if (ld > kMostSpan / n_rows || (residual && residual_ld > kMostSpan / n_rows)) return PS_ERR_INVALID_ARG;
    const int64_t n_out = ((n_rows - 1) * ld + h->N) * esz;
    if (overlap(out, n_out, x, ((n_rows - 1) * x_ld + h->K) * 2) ||
        overlap(out, n_out, h->w, ((h->N - 1) * h->w_ld + h->K) * 2) ||
        (h->bias && overlap(out, n_out, h->bias, (int64_t)h->N * elem_size(h->bias_dtype))))
        return PS_ERR_INVALID_ARG;
    if (residual && (residual == out ? residual_ld != ld
                                     : overlap(out, n_out, residual, ((n_rows - 1) * residual_ld + h->N) * esz)))
        return PS_ERR_INVALID_ARG;
    if (!all_on_device({x, h->w, h->bias, residual})) return PS_ERR_INVALID_ARG;
    int sms = 0;
    st = device_of(out, &sms);
    if (st != PS_OK) return st;
    LinearParams p{};
    p.lin = *h;
    p.x = x;
    p.x_ld = x_ld;
    p.n_rows = n_rows;
    p.dtype = dtype;
    p.residual = residual;
    p.residual_ld = residual_ld;
    p.out = out;
    p.ld = ld;
    return map_cuda(launch_linear(p, sms, lost, (cudaStream_t)cuda_stream));
}

}  // namespace

extern "C" {

ps_status ps_linear_rows(const ps_linear *linear, const void *x, int64_t x_ld, int32_t n_rows,
                         const void *residual, int64_t residual_ld, void *out, int64_t ld,
                         int32_t dtype, void *cuda_stream) {
    return linear_rows(linear, x, x_ld, n_rows, residual, residual_ld, out, ld, dtype, false, cuda_stream);
}

ps_status ps_selftest_linear_wait(const ps_linear *linear, const void *x, int64_t x_ld, int32_t n_rows,
                                  const void *residual, int64_t residual_ld, void *out, int64_t ld,
                                  int32_t dtype, void *cuda_stream) {
    return linear_rows(linear, x, x_ld, n_rows, residual, residual_ld, out, ld, dtype, true, cuda_stream);
}

ps_status ps_sample_rows(const ps_sampling *sampling, int32_t V, int32_t dtype, int64_t n_rows,
                         const void *logits, int64_t ld, const double *u, int32_t *tokens,
                         double *lp0, double *lq, double *entropy, int32_t *status,
                         void *cuda_stream) {
    if (n_rows < 0 || V < 1 || !status) return PS_ERR_INVALID_ARG;
    const int esz = elem_size(dtype);
    if (esz == 0) return PS_ERR_UNSUPPORTED;
    ps_status st = check_sampling_host(sampling, V, n_rows);
    if (st != PS_OK || n_rows == 0) return st;
    st = check_rows_layout(logits, V, dtype, ld);
    if (st != PS_OK) return st;
    if (!u || !tokens || n_rows > (int64_t(1) << 62) / ld / esz) return PS_ERR_INVALID_ARG;
    if (!aligned(u, 8) || !aligned(tokens, 4) || !aligned(lp0, 8) || !aligned(lq, 8) || !aligned(entropy, 8) || !aligned(status, 4))
        return PS_ERR_INVALID_ARG;
    if (!all_on_device({u, tokens, lp0, lq, entropy, status}) || !sampling_on_device(sampling)) return PS_ERR_INVALID_ARG;
    int sms = 0;
    st = device_of(logits, &sms);
    if (st != PS_OK) return st;
    SampleParams p{};
    p.set = *sampling;
    p.logits = (const uint8_t *)logits;
    p.ld_bytes = ld * esz;
    p.n_logit_rows = n_rows;
    p.n_rows = n_rows;
    p.V = V;
    p.dtype = dtype;
    p.u = u;
    p.drawn = tokens;
    p.lp0 = lp0;
    p.lq = lq;
    p.entropy = entropy;
    p.status = status;
    return map_cuda(launch_sample(p, sms, (cudaStream_t)cuda_stream));
}

ps_status ps_score_rows_truncated(const ps_subtree_batch *b, const ps_sampling *sampling,
                                  double *lp0, double *lq, double *entropy, int32_t *status,
                                  void *cuda_stream) {
    ps_status st = check_batch_host(b);
    if (st != PS_OK) return st;
    if (!status || (b->n_rows > 0 && (!lp0 || !lq))) return PS_ERR_INVALID_ARG;
    st = check_sampling_host(sampling, b->V, b->n_rows);
    if (st != PS_OK || b->n_rows == 0) return st;
    if (!aligned(b->tokens, 4) || !aligned(b->row_index, 8) || !aligned(lp0, 8) || !aligned(lq, 8) || !aligned(entropy, 8) ||
        !aligned(status, 4))
        return PS_ERR_INVALID_ARG;
    if (!all_on_device({b->tokens, b->row_index, lp0, lq, entropy, status}) || !sampling_on_device(sampling))
        return PS_ERR_INVALID_ARG;
    int sms = 0;
    st = device_of(b->logits, &sms);
    if (st != PS_OK) return st;
    SampleParams p{};
    p.set = *sampling;
    p.logits = (const uint8_t *)b->logits;
    p.ld_bytes = b->ld * elem_size(b->dtype);
    p.row_index = b->row_index;
    p.n_logit_rows = b->row_index ? b->n_logit_rows : b->n_rows;
    p.n_rows = b->n_rows;
    p.V = b->V;
    p.dtype = b->dtype;
    p.tokens = b->tokens;
    p.lp0 = lp0;
    p.lq = lq;
    p.entropy = entropy;
    p.status = status;
    return map_cuda(launch_sample(p, sms, (cudaStream_t)cuda_stream));
}

}  // extern "C"
