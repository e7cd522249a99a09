// Host side of the entry points around the rows: rules on logits rows and the
// 4-bit output head.  See include/ps.h for the contract.
#include "ps_api.cuh"
#include "ps_head.cuh"
#include "ps_rules.cuh"

using namespace ps;

namespace {

// A matrix of rows as the logits of a batch are laid out.
ps_status check_rows_layout(const void *p, int32_t V, int32_t dtype, int64_t ld) {
    const int esz = elem_size(dtype);
    if (esz == 0) return PS_ERR_UNSUPPORTED;
    if (V < 1 || ld < V || ld > (int64_t(1) << 40)) return PS_ERR_INVALID_ARG;
    const int64_t row_bytes = ((int64_t)V * esz + 15) / 16 * 16;
    if (row_bytes > (int64_t(1) << 30)) return PS_ERR_INVALID_ARG;
    if ((ld * esz) % 16 != 0 || !p || !aligned(p, 16)) return PS_ERR_INVALID_ARG;
    return PS_OK;
}

// What the host can see of the rules.
ps_status check_rules_host(const ps_logit_rules *u, int32_t V, int64_t n_rows) {
    if (!u || u->n_seqs < 0 || u->n_masks < 0 || u->n_tokens < 0 || u->n_bias < 0)
        return PS_ERR_INVALID_ARG;
    if (u->seq_begin && u->n_tokens > 0 && !u->seq_tokens) return PS_ERR_INVALID_ARG;
    if (u->bias_begin && u->n_bias > 0 && (!u->bias_ids || !u->bias_values))
        return PS_ERR_INVALID_ARG;
    if ((u->seq_begin || u->bias_begin) && !u->row_seq && u->n_seqs < n_rows)
        return PS_ERR_INVALID_ARG;
    if (u->mask) {
        if (u->mask_ld < ((int64_t)V + 31) / 32 || !aligned(u->mask, 4)) return PS_ERR_INVALID_ARG;
        if (!u->row_mask && u->n_masks < n_rows) return PS_ERR_INVALID_ARG;
    }
    return PS_OK;
}

// Workspace of ps_score_rows_rules.  Its size is what the most demanding batch of up to
// as many rows takes, so that one for the largest batch serves all.
struct ScoreWs {
    RuleCut cut;
    size_t tok_off, bad_off, total;
};

ScoreWs score_ws(const ps_subtree_batch *b) {
    ScoreWs w;
    w.cut = score_cut(b->V, b->dtype, b->n_rows);
    const size_t n = (size_t)b->n_rows;
    w.tok_off = align_up(n * w.cut.n_slices * kScoreParts * sizeof(ChunkPart), kAlign);
    w.bad_off = w.tok_off + align_up(n * sizeof(float), kAlign);
    w.total = align_up((size_t)score_slices(b->V, b->dtype, b->n_rows) * kScoreParts * sizeof(ChunkPart), kAlign) +
              align_up(n * sizeof(float), kAlign) + align_up(n * sizeof(int32_t), kAlign);
    return w;
}

// What the host can see of a head's call; its parameters, for n_rows > 0.
ps_status head_params(const ps_head *h, const void *hidden, int64_t hidden_ld, int32_t n_rows, void *logits,
                      int64_t ld, int32_t dtype, HeadParams *p, int *sms) {
    if (!h || n_rows < 0 || h->V < 1 || h->K < 1) return PS_ERR_INVALID_ARG;
    if (elem_size(h->scale_dtype) == 0 || elem_size(dtype) == 0) return PS_ERR_UNSUPPORTED;
    if (h->group != 32 && h->group != 64 && (h->group < 128 || h->group % 128 != 0))
        return PS_ERR_UNSUPPORTED;
    if (h->K % h->group != 0 || !h->q || !h->scales || !aligned(h->q, 16) ||
        !aligned(h->scales, (size_t)elem_size(h->scale_dtype)))
        return PS_ERR_INVALID_ARG;
    if (n_rows == 0) return PS_OK;
    if (!hidden || !aligned(hidden, 16) || hidden_ld < h->K || hidden_ld % 8 != 0 ||
        hidden_ld > (int64_t(1) << 40))
        return PS_ERR_INVALID_ARG;
    ps_status st = check_rows_layout(logits, h->V, dtype, ld);
    if (st != PS_OK) return st;
    if (!on_device(hidden) || !on_device(h->q)) return PS_ERR_INVALID_ARG;
    st = device_of(logits, sms);
    if (st != PS_OK) return st;
    p->head = *h;
    p->hidden = (const uint16_t *)hidden;
    p->hidden_ld = hidden_ld;
    p->n_rows = n_rows;
    p->logits = logits;
    p->ld = ld;
    p->dtype = dtype;
    return PS_OK;
}

}  // namespace

extern "C" {

ps_status ps_process_rows(const ps_logit_rules *rules, int32_t V, int32_t dtype, int64_t n_rows,
                          const void *logits, int64_t ld, void *out, int64_t out_ld,
                          int32_t *status, void *cuda_stream) {
    if (n_rows < 0 || !status) return PS_ERR_INVALID_ARG;
    if (n_rows == 0) {
        if (elem_size(dtype) == 0) return PS_ERR_UNSUPPORTED;
        return V < 1 ? PS_ERR_INVALID_ARG : check_rules_host(rules, V, 0);
    }
    ps_status st = check_rows_layout(logits, V, dtype, ld);
    if (st != PS_OK) return st;
    st = check_rows_layout(out, V, dtype, out_ld);
    if (st != PS_OK) return st;
    st = check_rules_host(rules, V, n_rows);
    if (st != PS_OK) return st;
    const int esz = elem_size(dtype);
    if (n_rows > (int64_t(1) << 62) / (ld > out_ld ? ld : out_ld) / esz) return PS_ERR_INVALID_ARG;
    const uint8_t *a = (const uint8_t *)logits, *b = (const uint8_t *)out;
    const int64_t na = ((n_rows - 1) * ld + V) * esz, nb = ((n_rows - 1) * out_ld + V) * esz;
    if (a == b ? ld != out_ld : (a < b + nb && b < a + na)) return PS_ERR_INVALID_ARG;
    int sms = 0;
    if (a != b && !on_device(logits)) return PS_ERR_INVALID_ARG;
    st = device_of(out, &sms);
    if (st != PS_OK) return st;
    ProcessParams p{};
    p.r.rules = *rules;
    p.r.n_rows = n_rows;
    p.r.V = V;
    p.r.status = status;
    p.logits = a;
    p.out = (uint8_t *)out;
    p.ld_bytes = ld * esz;
    p.out_ld_bytes = out_ld * esz;
    return map_cuda(launch_process_rows(p, dtype, sms, (cudaStream_t)cuda_stream));
}

size_t ps_rules_workspace_bytes(const ps_subtree_batch *b) {
    if (!b || b->n_rows <= 0 || b->V < 1 || elem_size(b->dtype) == 0) return kAlign;
    return score_ws(b).total;
}

ps_status ps_score_rows_rules(const ps_subtree_batch *b, const ps_logit_rules *rules, double *lp0,
                              double *lq, double *entropy, int32_t *status, void *workspace,
                              size_t workspace_bytes, void *cuda_stream) {
    ps_status st = check_batch_host(b);
    if (st != PS_OK) return st;
    if (!status || (b->n_rows > 0 && (!lp0 || !lq))) return PS_ERR_INVALID_ARG;
    st = check_rules_host(rules, b->V, b->n_rows);
    if (st != PS_OK) return st;
    if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < ps_rules_workspace_bytes(b))
        return PS_ERR_WORKSPACE;
    if (b->n_rows == 0) return PS_OK;
    int sms = 0;
    st = device_of(b->logits, &sms);
    if (st != PS_OK) return st;
    ScoreRulesParams p{};
    p.r.rules = *rules;
    p.r.n_rows = b->n_rows;
    p.r.V = b->V;
    p.r.status = status;
    const ScoreWs ws = score_ws(b);
    p.cut = ws.cut;
    p.parts = (ChunkPart *)workspace;
    p.tok_logit = (float *)((uint8_t *)workspace + ws.tok_off);
    p.row_bad = (int32_t *)((uint8_t *)workspace + ws.bad_off);
    RowsParams &q = p.rows;
    const int esz = elem_size(b->dtype);
    q.logits = (const uint8_t *)b->logits;
    q.ld_bytes = b->ld * esz;
    q.n_logit_rows = b->row_index ? b->n_logit_rows : b->n_rows;
    q.row_index = b->row_index;
    q.tokens = b->tokens;
    q.n_rows = b->n_rows;
    q.V = b->V;
    q.dtype = b->dtype;
    q.flags = b->flags;
    q.npow = integer_power(b->tau);
    q.g = (float)(1.0 / b->tau);
    q.lp0 = lp0;
    q.lq = lq;
    q.entropy = entropy;
    q.status = status;
    return map_cuda(launch_score_rules(p, sms, (cudaStream_t)cuda_stream));
}

ps_status ps_head_rows(const ps_head *h, const void *hidden, int64_t hidden_ld, int32_t n_rows,
                       void *logits, int64_t ld, int32_t dtype, void *cuda_stream) {
    HeadParams p{};
    int sms = 0;
    const ps_status st = head_params(h, hidden, hidden_ld, n_rows, logits, ld, dtype, &p, &sms);
    if (st != PS_OK || n_rows == 0) return st;
    return map_cuda(launch_head_rows(p, sms, (cudaStream_t)cuda_stream));
}

ps_status ps_selftest_head_wait(const ps_head *h, const void *hidden, int64_t hidden_ld, int32_t n_rows,
                                void *logits, int64_t ld, int32_t dtype, void *cuda_stream) {
    if (!h || n_rows < 33 || n_rows > 64 || h->K < 256 || h->K > 2048 || h->group < 128 ||
        h->scale_dtype != PS_BF16)
        return PS_ERR_INVALID_ARG;
    HeadParams p{};
    int sms = 0;
    const ps_status st = head_params(h, hidden, hidden_ld, n_rows, logits, ld, dtype, &p, &sms);
    if (st != PS_OK) return st;
    return map_cuda(launch_head_lost(p, sms, (cudaStream_t)cuda_stream));
}

}  // extern "C"
