// C entry points of linear attention and of the 8-bit state cache: argument
// checks, roles of the recurrences, launch order.  Declared in include/ssd.h.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "ssd.h"
#include "ssd_linear_attn.hpp"

namespace {

using ssd::la::Op;
using ssd::la::Params;
using ssd::la::Rows;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRow = 1 << 22;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

bool dim_ok(int d) { return d <= SSD_LINEAR_ATTN_MAX_DIM && d % 8 == 0; }

ssd_status check(const ssd_linear_attn_problem *p) {
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len < 0 || p->total_len > INT32_MAX || p->batch < 1 || p->nheads < 1 || p->ngroups < 1 ||
        p->key_dim < 1 || p->value_dim < 1 || p->max_slots < 1 || p->nheads % p->ngroups != 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->state_dtype != SSD_STATE_F32 && p->state_dtype != SSD_STATE_BF16) return SSD_ERR_UNSUPPORTED;
    if (!dim_ok(p->key_dim) || !dim_ok(p->value_dim)) return SSD_ERR_UNSUPPORTED;
    // numbers of workgroups are ints (up to 4 blocks of channels, 3 recurrences); threads are counted with the layout
    if (((int64_t)p->batch + p->total_len / 256) * p->nheads > INT32_MAX / 64) return SSD_ERR_UNSUPPORTED;
    if (!isfinite(p->scale)) return SSD_ERR_UNSUPPORTED;
    const int64_t qk = (int64_t)p->ngroups * p->key_dim, vv = (int64_t)p->nheads * p->value_dim;
    const int64_t strides[3] = {p->q_stride, p->k_stride, p->v_stride}, rows[3] = {qk, qk, vv};
    for (int i = 0; i < 3; ++i)
        if (strides[i] != 0 && (strides[i] < rows[i] || strides[i] % 8 != 0)) return SSD_ERR_BAD_SHAPE;
    for (int i = 0; i < 3; ++i)  // 64 rows are addressed with 31 bits
        if ((strides[i] != 0 ? strides[i] : rows[i]) > kMaxRow) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)p->nheads * p->key_dim > kMaxRow) return SSD_ERR_UNSUPPORTED;  // gradients before heads are summed
    return SSD_OK;
}

int64_t stride_or(int64_t s, int64_t dense) { return s != 0 ? s : dense; }

// Workspace: the segments' states of a launch, and in the backward pass fp32
// dq and dk per head, where several heads share a row of q and k.
struct Layout {
    ssd::la::Shape shape;
    bool shared;
    size_t dq, dk, bytes;  // the segments' states come first
    int64_t threads;       // of the largest launch
};
Layout layout_of(const ssd_linear_attn_problem *p, bool backward) {
    Layout L = {};
    // dq, dk and dv share one launch, which holds the wider of K and V for all
    // (apart, dv and the others leave the card half empty: packed documents with
    // K 96, V 200 582 us instead of 413)
    const int K = p->key_dim, V = p->value_dim, o[1] = {V}, grads[3] = {K, V, K};
    const int share = p->nheads / p->ngroups;
    if (backward)
        L.shape = ssd::la::shape_of(p->total_len, p->batch, p->nheads, share, K > V ? K : V, grads, 3, 2);
    else
        L.shape = ssd::la::shape_of(p->total_len, p->batch, p->nheads, share, K, o, 1, 1);
    L.bytes = align_up(L.shape.bytes);
    L.threads = L.shape.threads;
    L.shared = backward && p->nheads != p->ngroups;
    if (L.shared) {
        L.threads = std::max(L.threads, p->total_len * p->ngroups * (p->key_dim / 8) + 255);
        const size_t n = align_up((size_t)p->total_len * p->nheads * p->key_dim * sizeof(float));
        L.dq = L.bytes;
        L.dk = L.dq + n;
        L.bytes = L.dk + n;
    }
    return L;
}

ssd_status check_workspace(const Layout &L, const void *ws, size_t bytes) {
    if (L.bytes == 0) return SSD_OK;
    return ws == nullptr || bytes < L.bytes || !aligned(ws, kAlign) ? SSD_ERR_WORKSPACE : SSD_OK;
}

Params common(const ssd_linear_attn_problem *p, const float *log_decay, const int32_t *qsl) {
    Params q;
    memset(&q, 0, sizeof q);
    q.T = p->total_len;
    q.batch = p->batch;
    q.H = p->nheads;
    q.share = p->nheads / p->ngroups;
    q.state_size = p->key_dim * p->value_dim;
    q.state_bf16 = p->state_dtype == SSD_STATE_BF16;
    q.log_decay = log_decay;
    q.qsl = qsl;
    q.max_slots = (uint32_t)p->batch;
    return q;
}

Rows group_rows(const ssd_linear_attn_problem *p, const void *ptr, int64_t stride) {
    return Rows{static_cast<const uint16_t *>(ptr), stride_or(stride, (int64_t)p->ngroups * p->key_dim),
                p->nheads / p->ngroups};
}
Rows head_rows(const ssd_linear_attn_problem *p, const void *ptr, int64_t stride) {
    return Rows{static_cast<const uint16_t *>(ptr), stride_or(stride, (int64_t)p->nheads * p->value_dim), 1};
}

ssd_status forward(const ssd_linear_attn_problem *p, void *o, const void *q, const void *k, const void *v,
                   const float *log_decay, const void *state_in, void *state_out, const int32_t *qsl,
                   const uint8_t *has_init, const uint32_t *cache_idx, bool init_all, void *ws, size_t ws_bytes,
                   void *stream) {
    const ssd_status st = check(p);
    if (st != SSD_OK) return st;
    if (log_decay == nullptr || state_out == nullptr || qsl == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len > 0 && (o == nullptr || q == nullptr || k == nullptr || v == nullptr)) return SSD_ERR_NULL_ARG;
    if (!aligned(o, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(state_in, 16) ||
        !aligned(state_out, 16) || !aligned(log_decay, 4) || !aligned(qsl, 4) || !aligned(cache_idx, 4))
        return SSD_ERR_MISALIGNED;
    const Layout L = layout_of(p, false);
    if (L.threads > UINT32_MAX) return SSD_ERR_UNSUPPORTED;
    const ssd_status sw = check_workspace(L, ws, ws_bytes);
    if (sw != SSD_OK) return sw;

    Params a = common(p, log_decay, qsl);
    a.parts = static_cast<float *>(ws);
    a.has_init = has_init;
    a.cache_idx = cache_idx;
    a.init_all = init_all;
    if (cache_idx != nullptr) a.max_slots = (uint32_t)p->max_slots;
    Op &op = a.op[0];
    op.q = group_rows(p, q, p->q_stride);
    op.k = group_rows(p, k, p->k_stride);
    op.v = head_rows(p, v, p->v_stride);
    op.out = o;
    op.kd = p->key_dim;
    op.vd = p->value_dim;
    op.scale_pair = op.scale_state = p->scale;
    op.scale_update = 1.f;
    op.state_in = state_in;
    op.state_out = state_out;
    op.sv = p->key_dim;
    op.sk = 1;
    return ssd::la::launch_walk(a, L.shape, 1, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd::CacheParams cache_params(const ssd_state_cache_problem *p, const uint32_t *pool_idx, const uint32_t *entry_idx) {
    return ssd::CacheParams{pool_idx, entry_idx, (int64_t)p->nheads * p->head_dim, p->count, p->dstate,
                            (uint32_t)p->max_slots, (uint32_t)p->max_entries};
}

ssd_status check_cache(const ssd_state_cache_problem *p, const void *codes, const void *scales, const void *pool,
                       const void *pool_idx, const void *entry_idx) {
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->count < 0 || p->nheads < 1 || p->head_dim < 1 || p->dstate < 1 || p->max_slots < 1 || p->max_entries < 1)
        return SSD_ERR_BAD_SHAPE;
    if (p->state_dtype != SSD_STATE_F32 && p->state_dtype != SSD_STATE_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->code_format != SSD_CODE_I8 && p->code_format != SSD_CODE_E4M3) return SSD_ERR_UNSUPPORTED;
    if (p->dstate > SSD_MAX_DSTATE || p->dstate % 8 != 0) return SSD_ERR_UNSUPPORTED;
    // blocks and threads of the launches (a block holds at least 16 rows)
    if (((int64_t)p->nheads * p->head_dim + 15) / 16 > INT32_MAX / (p->count > 0 ? p->count : 1) ||
        ssd::state_cache_threads(cache_params(p, nullptr, nullptr), p->state_dtype == SSD_STATE_BF16) > UINT32_MAX)
        return SSD_ERR_UNSUPPORTED;
    if (p->count > 0 && (codes == nullptr || scales == nullptr || pool == nullptr || pool_idx == nullptr ||
                         entry_idx == nullptr))
        return SSD_ERR_NULL_ARG;
    if (!aligned(pool, 16) || !aligned(codes, 8) || !aligned(scales, 4) || !aligned(pool_idx, 4) ||
        !aligned(entry_idx, 4))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_linear_attn_workspace_size(const ssd_linear_attn_problem *prob, int backward, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_NULL_ARG;
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    const Layout L = layout_of(prob, backward != 0);
    if (L.threads > UINT32_MAX) return SSD_ERR_UNSUPPORTED;
    *bytes = L.bytes;
    return SSD_OK;
}

ssd_status ssd_linear_attn_varlen_fwd_inplace(
    const ssd_linear_attn_problem *prob, void *o, const void *q, const void *k, const void *v,
    const float *log_decay, void *pool, const int32_t *query_start_loc, const uint8_t *has_initial_state,
    const uint32_t *cache_indices, void *workspace, size_t workspace_bytes, void *stream) {
    if (cache_indices == nullptr) return SSD_ERR_NULL_ARG;
    return forward(prob, o, q, k, v, log_decay, pool, pool, query_start_loc, has_initial_state, cache_indices, false,
                   workspace, workspace_bytes, stream);
}

ssd_status ssd_linear_attn_varlen_fwd(
    const ssd_linear_attn_problem *prob, void *o, const void *q, const void *k, const void *v,
    const float *log_decay, const void *initial_states, void *final_states, const int32_t *query_start_loc,
    void *workspace, size_t workspace_bytes, void *stream) {
    return forward(prob, o, q, k, v, log_decay, initial_states, final_states, query_start_loc, nullptr, nullptr, true,
                   workspace, workspace_bytes, stream);
}

ssd_status ssd_linear_attn_varlen_bwd(
    const ssd_linear_attn_problem *prob, void *dq, void *dk, void *dv, void *d_initial, const void *q, const void *k,
    const void *v, const void *d_o, const float *log_decay, const void *initial_states, const void *d_final,
    const int32_t *query_start_loc, void *workspace, size_t workspace_bytes, void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (log_decay == nullptr || query_start_loc == nullptr) return SSD_ERR_NULL_ARG;
    if (prob->total_len > 0 && (dq == nullptr || dk == nullptr || dv == nullptr || q == nullptr || k == nullptr ||
                                v == nullptr || d_o == nullptr))
        return SSD_ERR_NULL_ARG;
    if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(d_initial, 16) || !aligned(q, 16) ||
        !aligned(k, 16) || !aligned(v, 16) || !aligned(d_o, 16) || !aligned(initial_states, 16) ||
        !aligned(d_final, 16) || !aligned(log_decay, 4) || !aligned(query_start_loc, 4))
        return SSD_ERR_MISALIGNED;
    const Layout L = layout_of(prob, true);
    if (L.threads > UINT32_MAX) return SSD_ERR_UNSUPPORTED;
    const ssd_status sw = check_workspace(L, workspace, workspace_bytes);
    if (sw != SSD_OK) return sw;
    // dq reads initial_states in the launch in which dv writes d_initial
    if (d_initial != nullptr && d_initial == initial_states) return SSD_ERR_UNSUPPORTED;

    const ssd_linear_attn_problem *p = prob;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool shared = L.shared;
    char *ws = static_cast<char *>(workspace);
    const Rows rq = group_rows(p, q, p->q_stride), rk = group_rows(p, k, p->k_stride);
    const Rows rv = head_rows(p, v, p->v_stride), rg = head_rows(p, d_o, 0);
    Params a = common(p, log_decay, query_start_loc);
    a.init_all = 1;
    a.parts = reinterpret_cast<float *>(ws);
    Op &oq = a.op[0], &ok = a.op[1], &ov = a.op[2];
    // dq: the forward chain, with the state transposed
    oq.q = rg;
    oq.k = rv;
    oq.v = rk;
    oq.out = shared ? ws + L.dq : dq;
    oq.out_f32 = shared;
    oq.kd = p->value_dim;
    oq.vd = p->key_dim;
    oq.scale_pair = oq.scale_state = p->scale;
    oq.scale_update = 1.f;
    oq.state_in = initial_states;
    oq.sv = 1;
    oq.sk = p->key_dim;
    // dk and dv: the reverse chain, which takes the scale as it is summed
    ok = oq;
    ok.q = rv;
    ok.k = rg;
    ok.v = rq;
    ok.out = shared ? ws + L.dk : dk;
    ok.reverse = 1;
    ok.scale_state = 1.f;
    ok.scale_update = p->scale;
    ok.state_in = d_final;
    ov = ok;
    ov.q = rk;
    ov.k = rq;
    ov.v = rg;
    ov.out = dv;
    ov.out_f32 = 0;
    ov.kd = p->key_dim;
    ov.vd = p->value_dim;
    ov.sv = p->key_dim;
    ov.sk = 1;
    ov.state_out = d_initial;
    if (d_initial != nullptr && d_initial == d_final) {
        // dv overwrites d_final, which dk reads too, with d_initial: dv last
        Params b = a;
        b.op[0] = ov;
        if (ssd::la::launch_walk(a, L.shape, 2, s) != hipSuccess ||
            ssd::la::launch_walk(b, L.shape, 1, s) != hipSuccess)
            return SSD_ERR_HIP;
    } else {
        ok.twin = 1;
        ov.mirror = 1;
        if (ssd::la::launch_walk(a, L.shape, 3, s) != hipSuccess) return SSD_ERR_HIP;
    }
    if (shared && p->total_len > 0) {
        const int div = p->nheads / p->ngroups;
        const ssd::la::GroupSum sums = {
            {reinterpret_cast<const float *>(ws + L.dq), reinterpret_cast<const float *>(ws + L.dk)},
            {static_cast<uint16_t *>(dq), static_cast<uint16_t *>(dk)}};
        if (ssd::la::launch_group_sum(sums, a, div, p->key_dim, s) != hipSuccess) return SSD_ERR_HIP;
    }
    return SSD_OK;
}

ssd_status ssd_linear_attn_step_inplace(
    const ssd_linear_attn_problem *prob, void *o, const void *q, const void *k, const void *v,
    const float *log_decay, void *pool, const uint8_t *has_initial_state, const uint32_t *cache_indices,
    void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (prob->total_len != prob->batch) return SSD_ERR_BAD_SHAPE;
    if ((int64_t)prob->batch * prob->nheads > UINT32_MAX / 256) return SSD_ERR_UNSUPPORTED;  // 256 threads each
    if (o == nullptr || q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || pool == nullptr ||
        cache_indices == nullptr)
        return SSD_ERR_NULL_ARG;
    if (!aligned(o, 2) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 2) || !aligned(pool, 16) ||
        !aligned(log_decay, 4) || !aligned(cache_indices, 4))
        return SSD_ERR_MISALIGNED;
    const Rows rq = group_rows(prob, q, prob->q_stride), rk = group_rows(prob, k, prob->k_stride);
    const Rows rv = head_rows(prob, v, prob->v_stride);
    ssd::la::StepParams a;
    a.q = rq.p;
    a.k = rk.p;
    a.v = rv.p;
    a.qs = rq.stride;
    a.ks = rk.stride;
    a.vs = rv.stride;
    a.o = static_cast<uint16_t *>(o);
    a.log_decay = log_decay;
    a.pool = pool;
    a.has_init = has_initial_state;
    a.cache_idx = cache_indices;
    a.batch = prob->batch;
    a.H = prob->nheads;
    a.div = rq.div;
    a.K = prob->key_dim;
    a.V = prob->value_dim;
    a.max_slots = (uint32_t)prob->max_slots;
    a.state_bf16 = prob->state_dtype == SSD_STATE_BF16;
    a.scale = prob->scale;
    return ssd::la::launch_step(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_state_quantize(const ssd_state_cache_problem *prob, void *codes, float *scales, const void *pool,
                              const uint32_t *pool_indices, const uint32_t *entry_indices, void *stream) {
    const ssd_status st = check_cache(prob, codes, scales, pool, pool_indices, entry_indices);
    if (st != SSD_OK || prob->count == 0) return st;
    return ssd::launch_state_quantize(cache_params(prob, pool_indices, entry_indices), pool,
                                      prob->state_dtype == SSD_STATE_BF16, prob->code_format == SSD_CODE_E4M3, codes,
                                      scales, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

ssd_status ssd_state_dequantize(const ssd_state_cache_problem *prob, void *pool, const void *codes,
                                const float *scales, const uint32_t *pool_indices, const uint32_t *entry_indices,
                                void *stream) {
    const ssd_status st = check_cache(prob, codes, scales, pool, pool_indices, entry_indices);
    if (st != SSD_OK || prob->count == 0) return st;
    return ssd::launch_state_dequantize(cache_params(prob, pool_indices, entry_indices), pool,
                                        prob->state_dtype == SSD_STATE_BF16, prob->code_format == SSD_CODE_E4M3,
                                        codes, scales, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK
               : SSD_ERR_HIP;
}

}  // extern "C"
