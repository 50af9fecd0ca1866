// C entry points of the norm, the short convolution and the selective scan:
// argument checks, workspaces, launch order.  Declared in include/ssd.h.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "ssd.h"
#include "ssd_layer.hpp"

namespace {

using ssd::layer::ConvParams;
using ssd::layer::NormGradParams;
using ssd::layer::NormParams;
using ssd::layer::ScanParams;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRow = 1 << 22;        // elements from one row to the next
constexpr int64_t kMaxTokens = (1 << 30) - 1;  // so that a token's number and a tile or a segment fit 32 bits
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }
template <typename... P>
bool all_aligned(size_t a, P... ptr) { return (aligned(ptr, a) && ...); }
bool stride_ok(int64_t s, int64_t row, int64_t step) { return s == 0 || (s >= row && s % step == 0); }
int64_t stride_or(int64_t s, int64_t dense) { return s != 0 ? s : dense; }
ssd_status launched(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }
ssd_status check_workspace(size_t need, const void *ws, size_t bytes) {
    if (need == 0) return SSD_OK;
    return ws == nullptr || bytes < need || !aligned(ws, kAlign) ? SSD_ERR_WORKSPACE : SSD_OK;
}

// ---------------------------------------------------------------- norm

ssd_status check(const ssd_norm_problem *p) {
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->rows < 0 || p->width < 1 || !stride_ok(p->x_stride, p->width, 8)) return SSD_ERR_BAD_SHAPE;
    if (p->width > SSD_NORM_MAX_WIDTH || p->width % 8 != 0) return SSD_ERR_UNSUPPORTED;
    if (p->residual_dtype != SSD_STATE_F32 && p->residual_dtype != SSD_STATE_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->out_format != SSD_OUT_BF16 && p->out_format != SSD_CODE_I8 && p->out_format != SSD_CODE_E4M3)
        return SSD_ERR_UNSUPPORTED;
    if (!(p->eps >= 0.f) || !isfinite(p->eps)) return SSD_ERR_UNSUPPORTED;
    if (p->x_stride > kMaxRow || ssd::layer::norm_threads(p->rows, p->width) > UINT32_MAX) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// ---------------------------------------------------------------- convolution

ssd_status check(const ssd_conv_problem *p) {
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len < 0 || p->total_len > INT32_MAX || p->batch < 1 || p->channels < 1 || p->max_slots < 1 ||
        !stride_ok(p->x_stride, p->channels, 8))
        return SSD_ERR_BAD_SHAPE;
    if (p->width < 2 || p->width > SSD_CONV_MAX_WIDTH || p->channels % 8 != 0) return SSD_ERR_UNSUPPORTED;
    if (p->total_len > kMaxTokens || std::max<int64_t>(p->x_stride, p->channels) > kMaxRow) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
ConvParams common(const ssd_conv_problem *p) {
    ConvParams a;
    memset(&a, 0, sizeof a);
    a.T = (int)p->total_len;
    a.batch = p->batch;
    a.D = p->channels;
    a.xs = stride_or(p->x_stride, p->channels);
    a.silu = p->silu != 0;
    a.max_slots = (uint32_t)p->batch;
    return a;
}
// Whether the dense rows [rows][width] at `a` share memory with as many of that width at `b`, `stride` elements apart
bool rows_meet(const void *a, const void *b, int64_t rows, int64_t width, int64_t stride) {
    const int64_t row = width * 2, step = stride * 2, begin = (int64_t)(uintptr_t)a - (int64_t)(uintptr_t)b;
    const int64_t r = begin < row ? 0 : (begin - row) / step + 1;  // the first at b that ends behind a's begin
    return r < rows && r * step < begin + rows * row;
}
bool fits(const ConvParams &a) { return a.places <= INT32_MAX && conv_threads(a) <= UINT32_MAX; }

ssd_status conv_forward(const ssd_conv_problem *p, void *y, const void *x, const float *weight, const float *bias,
                        const void *state_in, void *state_out, const int32_t *qsl, const uint8_t *has_init,
                        const uint32_t *cache_idx, bool init_all, void *stream) {
    const ssd_status st = check(p);
    if (st != SSD_OK) return st;
    if (weight == nullptr || state_out == nullptr || qsl == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len > 0 && (y == nullptr || x == nullptr)) return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, y, x, weight, bias, state_in, state_out) || !all_aligned(4, qsl, cache_idx))
        return SSD_ERR_MISALIGNED;
    ConvParams a = common(p);
    conv_shape(a, p->width, false);
    if (!fits(a)) return SSD_ERR_UNSUPPORTED;
    // a piece reads the rows ahead of it, which another workgroup writes in y
    if (rows_meet(y, x, a.T, a.D, a.xs)) return SSD_ERR_UNSUPPORTED;
    a.y = static_cast<uint16_t *>(y);
    a.x = static_cast<const uint16_t *>(x);
    a.weight = weight;
    a.bias = bias;
    a.state_in = static_cast<const uint16_t *>(state_in);
    a.state_out = static_cast<uint16_t *>(state_out);
    a.qsl = qsl;
    a.has_init = has_init;
    a.cache_idx = cache_idx;
    a.init_all = init_all;
    if (cache_idx != nullptr) a.max_slots = (uint32_t)p->max_slots;
    return launched(launch_conv(a, p->width, static_cast<hipStream_t>(stream)));
}

size_t conv_workspace(const ConvParams &a, int width) {
    return align_up((size_t)conv_parts(a) * (size_t)(width + 1) * (size_t)a.D * sizeof(float));
}

// ---------------------------------------------------------------- selective scan

ssd_status check(const ssd_selective_problem *p) {
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len < 0 || p->total_len > INT32_MAX || p->batch < 1 || p->channels < 1 || p->ngroups < 1 ||
        p->dstate < 1 || p->max_slots < 1 || p->channels % p->ngroups != 0)
        return SSD_ERR_BAD_SHAPE;
    const int64_t bc = (int64_t)p->ngroups * p->dstate;
    if (!stride_ok(p->x_stride, p->channels, 8) || !stride_ok(p->dt_stride, p->channels, 8) ||
        !stride_ok(p->z_stride, p->channels, 8) || !stride_ok(p->b_stride, bc, 2) || !stride_ok(p->c_stride, bc, 2))
        return SSD_ERR_BAD_SHAPE;
    if (p->dstate > SSD_SELECTIVE_MAX_DSTATE || p->dstate % 4 != 0 || p->channels / p->ngroups % 8 != 0)
        return SSD_ERR_UNSUPPORTED;
    if (p->state_dtype != SSD_STATE_F32 && p->state_dtype != SSD_STATE_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->total_len > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    const int64_t rows[] = {p->x_stride, p->dt_stride, p->z_stride, p->b_stride, p->c_stride, p->channels, bc};
    for (const int64_t r : rows)
        if (r > kMaxRow) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
ScanParams common(const ssd_selective_problem *p) {
    ScanParams a;
    memset(&a, 0, sizeof a);
    a.T = (int)p->total_len;
    a.batch = p->batch;
    a.D = p->channels;
    a.G = p->ngroups;
    a.N = p->dstate;
    a.Dg = p->channels / p->ngroups;
    a.xs = stride_or(p->x_stride, p->channels);
    a.dts = stride_or(p->dt_stride, p->channels);
    a.zs = stride_or(p->z_stride, p->channels);
    a.bs = stride_or(p->b_stride, (int64_t)p->ngroups * p->dstate);
    a.cs = stride_or(p->c_stride, (int64_t)p->ngroups * p->dstate);
    a.softplus = p->dt_softplus != 0;
    a.state_bf16 = p->state_dtype == SSD_STATE_BF16;
    a.max_slots = (uint32_t)p->batch;
    return a;
}
bool fits(const ScanParams &a, bool backward) {
    return a.places <= INT32_MAX && scan_threads(a, backward) <= UINT32_MAX;
}

// Carves the workspace; the size without one.
size_t carve(ScanParams &a, bool backward, char *base) {
    size_t at = 0;
    auto take = [&](float *&ptr, size_t n) {
        ptr = reinterpret_cast<float *>(base + at);
        at += align_up(n * sizeof(float));
    };
    const size_t DN = (size_t)a.D * (size_t)a.N, cut = (size_t)a.cut_places;
    if (cut > 0) {
        take(a.parts, cut * DN);
        take(a.steps, cut * (size_t)a.D);
        if (backward) take(a.adj, cut * DN);
    }
    if (backward) {
        take(a.marks, ((size_t)a.T / ssd::layer::kGradTile + (size_t)a.batch) * DN);
        take(a.bc, (size_t)a.blocks * (size_t)a.T * 2 * (size_t)a.N);
        take(a.dA_part, (size_t)a.places * DN);
        take(a.dD_part, (size_t)a.places * 2 * (size_t)a.D);
    }
    return at;
}

ssd_status scan_forward(const ssd_selective_problem *p, void *y, const void *x, const void *dt, const float *A,
                        const void *B, const void *C, const float *D, const void *z, const float *dt_bias,
                        const void *state_in, void *state_out, const int32_t *qsl, const uint8_t *has_init,
                        const uint32_t *cache_idx, bool init_all, void *ws, size_t ws_bytes, void *stream) {
    const ssd_status st = check(p);
    if (st != SSD_OK) return st;
    if (A == nullptr || state_out == nullptr || qsl == nullptr) return SSD_ERR_NULL_ARG;
    if (p->total_len > 0 && (y == nullptr || x == nullptr || dt == nullptr || B == nullptr || C == nullptr))
        return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, y, x, dt, z, A, state_in, state_out) || !all_aligned(4, B, C, D, dt_bias, qsl, cache_idx))
        return SSD_ERR_MISALIGNED;
    ScanParams a = common(p);
    scan_shape(a, false);
    if (!fits(a, false)) return SSD_ERR_UNSUPPORTED;
    const ssd_status sw = check_workspace(carve(a, false, nullptr), ws, ws_bytes);
    if (sw != SSD_OK) return sw;
    carve(a, false, static_cast<char *>(ws));
    a.y = static_cast<uint16_t *>(y);
    a.x = static_cast<const uint16_t *>(x);
    a.dt = static_cast<const uint16_t *>(dt);
    a.z = static_cast<const uint16_t *>(z);
    a.A = A;
    a.B = static_cast<const uint16_t *>(B);
    a.C = static_cast<const uint16_t *>(C);
    a.Dskip = D;
    a.bias = dt_bias;
    a.state_in = state_in;
    a.state_out = state_out;
    a.qsl = qsl;
    a.has_init = has_init;
    a.cache_idx = cache_idx;
    a.init_all = init_all;
    if (cache_idx != nullptr) a.max_slots = (uint32_t)p->max_slots;
    return launched(launch_scan(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

ssd_status ssd_rms_norm_fwd(const ssd_norm_problem *prob, void *y, float *scales, void *residual_out, const void *x,
                            const void *residual, const float *weight, void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    const bool codes = prob->out_format != SSD_OUT_BF16;
    if (weight == nullptr || (residual == nullptr) != (residual_out == nullptr)) return SSD_ERR_NULL_ARG;
    if (prob->rows > 0 && (y == nullptr || x == nullptr || (codes && scales == nullptr))) return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, x, residual, residual_out, weight) || !aligned(y, codes ? 8 : 16) || !aligned(scales, 4))
        return SSD_ERR_MISALIGNED;
    if (prob->rows == 0) return SSD_OK;
    NormParams a;
    a.rows = prob->rows;
    a.xs = stride_or(prob->x_stride, prob->width);
    a.width = prob->width;
    a.eps = prob->eps;
    a.res_bf16 = prob->residual_dtype == SSD_STATE_BF16;
    a.out = prob->out_format;
    a.y = y;
    a.scales = scales;
    a.res_out = residual_out;
    a.x = static_cast<const uint16_t *>(x);
    a.res = residual;
    a.weight = weight;
    return launched(launch_norm(a, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_rms_norm_workspace_size(const ssd_norm_problem *prob, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_NULL_ARG;
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    *bytes = align_up((size_t)ssd::layer::norm_grad_parts(prob->rows, prob->width) * (size_t)prob->width *
                      sizeof(float));
    return SSD_OK;
}

ssd_status ssd_rms_norm_bwd(const ssd_norm_problem *prob, void *dx, void *d_residual, float *dweight, const void *r,
                            const float *weight, const void *d_y, const void *d_r, void *workspace,
                            size_t workspace_bytes, void *stream) {
    size_t need = 0;
    const ssd_status st = ssd_rms_norm_workspace_size(prob, &need);
    if (st != SSD_OK) return st;
    if (dweight == nullptr || weight == nullptr) return SSD_ERR_NULL_ARG;
    if (prob->rows > 0 && (dx == nullptr || r == nullptr || d_y == nullptr)) return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, dx, d_residual, dweight, r, weight, d_y, d_r)) return SSD_ERR_MISALIGNED;
    const ssd_status sw = check_workspace(need, workspace, workspace_bytes);
    if (sw != SSD_OK) return sw;
    NormGradParams a;
    a.rows = prob->rows;
    a.width = prob->width;
    a.eps = prob->eps;
    a.res_bf16 = prob->residual_dtype == SSD_STATE_BF16;
    a.dx = static_cast<uint16_t *>(dx);
    a.d_res = d_residual;
    a.r = r;
    a.weight = weight;
    a.dy = static_cast<const uint16_t *>(d_y);
    a.d_r = d_r;
    a.part = static_cast<float *>(workspace);
    a.dweight = dweight;
    a.parts = ssd::layer::norm_grad_parts(prob->rows, prob->width);
    return launched(launch_norm_grad(a, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_causal_conv_varlen_fwd_inplace(const ssd_conv_problem *prob, void *y, const void *x,
                                              const float *weight, const float *bias, void *pool,
                                              const int32_t *query_start_loc, const uint8_t *has_initial_state,
                                              const uint32_t *cache_indices, void *stream) {
    if (cache_indices == nullptr) return SSD_ERR_NULL_ARG;
    return conv_forward(prob, y, x, weight, bias, pool, pool, query_start_loc, has_initial_state, cache_indices,
                        false, stream);
}

ssd_status ssd_causal_conv_varlen_fwd(const ssd_conv_problem *prob, void *y, const void *x, const float *weight,
                                      const float *bias, const void *initial_states, void *final_states,
                                      const int32_t *query_start_loc, void *stream) {
    return conv_forward(prob, y, x, weight, bias, initial_states, final_states, query_start_loc, nullptr, nullptr,
                        true, stream);
}

ssd_status ssd_causal_conv_workspace_size(const ssd_conv_problem *prob, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_NULL_ARG;
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    ConvParams a = common(prob);
    conv_shape(a, prob->width, true);
    if (!fits(a)) return SSD_ERR_UNSUPPORTED;
    *bytes = conv_workspace(a, prob->width);
    return SSD_OK;
}

ssd_status ssd_causal_conv_varlen_bwd(const ssd_conv_problem *prob, void *dx, float *dweight, float *dbias,
                                      void *d_initial, const void *x, const float *weight, const float *bias,
                                      const void *d_y, const void *initial_states, const void *d_final,
                                      const int32_t *query_start_loc, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (dweight == nullptr || weight == nullptr || query_start_loc == nullptr) return SSD_ERR_NULL_ARG;
    if (prob->total_len > 0 && (dx == nullptr || x == nullptr || d_y == nullptr)) return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, dx, dweight, dbias, d_initial, x, weight, bias, d_y, initial_states, d_final) ||
        !aligned(query_start_loc, 4))
        return SSD_ERR_MISALIGNED;
    ConvParams a = common(prob);
    conv_shape(a, prob->width, true);
    if (!fits(a)) return SSD_ERR_UNSUPPORTED;
    const ssd_status sw = check_workspace(conv_workspace(a, prob->width), workspace, workspace_bytes);
    if (sw != SSD_OK) return sw;
    if (rows_meet(dx, x, a.T, a.D, a.xs) || rows_meet(dx, d_y, a.T, a.D, a.D)) return SSD_ERR_UNSUPPORTED;
    a.x = static_cast<const uint16_t *>(x);
    a.weight = weight;
    a.bias = bias;
    a.state_in = static_cast<const uint16_t *>(initial_states);
    a.qsl = query_start_loc;
    a.init_all = 1;
    a.dy = static_cast<const uint16_t *>(d_y);
    a.d_final = static_cast<const uint16_t *>(d_final);
    a.dx = static_cast<uint16_t *>(dx);
    a.d_init = static_cast<uint16_t *>(d_initial);
    a.part = static_cast<float *>(workspace);
    a.dweight = dweight;
    a.dbias = dbias;
    return launched(launch_conv_grad(a, prob->width, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_causal_conv_step_inplace(const ssd_conv_problem *prob, void *y, const void *x, const float *weight,
                                        const float *bias, void *pool, const uint8_t *has_initial_state,
                                        const uint32_t *cache_indices, void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (prob->total_len != prob->batch) return SSD_ERR_BAD_SHAPE;
    if ((int64_t)prob->batch * (prob->channels / 8) > (int64_t)UINT32_MAX - 255) return SSD_ERR_UNSUPPORTED;
    if (y == nullptr || x == nullptr || weight == nullptr || pool == nullptr || cache_indices == nullptr)
        return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, y, x, weight, bias, pool) || !aligned(cache_indices, 4)) return SSD_ERR_MISALIGNED;
    ConvParams a = common(prob);
    a.y = static_cast<uint16_t *>(y);
    a.x = static_cast<const uint16_t *>(x);
    a.weight = weight;
    a.bias = bias;
    a.state_out = static_cast<uint16_t *>(pool);
    a.has_init = has_initial_state;
    a.cache_idx = cache_indices;
    a.max_slots = (uint32_t)prob->max_slots;
    return launched(launch_conv_step(a, prob->width, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_selective_scan_workspace_size(const ssd_selective_problem *prob, int backward, size_t *bytes) {
    if (bytes == nullptr) return SSD_ERR_NULL_ARG;
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    ScanParams a = common(prob);
    scan_shape(a, backward != 0);
    if (!fits(a, backward != 0)) return SSD_ERR_UNSUPPORTED;
    *bytes = carve(a, backward != 0, nullptr);
    return SSD_OK;
}

ssd_status ssd_selective_scan_varlen_fwd_inplace(
    const ssd_selective_problem *prob, void *y, const void *x, const void *dt, const float *A, const void *B,
    const void *C, const float *D, const void *z, const float *dt_bias, void *pool, const int32_t *query_start_loc,
    const uint8_t *has_initial_state, const uint32_t *cache_indices, void *workspace, size_t workspace_bytes,
    void *stream) {
    if (cache_indices == nullptr) return SSD_ERR_NULL_ARG;
    return scan_forward(prob, y, x, dt, A, B, C, D, z, dt_bias, pool, pool, query_start_loc, has_initial_state,
                        cache_indices, false, workspace, workspace_bytes, stream);
}

ssd_status ssd_selective_scan_varlen_fwd(
    const ssd_selective_problem *prob, void *y, const void *x, const void *dt, const float *A, const void *B,
    const void *C, const float *D, const void *z, const float *dt_bias, const void *initial_states,
    void *final_states, const int32_t *query_start_loc, void *workspace, size_t workspace_bytes, void *stream) {
    return scan_forward(prob, y, x, dt, A, B, C, D, z, dt_bias, initial_states, final_states, query_start_loc,
                        nullptr, nullptr, true, workspace, workspace_bytes, stream);
}

ssd_status ssd_selective_scan_varlen_bwd(
    const ssd_selective_problem *prob, void *dx, void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz,
    float *ddt_bias, void *d_initial, const void *x, const void *dt, const float *A, const void *B, const void *C,
    const float *D, const void *z, const float *dt_bias, const void *d_y, const void *initial_states,
    const void *d_final, const int32_t *query_start_loc, void *workspace, size_t workspace_bytes, void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (dA == nullptr || A == nullptr || query_start_loc == nullptr) return SSD_ERR_NULL_ARG;
    if (prob->total_len > 0 &&
        (dx == nullptr || ddt == nullptr || dB == nullptr || dC == nullptr || x == nullptr || dt == nullptr ||
         B == nullptr || C == nullptr || d_y == nullptr || (z == nullptr) != (dz == nullptr)))
        return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_initial, x, dt, A, z, d_y, initial_states, d_final) ||
        !all_aligned(4, B, C, D, dt_bias, query_start_loc))
        return SSD_ERR_MISALIGNED;
    ScanParams a = common(prob);
    scan_shape(a, true);
    if (!fits(a, true)) return SSD_ERR_UNSUPPORTED;
    const ssd_status sw = check_workspace(carve(a, true, nullptr), workspace, workspace_bytes);
    if (sw != SSD_OK) return sw;
    carve(a, true, static_cast<char *>(workspace));
    a.x = static_cast<const uint16_t *>(x);
    a.dt = static_cast<const uint16_t *>(dt);
    a.z = static_cast<const uint16_t *>(z);
    a.A = A;
    a.B = static_cast<const uint16_t *>(B);
    a.C = static_cast<const uint16_t *>(C);
    a.Dskip = D;
    a.bias = dt_bias;
    a.state_in = initial_states;
    a.init_all = 1;
    a.qsl = query_start_loc;
    a.dy = static_cast<const uint16_t *>(d_y);
    a.d_final = d_final;
    a.dx = static_cast<uint16_t *>(dx);
    a.ddt = static_cast<uint16_t *>(ddt);
    a.dz = static_cast<uint16_t *>(dz);
    a.dB = static_cast<uint16_t *>(dB);
    a.dC = static_cast<uint16_t *>(dC);
    a.d_init = d_initial;
    a.dA = dA;
    a.dD = dD;
    a.dbias = ddt_bias;
    return launched(launch_scan_grad(a, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_selective_scan_step_inplace(
    const ssd_selective_problem *prob, void *y, const void *x, const void *dt, const float *A, const void *B,
    const void *C, const float *D, const void *z, const float *dt_bias, void *pool,
    const uint8_t *has_initial_state, const uint32_t *cache_indices, void *stream) {
    const ssd_status st = check(prob);
    if (st != SSD_OK) return st;
    if (prob->total_len != prob->batch) return SSD_ERR_BAD_SHAPE;
    if ((int64_t)prob->batch * ((int64_t)prob->channels + 256) * 16 > UINT32_MAX) return SSD_ERR_UNSUPPORTED;
    if (y == nullptr || x == nullptr || dt == nullptr || A == nullptr || B == nullptr || C == nullptr ||
        pool == nullptr || cache_indices == nullptr)
        return SSD_ERR_NULL_ARG;
    if (!all_aligned(16, A, pool) || !all_aligned(4, B, C, D, dt_bias, cache_indices) || !all_aligned(2, y, x, dt, z))
        return SSD_ERR_MISALIGNED;
    ScanParams a = common(prob);
    a.y = static_cast<uint16_t *>(y);
    a.x = static_cast<const uint16_t *>(x);
    a.dt = static_cast<const uint16_t *>(dt);
    a.z = static_cast<const uint16_t *>(z);
    a.A = A;
    a.B = static_cast<const uint16_t *>(B);
    a.C = static_cast<const uint16_t *>(C);
    a.Dskip = D;
    a.bias = dt_bias;
    a.state_in = pool;
    a.state_out = pool;
    a.has_init = has_initial_state;
    a.cache_idx = cache_indices;
    a.max_slots = (uint32_t)prob->max_slots;
    return launched(launch_scan_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
