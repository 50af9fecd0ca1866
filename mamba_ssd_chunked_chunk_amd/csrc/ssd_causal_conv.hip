// Short causal depthwise convolution over ragged batches, its step for single
// tokens and its backward pass.  A wavefront takes a piece of one sequence and
// 512 channels, 8 consecutive ones a lane, and walks along the tokens with the
// last width - 1 inputs in registers, so a row is read once but for the few
// ahead of a piece.  Only the first piece of a sequence, which alone reads its
// state, writes the one that it leaves, so the pool needs no second launch.
#include "ssd_layer.hpp"

namespace ssd {
namespace layer {
namespace {

constexpr int kAhead = 8;  // rows in flight

// weights [channels][W] of 8 channels
template <int W>
__device__ __forceinline__ void load_taps(const float *weight, int c, float (&w)[W][8]) {
    const float *at = weight + (int64_t)c * W;
    float f[8 * W];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
        const f32x4 v = reinterpret_cast<const f32x4 *>(at)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
}
__device__ __forceinline__ u32x4 row8(const uint16_t *base, int64_t at) {
    return *reinterpret_cast<const u32x4 *>(base + at);
}
__device__ __forceinline__ void put8(uint16_t *base, int64_t at, const u32x4 &v) {
    *reinterpret_cast<u32x4 *>(base + at) = v;
}

// The W - 1 inputs ahead of token `t` of a sequence, as they are stored: of the
// sequence, of its state ahead of it, or zero.  `state`: its rows, or null.
template <int W>
__device__ __forceinline__ void load_window(const ConvParams &p, const Seq &q, int t, const uint16_t *state, int c,
                                            u32x4 (&win)[W - 1]) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int i = t - (W - 1) + r;
        win[r] = u32x4{0, 0, 0, 0};
        if (i >= 0)
            win[r] = row8(p.x, (int64_t)(q.begin + i) * p.xs + c);
        else if (state != nullptr)
            win[r] = row8(state, (int64_t)(W - 1 + i) * p.D + c);
    }
}

template <int W>
__global__ __launch_bounds__(256) void conv_fwd(ConvParams p) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int cblocks = (p.D + 511) / 512;
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int place = (int)(item / cblocks), c = (int)(item % cblocks) * 512 + lane * 8;
    if (place >= p.places) return;
    Seq q;
    int s;
    if (!find_piece(p.qsl, p.batch, p.T, p.tile, place, q, s)) return;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[q.b] : q.b;
    if (slot >= (int64_t)p.max_slots) return;  // padding
    if (c >= p.D) return;
    const bool init = p.state_in != nullptr && (p.init_all || (p.has_init != nullptr && p.has_init[q.b] != 0));
    const int64_t at = slot * (W - 1) * p.D;
    const uint16_t *state = init ? p.state_in + at : nullptr;
    const int t0 = s * p.tile, t1 = min(q.len, t0 + p.tile);

    u32x4 win[W - 1];
    load_window<W>(p, q, t0, state, c, win);
    if (s == 0) {
        // the state that the sequence leaves
        u32x4 last[W - 1];
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const int i = q.len - (W - 1) + r;
            last[r] = u32x4{0, 0, 0, 0};
            if (i >= 0)
                last[r] = row8(p.x, (int64_t)(q.begin + i) * p.xs + c);
            else {
#pragma unroll
                for (int m = 0; m < W - 1; ++m)
                    if (m == W - 1 + i) last[r] = win[m];
            }
        }
#pragma unroll
        for (int r = 0; r < W - 1; ++r) put8(p.state_out, at + (int64_t)r * p.D + c, last[r]);
    }
    if (t0 >= t1) return;
    float w[W][8], bias[8] = {}, v[W][8];
    load_taps<W>(p.weight, c, w);
    if (p.bias != nullptr) load_state8<false>(p.bias, c, bias);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) widen8(win[r], v[r]);
    const uint16_t *x = p.x + (int64_t)q.begin * p.xs + c;
    uint16_t *y = p.y + (int64_t)q.begin * p.D + c;
    u32x4 next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (t0 + i < t1) next[i] = row8(x, (int64_t)(t0 + i) * p.xs);
    for (int t = t0; t < t1; t += kAhead) {
        u32x4 rows[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) rows[i] = next[i];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t + kAhead + i < t1) next[i] = row8(x, (int64_t)(t + kAhead + i) * p.xs);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t + i >= t1) break;
            widen8(rows[i], v[W - 1]);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a = bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][e], v[j][e], a);
                o[e] = p.silu ? a * sigmoid_f(a) : a;
            }
            put8(y, (int64_t)(t + i) * p.D, narrow8(o));
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = v[j + 1][e];
        }
    }
}

// One token a sequence.  A thread takes 8 channels.
template <int W>
__global__ __launch_bounds__(256) void conv_step(ConvParams p) {
    const int cthreads = p.D / 8;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = item / cthreads;
    if (b >= p.batch) return;
    const int c = (int)(item % cthreads) * 8;
    const int64_t slot = p.cache_idx[b];
    if (slot >= (int64_t)p.max_slots) return;  // padding
    const bool init = p.has_init != nullptr && p.has_init[b] != 0;
    uint16_t *state = p.state_out + slot * (W - 1) * p.D + c;
    u32x4 win[W];
    win[W - 1] = row8(p.x, b * p.xs + c);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) win[r] = init ? row8(state, (int64_t)r * p.D) : u32x4{0, 0, 0, 0};
    float w[W][8], a[8] = {};
    load_taps<W>(p.weight, c, w);
    if (p.bias != nullptr) load_state8<false>(p.bias, c, a);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[8];
        widen8(win[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = __builtin_fmaf(w[j][e], v[e], a[e]);
    }
    if (p.silu)
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] *= sigmoid_f(a[e]);
    put8(p.y, b * p.D + c, narrow8(a));
#pragma unroll
    for (int r = 0; r < W - 1; ++r) put8(state, (int64_t)r * p.D, win[r + 1]);
}

// Backward.  With g_t = dy_t silu'(p_t) (0 behind the sequence's end),
//     dx_u = sum_k w[W-1-k] g_{u+k},  dw[j] = sum_t g_t x_{t-(W-1)+j},
// so the walk keeps the last g's as it keeps the inputs and finishes dx_u at
// token u + W - 1; a piece walks W - 1 tokens past its end, whose g's count
// for the next piece's weights alone.  The four pieces of a block add their
// weights' gradients before they store them.
template <int W>
__global__ __launch_bounds__(256) void conv_grad(ConvParams p) {
    __shared__ float sums[3][(W + 1) * 8][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int cblocks = (p.D + 511) / 512;
    const int64_t quad = blockIdx.x / cblocks;
    const int c = (int)(blockIdx.x % cblocks) * 512 + lane * 8;
    const bool in = c < p.D;
    float dw[W][8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    Seq q;
    int s;
    const int64_t place = quad * 4 + wave;
    if (place < p.places && find_piece(p.qsl, p.batch, p.T, p.tile, (int)place, q, s) && in) {
        const int64_t at = (int64_t)q.b * (W - 1) * p.D;
        const uint16_t *state = p.state_in != nullptr ? p.state_in + at : nullptr;
        const int t0 = s * p.tile, t1 = min(q.len, t0 + p.tile);
        // tokens walked: W - 1 past the end of the piece (behind the sequence they hold nothing)
        const int t2 = t1 + W - 1;
        float w[W][8], bias[8] = {}, v[W][8], g[W][8];
        load_taps<W>(p.weight, c, w);
        if (p.bias != nullptr) load_state8<false>(p.bias, c, bias);
        u32x4 win[W - 1];
        load_window<W>(p, q, t0, state, c, win);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            widen8(win[r], v[r]);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[r][e] = 0.f;
        }
        const uint16_t *x = p.x + (int64_t)q.begin * p.xs + c;
        const uint16_t *dy = p.dy + (int64_t)q.begin * p.D + c;
        uint16_t *dx = p.dx + (int64_t)q.begin * p.D + c;
        const int live = min(q.len, t2);
        u32x4 nx[kAhead], ng[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            nx[i] = ng[i] = u32x4{0, 0, 0, 0};
            if (t0 + i < live) {
                nx[i] = row8(x, (int64_t)(t0 + i) * p.xs);
                ng[i] = row8(dy, (int64_t)(t0 + i) * p.D);
            }
        }
        for (int t = t0; t < t2; t += kAhead) {
            u32x4 rx[kAhead], rg[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                rx[i] = nx[i];
                rg[i] = ng[i];
                nx[i] = ng[i] = u32x4{0, 0, 0, 0};
                if (t + kAhead + i < live) {
                    nx[i] = row8(x, (int64_t)(t + kAhead + i) * p.xs);
                    ng[i] = row8(dy, (int64_t)(t + kAhead + i) * p.D);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (t + i >= t2) break;
                const int u = t + i - (W - 1);  // finished by this token
                widen8(rx[i], v[W - 1]);
                widen8(rg[i], g[W - 1]);
                const bool count = t + i < t1;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (t + i >= q.len) {
                        g[W - 1][e] = 0.f;  // also where 0 silu'(p) is NaN
                    } else if (p.silu) {
                        float a = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][e], v[j][e], a);
                        const float o = sigmoid_f(a);
                        g[W - 1][e] *= __builtin_fmaf(a * o, 1.f - o, o);
                    }
                    if (count) {
                        db[e] += g[W - 1][e];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][e] = __builtin_fmaf(g[W - 1][e], v[j][e], dw[j][e]);
                    }
                }
                const bool ahead = u < 0;  // the state's rows, which the first piece finishes
                if (ahead ? s == 0 && p.d_init != nullptr : u >= t0) {
                    float o[8] = {};
                    const int r = u - (q.len - (W - 1));  // of the state that the sequence leaves
                    if (p.d_final != nullptr && r >= 0)
                        load_state8<true>(p.d_final, at + (int64_t)r * p.D + c, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int k = 0; k < W; ++k) o[e] = __builtin_fmaf(w[W - 1 - k][e], g[k][e], o[e]);
                    if (ahead)
                        put8(p.d_init, at + (int64_t)(u + W - 1) * p.D + c, narrow8(o));
                    else
                        put8(dx, (int64_t)u * p.D, narrow8(o));
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[j][e] = v[j + 1][e];
                        g[j][e] = g[j + 1][e];
                    }
            }
        }
    }
    // the four pieces' sums, by the first wavefront
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sums[wave - 1][W * 8 + e][lane] = db[e];
#pragma unroll
            for (int j = 0; j < W; ++j) sums[wave - 1][j * 8 + e][lane] = dw[j][e];
        }
    }
    __syncthreads();
    if (wave > 0 || !in) return;
    float *part = p.part + quad * (W + 1) * p.D;
    // [channel][tap] as the weights lie, then the bias
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            db[e] += sums[n][W * 8 + e][lane];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] += sums[n][j * 8 + e][lane];
        }
    }
    float f[8 * W];
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) f[e * W + j] = dw[j][e];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i)
        reinterpret_cast<f32x4 *>(part + (int64_t)c * W)[i] = f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
    store_state8<false>(part, (int64_t)W * p.D + c, db);
}

template <typename F>
hipError_t by_width(int width, F f) {
    if (width == 2) f(std::integral_constant<int, 2>{});
    else if (width == 3) f(std::integral_constant<int, 3>{});
    else f(std::integral_constant<int, 4>{});
    return hipGetLastError();
}
int64_t blocks_of(int64_t n, int64_t per) { return (n + per - 1) / per; }
}  // namespace

void conv_shape(ConvParams &p, bool backward) {
    p.tile = 32;
    p.places = p.T / p.tile + p.batch;
    (void)backward;
}
int64_t conv_parts(const ConvParams &p) { return blocks_of(p.places, 4); }
int64_t conv_threads(const ConvParams &p) { return blocks_of(p.places, 4) * 4 * blocks_of(p.D, 512) * 64; }

hipError_t launch_conv(const ConvParams &p, int width, hipStream_t s) {
    const dim3 grid((unsigned)blocks_of(p.places * blocks_of(p.D, 512), 4));
    return by_width(width, [&](auto w) { conv_fwd<decltype(w)::value><<<grid, 256, 0, s>>>(p); });
}
hipError_t launch_conv_step(const ConvParams &p, int width, hipStream_t s) {
    const dim3 grid((unsigned)blocks_of((int64_t)p.batch * (p.D / 8), 256));
    return by_width(width, [&](auto w) { conv_step<decltype(w)::value><<<grid, 256, 0, s>>>(p); });
}
hipError_t launch_conv_grad(const ConvParams &p, int width, hipStream_t s) {
    const int64_t quads = conv_parts(p);
    const dim3 grid((unsigned)(quads * blocks_of(p.D, 512)));
    hipError_t e = by_width(width, [&](auto w) { conv_grad<decltype(w)::value><<<grid, 256, 0, s>>>(p); });
    if (e != hipSuccess) return e;
    const int64_t row = (int64_t)(width + 1) * p.D;
    return launch_sums(Sums{{Sum{p.part, (int)quads, row, (int64_t)width * p.D, p.dweight},
                             Sum{p.part + (int64_t)width * p.D, (int)quads, row, p.D, p.dbias}}},
                       s);
}

}  // namespace layer
}  // namespace ssd
