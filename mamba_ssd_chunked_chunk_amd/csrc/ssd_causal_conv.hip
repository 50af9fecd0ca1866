// Short causal depthwise convolution over ragged batches, its step for single
// tokens and its backward pass.  A lane takes 8 consecutive channels (4 in the
// backward pass) of a piece of one sequence and walks along the tokens, the last
// `width` inputs in a ring of registers and the next rows on their way in others,
// so a row is read once but for the few ahead of a piece.  Only the first piece of
// a sequence, which alone reads its state, writes the one that it leaves, so the
// pool needs no second launch.
//
// Memory bounds it: 43898 tokens of 10240 channels, 1.80 GB, 353 us (5.1 TB/s); the
// backward pass of 4 x 4096 tokens of 1536 channels, 151 MB, 36 us (its arithmetic,
// 30 operations an element with the silu's slope, takes about half of that), and 5
// for the sum of the blocks' shares; a step of 512 sequences of 10240 channels, 84
// MB, 17 us.
#include "ssd_layer.hpp"

namespace ssd {
namespace layer {
namespace {

// Rows in flight, a multiple of the width, so that a token's place in the ring
// is known when the walk is unrolled.
template <int W>
constexpr int kAhead = W == 3 ? 6 : 8;

// E consecutive bf16 as they lie in memory, and as floats
template <int E>
using Raw = uint32_t __attribute__((ext_vector_type(E / 2)));
template <int E>
__device__ __forceinline__ Raw<E> row_of(const uint16_t *base, int64_t at) {
    return *reinterpret_cast<const Raw<E> *>(base + at);
}
template <int E>
__device__ __forceinline__ void put_row(uint16_t *base, int64_t at, const Raw<E> &v) {
    *reinterpret_cast<Raw<E> *>(base + at) = v;
}
template <int E>
__device__ __forceinline__ void widen(const Raw<E> &v, float (&o)[E]) {
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        o[2 * k] = bf16x2_lo(v[k]);
        o[2 * k + 1] = bf16x2_hi(v[k]);
    }
}
template <int E>
__device__ __forceinline__ Raw<E> narrow(const float (&v)[E]) {
    Raw<E> r;
#pragma unroll
    for (int k = 0; k < E / 2; ++k) r[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    return r;
}

// weights [channels][W] and bias of E channels
template <int W, int E>
__device__ __forceinline__ void load_taps(const float *weight, int c, float (&w)[W][E]) {
    const f32x4 *at = reinterpret_cast<const f32x4 *>(weight + (int64_t)c * W);
    float f[E * W];
#pragma unroll
    for (int i = 0; i < E * W / 4; ++i) {
        const f32x4 v = at[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
}
template <int E>
__device__ __forceinline__ void load_bias(const float *bias, int c, float (&b)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) b[e] = 0.f;
    if (bias == nullptr) return;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const f32x4 v = reinterpret_cast<const f32x4 *>(bias + c)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[4 * i + e] = v[e];
    }
}

// The W - 1 inputs ahead of token `t` of a sequence, as they are stored: of the
// sequence, of its state ahead of it, or zero.  `state`: its rows, or null.
template <int W, int E>
__device__ __forceinline__ void load_window(const ConvParams &p, const Seq &q, int t, const uint16_t *state, int c,
                                            Raw<E> (&win)[W - 1]) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int i = t - (W - 1) + r;
        win[r] = Raw<E>(0);
        if (i >= 0)
            win[r] = row_of<E>(p.x, (int64_t)(q.begin + i) * p.xs + c);
        else if (state != nullptr)
            win[r] = row_of<E>(state, (int64_t)(W - 1 + i) * p.D + c);
    }
}

// PAST: the outputs pass by the caches.
template <int W, bool PAST>
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

    constexpr int E = 8, R = kAhead<W>;
    Raw<E> win[W - 1];
    load_window<W, E>(p, q, t0, state, c, win);
    if (s == 0) {
        // the state that the sequence leaves
        Raw<E> last[W - 1];
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const int i = q.len - (W - 1) + r;
            last[r] = Raw<E>(0);
            if (i >= 0)
                last[r] = row_of<E>(p.x, (int64_t)(q.begin + i) * p.xs + c);
            else {
#pragma unroll
                for (int m = 0; m < W - 1; ++m)
                    if (m == W - 1 + i) last[r] = win[m];
            }
        }
#pragma unroll
        for (int r = 0; r < W - 1; ++r) put_row<E>(p.state_out, at + (int64_t)r * p.D + c, last[r]);
    }
    if (t0 >= t1) return;
    float w[W][E], bias[E], v[W][E];  // v: tap j of the walk's i-th token at (i + j) % W
    load_taps<W, E>(p.weight, c, w);
    load_bias<E>(p.bias, c, bias);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) widen<E>(win[r], v[r]);
    // rows by an address that all lanes share and the lane's own offset in bytes
    Scalar<const uint16_t> x(p.x + (int64_t)(q.begin + t0) * p.xs);
    Scalar<uint16_t> y(p.y + (int64_t)(q.begin + t0) * p.D);
    const uint32_t lo = c * 2;
    // (no branch ends a group early, and rows behind the piece are its last one: values that meet where branches
    // join would be copied)
    Raw<E> rows[R];
    int ahead = t0;  // the row that is fetched next
    auto fetch = [&](int i) {
        x.hold();
        rows[i] = x.at<Raw<E>>(lo);
        x.ptr += ahead < t1 - 1 ? p.xs : 0;
        ++ahead;
    };
#pragma unroll
    for (int i = 0; i < R; ++i) fetch(i);
    for (int t = t0; t < t1; t += R) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            widen<E>(rows[i], v[(i + W - 1) % W]);
            fetch(i);
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float a = bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][e], v[(i + j) % W][e], a);
                o[e] = p.silu ? a * sigmoid_f(a) : a;
            }
            y.hold();
            if (t + i < t1) {
                if constexpr (PAST)
                    y.put_past(lo, narrow<E>(o));
                else
                    y.put(lo, narrow<E>(o));
            }
            y.ptr += p.D;
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// One token a sequence.  A thread takes 8 channels of several sequences, whose
// rows are all on their way before the first is worked on.
constexpr int kStepSeqs = 2;
template <int W, int SEQS>
__global__ __launch_bounds__(256) void conv_step(ConvParams p) {
    constexpr int E = 8;
    const int cthreads = p.D / 8;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b0 = item / cthreads * SEQS;
    const int c = (int)(item % cthreads) * 8;
    Raw<E> win[SEQS][W];
    int64_t at[SEQS];
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const int64_t b = b0 + k;
        const int64_t slot = b < p.batch ? (int64_t)p.cache_idx[b] : (int64_t)p.max_slots;
        at[k] = slot < (int64_t)p.max_slots ? slot * (W - 1) * p.D + c : -1;  // none: padding
        if (at[k] < 0) continue;
        const bool init = p.has_init != nullptr && p.has_init[b] != 0;
        win[k][W - 1] = row_of<E>(p.x, b * p.xs + c);
#pragma unroll
        for (int r = 0; r < W - 1; ++r)
            win[k][r] = init ? row_of<E>(p.state_out, at[k] + (int64_t)r * p.D) : Raw<E>(0);
    }
    if (b0 >= p.batch) return;
    float w[W][E], bias[E];
    load_taps<W, E>(p.weight, c, w);
    load_bias<E>(p.bias, c, bias);
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        if (at[k] < 0) continue;
        float a[E];
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float v[E];
            widen<E>(win[k][j], v);
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = __builtin_fmaf(w[j][e], v[e], a[e]);
        }
        if (p.silu)
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] *= sigmoid_f(a[e]);
        put_row<E>(p.y, (b0 + k) * p.D + c, narrow<E>(a));
#pragma unroll
        for (int r = 0; r < W - 1; ++r) put_row<E>(p.state_out, at[k] + (int64_t)r * p.D, win[k][r + 1]);
    }
}

// Backward.  With g_t = dy_t silu'(p_t) (0 behind the sequence's end),
//     dx_u = sum_k w[W-1-k] g_{u+k},  dw[j] = sum_t g_t x_{t-(W-1)+j},
// so the walk keeps the last g's as it keeps the inputs and finishes dx_u at
// token u + W - 1; a piece walks W - 1 tokens past its end, whose g's count
// for the next piece's weights alone.  The four pieces of a block add their
// weights' gradients before they store them.
constexpr int kGradChannels = 4;  // of a lane
template <int W>
__global__ __launch_bounds__(256) void conv_grad(ConvParams p) {
    constexpr int E = kGradChannels, R = kAhead<W>;
    __shared__ float sums[3][(W + 1) * E][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int cblocks = (p.D + 64 * E - 1) / (64 * E);
    const int64_t quad = blockIdx.x / cblocks;
    const int c = (int)(blockIdx.x % cblocks) * 64 * E + lane * E;
    const bool in = c < p.D;
    float dw[W][E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
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
        const int t2 = t1 + W - 1, live = min(q.len, t2);
        float w[W][E], bias[E], v[W][E], g[W][E];  // v, g: of the walk's i-th token's window at (i + j) % W
        load_taps<W, E>(p.weight, c, w);
        load_bias<E>(p.bias, c, bias);
        Raw<E> win[W - 1];
        load_window<W, E>(p, q, t0, state, c, win);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            widen<E>(win[r], v[r]);
#pragma unroll
            for (int e = 0; e < E; ++e) g[r][e] = 0.f;
        }
        Scalar<const uint16_t> x(p.x + (int64_t)(q.begin + t0) * p.xs), dy(p.dy + (int64_t)(q.begin + t0) * p.D);
        Scalar<uint16_t> dx(p.dx + (int64_t)(q.begin + t0 - (W - 1)) * p.D);  // (row u of the walk)
        const uint32_t lo = c * 2;
        Raw<E> rx[R], rg[R];
        int next = t0;  // the row that is fetched next
        auto fetch = [&](int i) {
            x.hold();
            dy.hold();
            rx[i] = x.at<Raw<E>>(lo);
            rg[i] = dy.at<Raw<E>>(lo);
            x.ptr += next < live - 1 ? p.xs : 0;
            dy.ptr += next < live - 1 ? p.D : 0;
            ++next;
        };
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (live > t0)
                fetch(i);
            else  // a sequence without tokens
                rx[i] = rg[i] = Raw<E>(0);
        }
        // WHOLE: all tokens of the group are the piece's own.  INNER: and the rows that they finish as well.
        auto group = [&](int t, auto whole, auto inner) {
            constexpr bool WHOLE = decltype(whole)::value, INNER = decltype(inner)::value;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float(&vn)[E] = v[(i + W - 1) % W], (&gn)[E] = g[(i + W - 1) % W];
                widen<E>(rx[i], vn);
                widen<E>(rg[i], gn);
                if (live > t0) fetch(i);
                if (p.silu)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float a = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][e], v[(i + j) % W][e], a);
                        const float o = sigmoid_f(a);
                        gn[e] *= __builtin_fmaf(a * o, 1.f - o, o);
                    }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!WHOLE) gn[e] = t + i < q.len ? gn[e] : 0.f;
                    const float own = WHOLE || t + i < t1 ? gn[e] : 0.f;
                    db[e] += own;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        // (x behind the sequence is not there: 0 times it may be NaN)
                        const float xv = WHOLE || t + i < t1 ? v[(i + j) % W][e] : 0.f;
                        dw[j][e] = __builtin_fmaf(own, xv, dw[j][e]);
                    }
                }
                dx.hold();
                const int u = t + i - (W - 1);       // finished by this token
                const bool ahead = !INNER && u < 0;  // the state's rows, which the first piece finishes
                if (INNER || (ahead ? s == 0 && p.d_init != nullptr : u >= t0 && u < t1)) {
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = 0.f;
                    const int r = u - (q.len - (W - 1));  // of the state that the sequence leaves
                    if (!WHOLE && p.d_final != nullptr && r >= 0)
                        widen<E>(row_of<E>(p.d_final, at + (int64_t)r * p.D + c), o);
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            o[e] = __builtin_fmaf(w[W - 1 - k][e], g[(i + k) % W][e], o[e]);
                    if (ahead)
                        put_row<E>(p.d_init, at + (int64_t)(u + W - 1) * p.D + c, narrow<E>(o));
                    else
                        dx.put(lo, narrow<E>(o));
                }
                dx.ptr += p.D;
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        int t = t0;
        if (t + R <= t1) {
            group(t, std::true_type{}, std::false_type{});
            for (t += R; t + R <= t1; t += R) group(t, std::true_type{}, std::true_type{});
        }
        for (; t < t2; t += R) group(t, std::false_type{}, std::false_type{});
    }
    // the four pieces' sums, by the first wavefront
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sums[wave - 1][W * E + e][lane] = db[e];
#pragma unroll
            for (int j = 0; j < W; ++j) sums[wave - 1][j * E + e][lane] = dw[j][e];
        }
    }
    __syncthreads();
    if (wave > 0 || !in) return;
    float *part = p.part + quad * (W + 1) * p.D;
    float f[E * W];  // [channel][tap] as the weights lie
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            db[e] += sums[n][W * E + e][lane];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] += sums[n][j * E + e][lane];
        }
#pragma unroll
        for (int j = 0; j < W; ++j) f[e * W + j] = dw[j][e];
    }
#pragma unroll
    for (int i = 0; i < E * W / 4; ++i)
        reinterpret_cast<f32x4 *>(part + (int64_t)c * W)[i] = f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        reinterpret_cast<f32x4 *>(part + (int64_t)W * p.D + c)[i] =
            f32x4{db[4 * i], db[4 * i + 1], db[4 * i + 2], db[4 * i + 3]};
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

void conv_shape(ConvParams &p, int width, bool backward) {
    p.tile = 32;
    p.places = p.T / p.tile + p.batch;
    if (!backward) return;
    // whole groups with the W - 1 tokens behind a piece: as many pieces as are resident (two wavefronts a SIMD) where
    // they fit with 16 groups or fewer (32 x 1024 tokens, 1536 channels: 14 groups 71 us, 8 76, 4 80), or 8 groups,
    // which even out (40 ragged prompts of 80 on average, 10240 channels 73 us, with 16 groups 99; 64 x 512 tokens,
    // 4096 channels 190 and 201)
    const int rows = width == 3 ? kAhead<3> : kAhead<4>;
    const int64_t cblocks = blocks_of(p.D, 64 * kGradChannels);
    auto pieces = [&](int groups) {
        p.tile = groups * rows - (width - 1);
        p.places = p.T / p.tile + p.batch;
        return p.places * cblocks;
    };
    int groups = 2;
    while (groups <= 16 && pieces(groups) > 2048) ++groups;
    if (groups > 16) pieces(8);
}
int64_t conv_parts(const ConvParams &p) { return blocks_of(p.places, 4); }
int64_t conv_threads(const ConvParams &p) {
    return blocks_of(p.places, 4) * 4 * blocks_of(p.D, 64 * kGradChannels) * 64;
}

hipError_t launch_conv(const ConvParams &p, int width, hipStream_t s) {
    const dim3 grid((unsigned)blocks_of(p.places * blocks_of(p.D, 512), 4));
    // outputs that the 256 MB cache would not hold for the next kernel pass by it (0.9 GB 364 -> 353 us)
    const bool past = (int64_t)p.T * p.D * 2 > (int64_t)256 << 20;
    return by_width(width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        if (past)
            conv_fwd<W, true><<<grid, 256, 0, s>>>(p);
        else
            conv_fwd<W, false><<<grid, 256, 0, s>>>(p);
    });
}
hipError_t launch_conv_step(const ConvParams &p, int width, hipStream_t s) {
    return by_width(width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        auto grid = [&](int seqs) { return dim3((unsigned)blocks_of(blocks_of(p.batch, seqs) * (p.D / 8), 256)); };
        if (p.batch >= 16)
            conv_step<W, kStepSeqs><<<grid(kStepSeqs), 256, 0, s>>>(p);
        else
            conv_step<W, 1><<<grid(1), 256, 0, s>>>(p);
    });
}
hipError_t launch_conv_grad(const ConvParams &p, int width, hipStream_t s) {
    const int64_t quads = conv_parts(p);
    const dim3 grid((unsigned)(quads * blocks_of(p.D, 64 * kGradChannels)));
    hipError_t e = by_width(width, [&](auto w) { conv_grad<decltype(w)::value><<<grid, 256, 0, s>>>(p); });
    if (e != hipSuccess) return e;
    const int64_t row = (int64_t)(width + 1) * p.D;
    return launch_sums(Sums{{Sum{p.part, (int)quads, row, (int64_t)width * p.D, p.dweight},
                             Sum{p.part + (int64_t)width * p.D, (int)quads, row, p.D, p.dbias}}},
                       s);
}

}  // namespace layer
}  // namespace ssd
