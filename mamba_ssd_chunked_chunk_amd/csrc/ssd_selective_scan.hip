// Selective scan over ragged batches: h = exp(dts A) h + dts x B, y = C.h + D x,
// gated by silu(z).  Every channel and state decays on its own, so there is no
// matrix product in it: a token costs each (channel, state) an exponential, two
// products and two fused adds, and this, not memory, is what bounds it: 11 ns a
// state and token for the 64 channels of a wavefront on one SIMD, at which 8 x 2048
// tokens of 4096 channels and 16 states take 180 us, while all a wavefront does is 33
// instructions a token, 20 of them for its states.  They take 293 us (1.1 vector
// instructions a cycle and compute unit); 65536 tokens of 2048 channels, cut into 64
// segments, which all but doubles the work, 804 us.
//
// A workgroup takes 64 channels of a sequence (or of one of its segments) and a
// wavefront 4 states of them, a channel a lane.  What belongs to a token and
// channel alone (softplus, gate, input and output) is done once, by all threads
// together, for a tile of 16 tokens at a time, and handed over through LDS, as
// are B and C, which all lanes of a wavefront read alike.  (Scalar loads, which
// return in any order, would have to be waited for all at once: 8 x 2048 tokens
// of 4096 channels 441 us in place of 302, though a scalar operand costs the
// adds less.)
//
// Sequences longer than a share of the card are cut into segments, in two
// launches: the first walks whole sequences and first segments, which leave
// their states, and forms the states that the segments between the first and the
// last would leave from zero, with the sums of their time steps; the second
// walks the other segments, each after chaining what lies ahead of it.
#include <math.h>

#include <algorithm>

#include "ssd.h"
#include "ssd_layer.hpp"
#include "ssd_selective.hpp"

namespace ssd {
namespace layer {
namespace {

// kOutputs: the scan itself.  kMarks: the state ahead of every kGradTile tokens,
// for the backward pass.  kStates: the state a segment leaves from zero.
enum Walk { kOutputs, kMarks, kStates };

template <int NW>
struct Shared {
    float2 step[kTile][64];  // time step, and times x
    f32x4 B[kTile][NW], C[kTile][NW];
    float y[NW][kTile][64];  // a wavefront's share of C.h
};

// One segment of a sequence (or all of it) and 64 channels.
template <int NW, Walk WALK>
__device__ __forceinline__ void walk(const ScanParams &p, Shared<NW> &lds, const Seq &q, int s, int nseg,
                                     const Span &w) {
    constexpr int NT = NW * 64, kItems = (kTile * 16 + NT - 1) / NT;
    constexpr bool OUT = WALK == kOutputs, STATES = WALK == kStates;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int t0 = s * p.seg, t1 = nseg > 1 ? min(q.len, t0 + p.seg) : q.len;
    const bool init = p.state_in != nullptr && (p.init_all || (p.has_init != nullptr && p.has_init[q.b] != 0));

    // this lane's channel, and this wavefront's states
    const int n0 = wave * 4;
    const bool mine = lane < w.nch && n0 < p.N;
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    const int64_t at = (int64_t)ch * p.N + n0;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[q.b] : q.b;
    const int64_t state = slot * p.D * p.N + at;
    const int64_t first = nseg > 1 ? cut_place(p, q) : 0;  // of this sequence's segments' states
    float A[4] = {}, h[4] = {};
    if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = p.A[at + i] * kLog2e;
        if (!STATES && s == 0 && init) {
            const f32x4 v = p.state_bf16 ? load_state4<true>(p.state_in, state) : load_state4<false>(p.state_in, state);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = v[i];
        }
        if (!STATES && s > 0) chain_states(p, first, s, at, ch, A, h);
    }
    if (OUT && n0 >= p.N)  // no states, no share
        for (int i = 0; i < kTile; ++i) lds.y[wave][i][lane] = 0.f;

    // the tokens and channels this thread prepares and finishes: 4 channels of a token an item, the same ones in
    // every item
    const int c = (threadIdx.x % 16) * 4, r0 = threadIdx.x / 16;
    const bool in = c < w.nch;
    float bias[4] = {}, skip[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (in && p.bias != nullptr) bias[e] = p.bias[w.ch0 + c + e];
        if (OUT && in && p.Dskip != nullptr) skip[e] = p.Dskip[w.ch0 + c + e];
    }
    // rows by an address that all lanes share and the lane's own offset in bytes; rows and channels that are not there
    // are read as the last and the first there are, and go no further than LDS
    const int64_t row0 = q.begin + t0;
    const bool gate = OUT && p.z != nullptr;
    Scalar<const uint16_t> xp(p.x + row0 * p.xs + w.ch0), dp(p.dt + row0 * p.dts + w.ch0);
    Scalar<const uint16_t> zp(gate ? p.z + row0 * p.zs + w.ch0 : p.x);
    Scalar<uint16_t> yp(OUT ? p.y + row0 * p.D + w.ch0 : nullptr);
    const uint32_t xs = (uint32_t)p.xs * 2, ds = (uint32_t)p.dts * 2, zs = (uint32_t)p.zs * 2, ys = (uint32_t)p.D * 2;
    uint32_t xo[kItems], od[kItems], zo[kItems];
    auto offsets = [&](int n) {  // of a tile of n tokens
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const uint32_t r = min(r0 + k * (NT / 16), n - 1), cc = in ? c * 2 : 0;
            xo[k] = r * xs + cc;
            od[k] = r * ds + cc;
            zo[k] = r * zs + cc;
        }
    };
    // two elements of B or of C of a token, by a thread (twice where there are outputs)
    constexpr int kWords = OUT ? 2 : 1;
    const int half = p.N / 2, each = OUT ? p.N : half;
    uint32_t nw[kWords] = {};
    const uint16_t *wp[kWords];
    float *wl[kWords];
    int64_t ws[kWords];
    int wt[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int i = threadIdx.x + k * NT, t = i / each, j = i % each;
        const bool ofC = OUT && j >= half;
        const int e = (ofC ? j - half : j) * 2;
        wt[k] = t < kTile ? t : INT32_MAX;
        ws[k] = ofC ? p.cs : p.bs;
        wp[k] = (ofC ? p.C : p.B) + (row0 + t) * ws[k] + w.g * p.N + e;
        wl[k] = t < kTile ? reinterpret_cast<float *>(ofC ? &lds.C[t][0] : &lds.B[t][0]) + e : nullptr;
    }
    u32x2 nx[kItems], nd[kItems], nz[kItems];
    auto fetch = [&](int t) {
        if (t + kTile > t1) offsets(t1 - t);
        xp.hold();
        dp.hold();
        zp.hold();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            nx[k] = xp.at<u32x2>(xo[k]);
            nd[k] = dp.at<u32x2>(od[k]);
            nz[k] = u32x2{0, 0};
            if (gate) nz[k] = zp.at<u32x2>(zo[k]);
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if (wt[k] < t1 - t) nw[k] = *reinterpret_cast<const uint32_t *>(wp[k]);
            wp[k] += kTile * ws[k];
        }
        xp.ptr += kTile * p.xs;
        dp.ptr += kTile * p.dts;
        if (gate) zp.ptr += kTile * p.zs;
    };
    float steps = 0.f;  // sum of this lane's channel's time steps
    if (t0 < t1) {
        offsets(kTile);
        fetch(t0);
    }
    // (loads that have to be here before the loop: a wait inside it would be for the last tile's stores too)
#pragma unroll
    for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(bias[e]), "+v"(skip[e]), "+v"(A[e]), "+v"(h[e]));
    for (int t = t0; t < t1; t += kTile) {
        u32x2 rx[kItems], rz[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int r = r0 + k * (NT / 16);
            rx[k] = nx[k];
            rz[k] = nz[k];
            if (r >= kTile) continue;
            float x[4], d[4];
            widen4(nx[k], x);
            widen4(nd[k], d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float step = time_step(p, d[e] + bias[e]);
                lds.step[r][c + e] = make_float2(step, step * x[e]);
            }
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            if (wl[k] != nullptr) *reinterpret_cast<float2 *>(wl[k]) = make_float2(bf16x2_lo(nw[k]), bf16x2_hi(nw[k]));
        if (t + kTile < t1) fetch(t + kTile);
        __syncthreads();
        if (n0 < p.N) {
            const int n = min(kTile, t1 - t);
            struct Token {
                float2 e;
                f32x4 B, C;
            };
            auto read = [&](int i) {
                return Token{lds.step[i][lane], lds.B[i][wave], OUT ? lds.C[i][wave] : f32x4{0.f, 0.f, 0.f, 0.f}};
            };
            auto token = [&](int i, const Token &m) {
                if (WALK == kMarks && i % kGradTile == 0 && mine)
                    *reinterpret_cast<f32x4 *>(mark_at(p, q, t + i, n0, ch)) = f32x4{h[0], h[1], h[2], h[3]};
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = __builtin_fmaf(m.e.y, m.B[j], fast_exp2(m.e.x * A[j]) * h[j]);
                    if (OUT) y = j == 0 ? m.C[j] * h[j] : __builtin_fmaf(m.C[j], h[j], y);
                }
                if (STATES) steps += m.e.x;
                if (OUT) lds.y[wave][i][lane] = y;
            };
            if (n == kTile) {
                // a token is read while the one ahead of it is worked on (the compiler would not move it past the
                // stores between)
                Token next = read(0);
#pragma unroll
                for (int i = 0; i < kTile; ++i) {
                    const Token m = next;
                    if (i + 1 < kTile) next = read(i + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    token(i, m);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < n; ++i) token(i, read(i));
            }
        }
        __syncthreads();
        if constexpr (OUT) {
            u32x2 out[kItems];
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int r = min(r0 + k * (NT / 16), kTile - 1);
                f32x4 y = *reinterpret_cast<const f32x4 *>(&lds.y[0][r][c]);
#pragma unroll
                for (int v = 1; v < NW; ++v) y += *reinterpret_cast<const f32x4 *>(&lds.y[v][r][c]);
                float x[4];
                widen4(rx[k], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(skip[e], x[e], y[e]);
                if (gate) {
                    float z[4];
                    widen4(rz[k], z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] *= z[e] * sigmoid_f(z[e]);
                }
                out[k] = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            }
            yp.hold();
            // the next tile's rows are waited for here, ahead of the stores
#pragma unroll
            for (int k = 0; k < kItems; ++k) asm volatile("" : "+v"(nx[k]), "+v"(nd[k]), "+v"(nz[k]));
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int r = r0 + k * (NT / 16);
                if (r < kTile && t + r < t1 && in) yp.put((uint32_t)r * ys + c * 2, out[k]);
            }
            yp.ptr += (int64_t)kTile * p.D;
        }
    }
    if (!mine) return;
    const f32x4 v = {h[0], h[1], h[2], h[3]};
    if (s < nseg - 1) {
        // What chain_states reads: the first segment's state, which holds what entered it, and the others' from zero.
        // The later walk of those, from what entered them, leaves nothing: other workgroups of its launch read them.
        if (STATES || s == 0) *reinterpret_cast<f32x4 *>(p.parts + (first + s) * p.D * p.N + at) = v;
        if (STATES && wave == 0) p.steps[(first + s) * p.D + ch] = steps;
    } else if (OUT) {
        if (p.state_bf16)
            store_state4<true>(p.state_out, state, v);
        else
            store_state4<false>(p.state_out, state, v);
    }
}

__device__ __forceinline__ bool padding(const ScanParams &p, int b) {
    return p.cache_idx != nullptr && p.cache_idx[b] >= p.max_slots;
}

template <int NW, Walk WALK>
__global__ __launch_bounds__(NW * 64) void scan_first(ScanParams p) {
    __shared__ Shared<NW> lds;
    Piece w;
    if (!piece_at<false>(p, blockIdx.x / p.blocks, w) || padding(p, w.q.b)) return;
    const Span c = span_of(p, blockIdx.x % p.blocks);
    if (w.s == 0)
        walk<NW, WALK>(p, lds, w.q, w.s, w.nseg, c);
    else if (w.s < w.nseg - 1)
        walk<NW, kStates>(p, lds, w.q, w.s, w.nseg, c);
}

template <int NW, Walk WALK>
__global__ __launch_bounds__(NW * 64) void scan_rest(ScanParams p) {
    __shared__ Shared<NW> lds;
    Piece w;
    if (!piece_at<true>(p, blockIdx.x / p.blocks, w) || w.s == 0 || padding(p, w.q.b)) return;
    walk<NW, WALK>(p, lds, w.q, w.s, w.nseg, span_of(p, blockIdx.x % p.blocks));
}

template <Walk WALK>
hipError_t launch_walk(const ScanParams &p, hipStream_t s) {
    by_waves(waves_of(p.N), [&](auto n) {
        constexpr int NW = decltype(n)::value;
        scan_first<NW, WALK><<<dim3((unsigned)(p.places * p.blocks)), NW * 64, 0, s>>>(p);
        if (p.cut_places > 0)
            scan_rest<NW, WALK><<<dim3((unsigned)(p.cut_places * p.blocks)), NW * 64, 0, s>>>(p);
    });
    return hipGetLastError();
}
}  // namespace

// (total_len stays below 2^30)
constexpr int64_t kSegLimit = 1 << 29;
void scan_shape(ScanParams &p, bool backward) {
    p.Dg = p.D / p.G;
    p.blocks = p.G * ((p.Dg + 63) / 64);
    // Segments: long enough that a workgroup's chaining of those ahead of it stays below its walk (one sequence of 4096
    // tokens and 2048 channels 79, 68, 75 us with 64, 128, 256 tokens), and that there are no more of them than
    // balance the card: 8 wavefronts a SIMD (65536 tokens 888, 855, 895 us with 512, 1024, 2048), in the backward
    // pass, which would repeat more work, 2 (one of 4096 tokens 276, 250, 266, 407 us with 64, 128, 256, 512).  Where
    // the sequences alone come near 2 wavefronts a SIMD only those that stand out are cut (8 x 2048 tokens of 4096
    // channels 293 us uncut, 362 in segments of 512, their backward pass 1071 and 1433; 32 ragged prompts of 1372 on
    // average 959, 865, 866, 939 us with 512, 1024, 2048, 4096; with half as many wavefronts 16 x 1024 tokens of 4
    // states 172 us uncut and 187 in segments of 256, 4 x 1024 tokens of 16 states 125 and 113 in segments of 128).
    const int64_t waves = (int64_t)p.blocks * (backward ? grad_waves_of(p.N) : waves_of(p.N));
    const int64_t resident = 2048;
    int64_t seg = std::max<int64_t>(backward ? 32 : 64, (int64_t)((backward ? 1.0 : 1.5) * sqrt((double)p.T)));
    seg = std::max(seg, (int64_t)p.T * waves / (backward ? resident : 4 * resident));
    if (p.batch * waves >= resident * 3 / 4) seg = std::max<int64_t>(seg, p.T / p.batch);
    seg = (seg + kTile - 1) / kTile * kTile;
    if (seg > kSegLimit) seg = kSegLimit;
    p.seg = (int)seg;
    p.cut = 2 * p.seg;
    // (256 x 30 tokens 80 us with gaps, 107 without; 200 ragged prompts of 155 on average 305 and 245)
    p.listed = p.batch <= 64 || (p.batch <= 256 && p.T / p.batch >= 128);
    p.places = p.T / seg + p.batch;
    p.cuts = std::min<int64_t>(p.T / ((int64_t)p.cut + 1), p.batch);
    p.cut_places = p.cuts > 0 ? p.T / seg + p.cuts : 0;
}

int64_t scan_threads(const ScanParams &p, bool backward) {
    // (the gradients' workgroups are the larger ones with 4 states, the walks' above 16)
    const int waves = backward ? std::max(waves_of(p.N), grad_waves_of(p.N)) : waves_of(p.N);
    const int64_t walk = p.places * p.blocks * 64 * waves;
    const int64_t sums = backward ? (int64_t)p.T * p.G * (p.N / 2) + 8 * ((int64_t)p.D * (p.N + 2)) + 1024 : 0;
    return walk > sums ? walk : sums;
}

hipError_t launch_scan_marks(const ScanParams &p, hipStream_t s) { return launch_walk<kMarks>(p, s); }
hipError_t launch_scan(const ScanParams &p, hipStream_t s) { return launch_walk<kOutputs>(p, s); }

}  // namespace layer
}  // namespace ssd
