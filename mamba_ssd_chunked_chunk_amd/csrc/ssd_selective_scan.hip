// Selective scan over ragged batches: h = exp(dts A) h + dts x B, y = C.h + D x,
// gated by silu(z).  Every channel and state decays on its own, so there is no
// matrix product in it: a token costs each (channel, state) an exponential, two
// products and two fused adds, and this, not memory, is what bounds it.
//
// A workgroup takes 64 channels of a sequence (or of one of its segments) and a
// wavefront 4 states of them, a channel a lane: B and C are then the same for
// all lanes and come through scalar registers, and what belongs to a token and
// channel alone (softplus, gate, input and output) is done once, by all threads
// together, for a tile of 16 tokens at a time, and handed over through LDS.
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

constexpr int kGroup = 4;  // tokens whose B, C and steps are on their way while as many are worked on

// kOutputs: the scan itself.  kMarks: the state ahead of every kGradTile tokens,
// for the backward pass.  kStates: the state a segment leaves from zero.
enum Walk { kOutputs, kMarks, kStates };

template <int NW>
struct Shared {
    float2 step[kTile][64];  // time step, and times x
    union {
        float y[NW][kTile][64];  // a wavefront's share of C.h
        f32x4 B[kTile][NW];      // (walks without outputs)
    };
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
    const uint16_t *Bp = p.B + row0 * p.bs + w.g * p.N + n0, *Cp = p.C + row0 * p.cs + w.g * p.N + n0;
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
    // Walks without outputs take B through LDS, two elements of a token by each of the first threads: few wavefronts a
    // unit do not hide what scalar loads wait for (8 x 2048 tokens of 4096 channels 350 -> 245 us).
    const int bt = threadIdx.x / (p.N / 2), bj = threadIdx.x % (p.N / 2) * 2;
    const uint16_t *wp = OUT ? nullptr : p.B + (row0 + bt) * p.bs + w.g * p.N + bj;
    uint32_t nb = 0;
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
        if (!OUT && bt < kTile && t + bt < t1) nb = *reinterpret_cast<const uint32_t *>(wp);
        if (!OUT) wp += kTile * p.bs;
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
        if (!OUT && bt < kTile)
            *reinterpret_cast<float2 *>(reinterpret_cast<float *>(&lds.B[bt][0]) + bj) =
                make_float2(bf16x2_lo(nb), bf16x2_hi(nb));
        if (t + kTile < t1) fetch(t + kTile);
        __syncthreads();
        if (n0 < p.N) {
            const int n = min(kTile, t1 - t);
            auto token = [&](int i, const float2 &e, const Quad &B, const Quad &C) {
                if (WALK == kMarks && i % kGradTile == 0 && mine)
                    *reinterpret_cast<f32x4 *>(mark_at(p, q, t + i, n0, ch)) = f32x4{h[0], h[1], h[2], h[3]};
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = __builtin_fmaf(e.y, B.v[j], fast_exp2(e.x * A[j]) * h[j]);
                    if (OUT) y = j == 0 ? C.v[j] * h[j] : __builtin_fmaf(C.v[j], h[j], y);
                }
                if (STATES) steps += e.x;
                if (OUT) lds.y[wave][i][lane] = y;
            };
            if (n == kTile) {
                Words next[kGroup], now[kGroup];
                float2 en[kGroup], ee[kGroup];
                f32x4 bn[kGroup], bb[kGroup];
                auto ahead = [&](int g) {
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        if constexpr (OUT) {
                            words_at(Bp, next[i].b);
                            Bp += p.bs;
                            words_at(Cp, next[i].c);
                            Cp += p.cs;
                        } else {
                            bn[i] = lds.B[g + i][wave];
                        }
                        en[i] = lds.step[g + i][lane];
                    }
                };
                ahead(0);
#pragma unroll
                for (int g = 0; g < kTile; g += kGroup) {
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        if constexpr (OUT)
                            now[i] = next[i];
                        else
                            bb[i] = bn[i];
                        ee[i] = en[i];
                    }
                    if (g + kGroup < kTile) ahead(g + kGroup);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        if constexpr (OUT)
                            token(g + i, ee[i], quad_of(now[i].b[0], now[i].b[1]), quad_of(now[i].c[0], now[i].c[1]));
                        else
                            token(g + i, ee[i], Quad{{bb[i][0], bb[i][1], bb[i][2], bb[i][3]}}, Quad{});
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    if constexpr (OUT) {
                        token(i, lds.step[i][lane], quad_at(Bp + (int64_t)i * p.bs), quad_at(Cp + (int64_t)i * p.cs));
                    } else {
                        const f32x4 B = lds.B[i][wave];
                        token(i, lds.step[i][lane], Quad{{B[0], B[1], B[2], B[3]}}, Quad{});
                    }
                }
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
        *reinterpret_cast<f32x4 *>(p.parts + (first + s) * p.D * p.N + at) = v;
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

void scan_shape(ScanParams &p, bool backward) {
    p.Dg = p.D / p.G;
    p.blocks = p.G * ((p.Dg + 63) / 64);
    // Segments: long enough that a workgroup's chaining of those ahead of it stays below its walk (the root of T: one
    // sequence of 4096 tokens and 2048 channels 178, 88, 83, 104 us with 32, 64, 128, 256 tokens), and that there are
    // no more of them than balance the card: 16 workgroups of 4 wavefronts a unit (65536 tokens 849, 872, 1026 us with
    // 512, 768, 2048), in the backward pass, which would repeat more work, the two wavefronts a SIMD that are resident
    // (8 x 2048 tokens, 4096 channels 1.25 ms uncut, 1.58 in segments of 512).  Where the sequences alone fill
    // the card only those that stand out are cut (32 ragged prompts 936, 860, 890 us at 686, 1024, 1376 tokens; 40 of
    // 300 tokens 160 us in segments of 112, 110 uncut).
    const int64_t waves = (int64_t)p.blocks * waves_of(p.N);
    int64_t seg = std::max<int64_t>(backward ? 32 : 64, (int64_t)sqrt((double)p.T));
    seg = std::max(seg, (int64_t)p.T * waves / (backward ? 2048 : 16384));
    if (p.batch * waves >= (backward ? 2048 : 4096))
        seg = std::max<int64_t>(seg, (int64_t)(p.T / p.batch) * (backward ? 4 : 3) / 4);
    seg = (seg + kTile - 1) / kTile * kTile;
    p.seg = (int)seg;
    p.cut = (int)std::min<int64_t>(2 * seg, INT32_MAX);
    p.places = p.T / seg + p.batch;
    p.cuts = std::min<int64_t>(p.T / ((int64_t)p.cut + 1), p.batch);
    p.cut_places = p.cuts > 0 ? p.T / seg + p.cuts : 0;
}

int64_t scan_threads(const ScanParams &p, bool backward) {
    const int64_t walk = p.places * p.blocks * 64 * waves_of(p.N);
    const int64_t sums = backward ? (int64_t)p.T * p.G * (p.N / 2) + 8 * ((int64_t)p.D * (p.N + 2)) + 1024 : 0;
    return walk > sums ? walk : sums;
}

hipError_t launch_scan_marks(const ScanParams &p, hipStream_t s) { return launch_walk<kMarks>(p, s); }
hipError_t launch_scan(const ScanParams &p, hipStream_t s) { return launch_walk<kOutputs>(p, s); }

}  // namespace layer
}  // namespace ssd
