// Selective scan over ragged batches: h = exp(dts A) h + dts x B, y = C.h + D x,
// gated by silu(z).  Every channel and state decays on its own, so there is no
// matrix product in it: a token costs each (channel, state) an exponential, two
// products and two fused adds, about 8 issue slots with the exponential at a
// quarter of the rate, and this, not memory, is what bounds it.
//
// A workgroup takes 64 channels of a sequence (or of one of its segments) and a
// wavefront 4 states of them, a channel a lane: B and C are then the same for
// all lanes and come through scalar registers, and what belongs to a token and
// channel alone (softplus, gate, input and output) is done once, by all threads
// together, for a tile of 16 tokens at a time, and handed over through LDS.
//
// Sequences longer than a share of the card are cut into segments: a pass over
// all but their last ones leaves the states that each would from zero, with the
// sum of its time steps, and a segment's workgroup chains those ahead of it
// before it starts.
#include "ssd.h"
#include "ssd_layer.hpp"
#include "ssd_selective.hpp"

namespace ssd {
namespace layer {
namespace {

// kOutputs: the scan itself.  kStates: the pass that leaves the segments' states
// of cut sequences.  kMarks: the state ahead of every kGradTile tokens, for the
// backward pass.
enum Walk { kOutputs, kStates, kMarks };
template <int NW, Walk WALK>
__global__ __launch_bounds__(NW * 64) void scan_walk(ScanParams p) {
    constexpr int NT = NW * 64, kItems = (kTile * 16 + NT - 1) / NT;
    constexpr bool OUT = WALK == kOutputs, STATES = WALK == kStates;
    __shared__ float2 sdt[kTile][64];                   // time step, and times x
    __shared__ float sy[OUT ? NW : 1][kTile][64];    // a wavefront's share of C.h
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int place = blockIdx.x / p.blocks;
    Seq q;
    int s;
    if (!find_piece(p.qsl, p.batch, p.T, p.seg, place, q, s)) return;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[q.b] : q.b;
    if (slot >= (int64_t)p.max_slots) return;  // padding
    const int nseg = q.len > p.seg ? (q.len + p.seg - 1) / p.seg : 1;
    if (STATES && s >= nseg - 1) return;
    const Span w = span_of(p, blockIdx.x % p.blocks);
    const int t0 = s * p.seg, t1 = min(q.len, t0 + p.seg);
    const bool init = p.state_in != nullptr && (p.init_all || (p.has_init != nullptr && p.has_init[q.b] != 0));

    // this lane's channel, and this wavefront's states
    const int n0 = wave * 4;
    const bool mine = lane < w.nch && n0 < p.N;
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    const int64_t at = (int64_t)ch * p.N + n0;
    const int64_t state = slot * p.D * p.N + at;
    float A[4] = {}, h[4] = {};
    if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = p.A[at + i] * kLog2e;
    }
    const int64_t first = nseg > 1 ? cut_place(p, q) : 0;  // of this sequence's segments' states
    if (mine && s == 0) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (nseg > 1 && !STATES) {
            // the pass kept what the pool held, which the last segment may have replaced by now
            v = *reinterpret_cast<const f32x4 *>(p.parts + (first + nseg - 1) * p.D * p.N + at);
        } else if (init) {
            v = p.state_bf16 ? load_state4<true>(p.state_in, state) : load_state4<false>(p.state_in, state);
        }
        if (STATES) *reinterpret_cast<f32x4 *>(p.parts + (first + nseg - 1) * p.D * p.N + at) = v;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = v[i];
    }
    if (mine && !STATES && s > 0) chain_states(p, first, s, at, ch, A, h);

    // the tokens and channels this thread prepares and finishes: 4 channels of a token an item
    const uint16_t *xp = p.x + (int64_t)q.begin * p.xs + w.ch0, *dtp = p.dt + (int64_t)q.begin * p.dts + w.ch0;
    const uint16_t *zp = p.z != nullptr ? p.z + (int64_t)q.begin * p.zs + w.ch0 : nullptr;
    const uint16_t *Bp = p.B + (int64_t)q.begin * p.bs + w.g * p.N + n0;
    const uint16_t *Cp = p.C + (int64_t)q.begin * p.cs + w.g * p.N + n0;
    u32x2 nx[kItems], nd[kItems], nz[kItems];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = t + i / 16, c = (i % 16) * 4;
            nx[k] = nd[k] = nz[k] = u32x2{0, 0};
            if (i >= kTile * 16 || r >= t1 || c >= w.nch) continue;
            nx[k] = *reinterpret_cast<const u32x2 *>(xp + (int64_t)r * p.xs + c);
            nd[k] = *reinterpret_cast<const u32x2 *>(dtp + (int64_t)r * p.dts + c);
            if (OUT && zp != nullptr) nz[k] = *reinterpret_cast<const u32x2 *>(zp + (int64_t)r * p.zs + c);
        }
    };
    float steps = 0.f;  // sum of this lane's channel's time steps (first wavefront)
    fetch(t0);
    for (int t = t0; t < t1; t += kTile) {
        u32x2 rx[kItems], rz[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = i / 16, c = (i % 16) * 4;
            rx[k] = nx[k];
            rz[k] = nz[k];
            if (i >= kTile * 16 || c >= w.nch) continue;
            float x[4], d[4];
            widen4(nx[k], x);
            widen4(nd[k], d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float step = time_step(p, d[e], w.ch0 + c + e);
                sdt[r][c + e] = make_float2(step, step * x[e]);
            }
        }
        if (t + kTile < t1) fetch(t + kTile);
        __syncthreads();
        if (n0 < p.N) {
            const int n = min(kTile, t1 - t);
            auto token = [&](int i) {
                if (WALK == kMarks && i % kGradTile == 0 && mine)
                    *reinterpret_cast<f32x4 *>(mark_at(p, q, t + i, n0, ch)) = f32x4{h[0], h[1], h[2], h[3]};
                const float2 e = sdt[i][lane];
                const Quad B = quad_at(Bp + (int64_t)(t + i) * p.bs);
                float y = 0.f;
                Quad C = {};
                if (OUT) C = quad_at(Cp + (int64_t)(t + i) * p.cs);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = __builtin_fmaf(fast_exp2(e.x * A[j]), h[j], e.y * B.v[j]);
                    if (OUT) y = __builtin_fmaf(C.v[j], h[j], y);
                }
                if (STATES) steps += e.x;
                if (OUT) sy[wave][i][lane] = y;
            };
            if (n == kTile) {
#pragma unroll
                for (int i = 0; i < kTile; ++i) token(i);
            } else {
#pragma unroll 1
                for (int i = 0; i < n; ++i) token(i);
            }
        }
        __syncthreads();
        if constexpr (OUT) {
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int i = threadIdx.x + k * NT, r = i / 16, c = (i % 16) * 4;
                if (i >= kTile * 16 || t + r >= t1 || c >= w.nch) continue;
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < NW; ++v)
                    if (v * 4 < p.N) y += *reinterpret_cast<const f32x4 *>(&sy[v][r][c]);
                if (p.Dskip != nullptr) {
                    float x[4];
                    widen4(rx[k], x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(p.Dskip[w.ch0 + c + e], x[e], y[e]);
                }
                if (zp != nullptr) {
                    float z[4];
                    widen4(rz[k], z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] *= z[e] * sigmoid_f(z[e]);
                }
                *reinterpret_cast<u32x2 *>(p.y + (int64_t)(q.begin + t + r) * p.D + w.ch0 + c) =
                    u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            }
        }
    }
    if (!mine) return;
    const f32x4 v = {h[0], h[1], h[2], h[3]};
    if constexpr (STATES) {
        *reinterpret_cast<f32x4 *>(p.parts + (first + s) * p.D * p.N + at) = v;
        if (wave == 0) p.steps[(first + s) * p.D + ch] = steps;
    } else if (OUT && s == nseg - 1) {
        if (p.state_bf16)
            store_state4<true>(p.state_out, state, v);
        else
            store_state4<false>(p.state_out, state, v);
    }
}

template <Walk WALK>
hipError_t walk(const ScanParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.places * p.blocks));
    by_waves(waves_of(p.N), [&](auto n) {
        constexpr int NW = decltype(n)::value;
        scan_walk<NW, WALK><<<grid, NW * 64, 0, s>>>(p);
    });
    return hipGetLastError();
}
}  // namespace

void scan_shape(ScanParams &p, bool backward) {
    p.Dg = p.D / p.G;
    p.blocks = p.G * ((p.Dg + 63) / 64);
    // A workgroup's share of the card: four wavefronts a SIMD, 1024 workgroups of 4
    const int64_t share = (int64_t)p.T * p.blocks / 1024;
    int64_t seg = (share + kTile - 1) / kTile * kTile;
    seg = seg < 256 ? 256 : seg;
    p.seg = (int)seg;
    p.places = p.T / seg + p.batch;
    p.cuts = p.T / (seg + 1) < p.batch ? p.T / (seg + 1) : p.batch;
    p.cut_places = p.cuts > 0 ? p.T / seg + p.cuts : 0;
    (void)backward;
}

int64_t scan_threads(const ScanParams &p, bool backward) {
    const int64_t walk = p.places * p.blocks * 64 * waves_of(p.N);
    const int64_t sums = backward ? (int64_t)p.T * p.G * (p.N / 2) + 255 : 0;
    return walk > sums ? walk : sums;
}

hipError_t launch_scan_states(const ScanParams &p, hipStream_t s) {
    return p.cut_places > 0 ? walk<kStates>(p, s) : hipSuccess;
}
hipError_t launch_scan_marks(const ScanParams &p, hipStream_t s) { return walk<kMarks>(p, s); }
hipError_t launch_scan(const ScanParams &p, hipStream_t s) {
    const hipError_t e = launch_scan_states(p, s);
    return e != hipSuccess ? e : walk<kOutputs>(p, s);
}

}  // namespace layer
}  // namespace ssd
