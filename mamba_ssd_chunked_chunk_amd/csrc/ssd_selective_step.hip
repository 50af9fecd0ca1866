// Selective scan, one token per sequence, by the recurrence itself.  A thread
// holds 4 consecutive states of a channel (16 bytes in fp32) of several
// sequences, so the decays are read once for all of them; the lanes of a channel
// add their shares of C.h.  The states are read once and written once, and that
// is the bound: 512 sequences of 4096 channels and 16 states in fp32, 286 MB, 62 us
// (4.6 TB/s).
#include "ssd_selective.hpp"

namespace ssd {
namespace layer {
namespace {
constexpr int kThreads = 256;

// sum over each aligned group of LANES lanes
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES >= 2) v = dpp_add_all<0xB1>(v);   // quad_perm [1,0,3,2]
    if constexpr (LANES >= 4) v = dpp_add_all<0x4E>(v);   // quad_perm [2,3,0,1]
    if constexpr (LANES >= 8) v = dpp_add_all<0x141>(v);  // row_half_mirror
    if constexpr (LANES >= 16) v = dpp_add_all<0x140>(v); // row_mirror
    return v;
}

template <int LANES, int SEQS, bool SB>
__global__ __launch_bounds__(kThreads) void scan_step(ScanParams p, int cblocks) {
    const int cb = blockIdx.x % cblocks, b0 = blockIdx.x / cblocks * SEQS;
    const int ch = cb * (kThreads / LANES) + threadIdx.x / LANES, n0 = threadIdx.x % LANES * 4;
    const bool in = ch < p.D && n0 < p.N;
    const int64_t at = (int64_t)ch * p.N + n0;
    const int g = ch / p.Dg;
    f32x4 h[SEQS];
    int64_t slot[SEQS];
    uint32_t bw[SEQS][2], cw[SEQS][2], x[SEQS], dt[SEQS], z[SEQS];
    // all that is read, ahead of all that is computed
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const int64_t b = b0 + k;
        slot[k] = b < p.batch ? (int64_t)p.cache_idx[b] : (int64_t)p.max_slots;  // max_slots or more: nothing
        const bool init = b < p.batch && p.has_init != nullptr && p.has_init[b] != 0;
        h[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        x[k] = dt[k] = z[k] = bw[k][0] = bw[k][1] = cw[k][0] = cw[k][1] = 0;
        if (!in || slot[k] >= (int64_t)p.max_slots) continue;
        if (init) h[k] = load_state4<SB>(p.state_in, slot[k] * p.D * p.N + at);
        const uint32_t *B = reinterpret_cast<const uint32_t *>(p.B + b * p.bs + g * p.N + n0);
        const uint32_t *C = reinterpret_cast<const uint32_t *>(p.C + b * p.cs + g * p.N + n0);
        bw[k][0] = B[0];
        bw[k][1] = B[1];
        cw[k][0] = C[0];
        cw[k][1] = C[1];
        x[k] = p.x[b * p.xs + ch];
        dt[k] = p.dt[b * p.dts + ch];
        if (p.z != nullptr) z[k] = p.z[b * p.zs + ch];
    }
    f32x4 A = {0.f, 0.f, 0.f, 0.f};
    float bias = 0.f, skip = 0.f;
    if (in) {
        A = *reinterpret_cast<const f32x4 *>(p.A + at) * kLog2e;
        if (p.bias != nullptr) bias = p.bias[ch];
        if (p.Dskip != nullptr) skip = p.Dskip[ch];
    }
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        if (slot[k] >= (int64_t)p.max_slots) continue;
        float y = 0.f;
        const float xv = bf16_bits_to_float(x[k]), step = time_step(p, bf16_bits_to_float(dt[k]) + bias);
        const Quad B = quad_of(bw[k][0], bw[k][1]), C = quad_of(cw[k][0], cw[k][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[k][i] = __builtin_fmaf(fast_exp2(step * A[i]), h[k][i], step * xv * B.v[i]);
            y = __builtin_fmaf(C.v[i], h[k][i], y);
        }
        if (in) store_state4<SB>(p.state_out, slot[k] * p.D * p.N + at, h[k]);
        y = lanes_sum<LANES>(y);
        if (!in || n0 != 0) continue;
        y = __builtin_fmaf(skip, xv, y);
        if (p.z != nullptr) {
            const float zv = bf16_bits_to_float(z[k]);
            y *= zv * sigmoid_f(zv);
        }
        p.y[(b0 + k) * (int64_t)p.D + ch] = float_to_bf16_bits(y);
    }
}

template <int LANES, int SEQS>
hipError_t launch_as(const ScanParams &p, hipStream_t s) {
    constexpr int chans = kThreads / LANES;
    const int cblocks = (p.D + chans - 1) / chans;
    const dim3 grid((unsigned)((int64_t)cblocks * ((p.batch + SEQS - 1) / SEQS)));
    if (p.state_bf16)
        scan_step<LANES, SEQS, true><<<grid, kThreads, 0, s>>>(p, cblocks);
    else
        scan_step<LANES, SEQS, false><<<grid, kThreads, 0, s>>>(p, cblocks);
    return hipGetLastError();
}
template <int LANES>
hipError_t launch_lanes(const ScanParams &p, hipStream_t s) {
    return p.batch >= 16 ? launch_as<LANES, 2>(p, s) : launch_as<LANES, 1>(p, s);
}
}  // namespace

hipError_t launch_scan_step(const ScanParams &p, hipStream_t s) {
    const int need = p.N / 4;
    if (need <= 1) return launch_lanes<1>(p, s);
    if (need <= 2) return launch_lanes<2>(p, s);
    if (need <= 4) return launch_lanes<4>(p, s);
    if (need <= 8) return launch_lanes<8>(p, s);
    return launch_lanes<16>(p, s);
}

}  // namespace layer
}  // namespace ssd
