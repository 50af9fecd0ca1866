// Selective scan, one token per sequence, by the recurrence itself.  A thread
// holds 4 consecutive states of a channel, or 8 in bf16, of several sequences,
// so the decays are read once for all of them; the lanes of a channel add their
// shares of C.h.  The states are read once and written once, and that
// is the bound: 512 sequences of 4096 channels and 16 states in fp32, 286 MB, 57 us
// (5.0 TB/s).
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

// S states as they lie in a pool, 16 bytes of them (8 where bf16 ones are no
// multiple of 8).  They are used once, so they pass by the caches (512 sequences
// 62 -> 57 us).
template <bool SB, int S>
struct States {
    static constexpr int kWords = SB ? S / 2 : S;
    typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
    Words w;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        w = __builtin_nontemporal_load(
            reinterpret_cast<const Words *>(static_cast<const uint32_t *>(base) + at * kWords / S));
    }
    __device__ __forceinline__ void widen(float (&h)[S]) const {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if constexpr (SB)
                h[i] = i % 2 ? bf16x2_hi(w[i / 2]) : bf16x2_lo(w[i / 2]);
            else
                h[i] = __uint_as_float(w[i]);
        }
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, const float (&h)[S]) {
        Words v;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (SB)
                v[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
            else
                v[i] = __float_as_uint(h[i]);
        }
        __builtin_nontemporal_store(v, reinterpret_cast<Words *>(static_cast<uint32_t *>(base) + at * kWords / S));
    }
};

template <int LANES, int SEQS, bool SB, int S>
__global__ __launch_bounds__(kThreads) void scan_step(ScanParams p, int cblocks) {
    typedef uint32_t Row __attribute__((ext_vector_type(S / 2), aligned(4)));  // of B and C
    const int cb = blockIdx.x % cblocks, b0 = blockIdx.x / cblocks * SEQS;
    const int ch = cb * (kThreads / LANES) + threadIdx.x / LANES, n0 = threadIdx.x % LANES * S;
    const bool in = ch < p.D && n0 < p.N;
    const int64_t at = (int64_t)ch * p.N + n0;
    const int g = ch / p.Dg;
    States<SB, S> old[SEQS];
    int64_t slot[SEQS];
    Row bw[SEQS], cw[SEQS];
    uint32_t x[SEQS], dt[SEQS], z[SEQS];
    // all that is read, ahead of all that is computed
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const int64_t b = b0 + k;
        slot[k] = b < p.batch ? (int64_t)p.cache_idx[b] : (int64_t)p.max_slots;  // max_slots or more: nothing
        const bool init = b < p.batch && p.has_init != nullptr && p.has_init[b] != 0;
        old[k] = {};
        x[k] = dt[k] = z[k] = 0;
        bw[k] = cw[k] = Row(0);
        if (!in || slot[k] >= (int64_t)p.max_slots) continue;
        if (init) old[k].load(p.state_in, slot[k] * p.D * p.N + at);
        bw[k] = *reinterpret_cast<const Row *>(p.B + b * p.bs + g * p.N + n0);
        cw[k] = *reinterpret_cast<const Row *>(p.C + b * p.cs + g * p.N + n0);
        x[k] = p.x[b * p.xs + ch];
        dt[k] = p.dt[b * p.dts + ch];
        if (p.z != nullptr) z[k] = p.z[b * p.zs + ch];
    }
    float A[S] = {}, bias = 0.f, skip = 0.f;
    if (in) {
#pragma unroll
        for (int i = 0; i < S; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p.A + at + i) * kLog2e;
#pragma unroll
            for (int j = 0; j < 4; ++j) A[i + j] = v[j];
        }
        if (p.bias != nullptr) bias = p.bias[ch];
        if (p.Dskip != nullptr) skip = p.Dskip[ch];
    }
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        if (slot[k] >= (int64_t)p.max_slots) continue;
        float y = 0.f, h[S];
        old[k].widen(h);
        const float xv = bf16_bits_to_float(x[k]), step = time_step(p, bf16_bits_to_float(dt[k]) + bias);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const float B = i % 2 ? bf16x2_hi(bw[k][i / 2]) : bf16x2_lo(bw[k][i / 2]);
            const float C = i % 2 ? bf16x2_hi(cw[k][i / 2]) : bf16x2_lo(cw[k][i / 2]);
            h[i] = __builtin_fmaf(fast_exp2(step * A[i]), h[i], step * xv * B);
            y = __builtin_fmaf(C, h[i], y);
        }
        if (in) States<SB, S>::store(p.state_out, slot[k] * p.D * p.N + at, h);
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

template <int LANES, bool SB, int S>
hipError_t launch_lanes(const ScanParams &p, hipStream_t s) {
    constexpr int chans = kThreads / LANES;
    const int cblocks = (p.D + chans - 1) / chans;
    auto grid = [&](int seqs) { return dim3((unsigned)((int64_t)cblocks * ((p.batch + seqs - 1) / seqs))); };
    if (p.batch >= 16)
        scan_step<LANES, 2, SB, S><<<grid(2), kThreads, 0, s>>>(p, cblocks);
    else
        scan_step<LANES, 1, SB, S><<<grid(1), kThreads, 0, s>>>(p, cblocks);
    return hipGetLastError();
}
template <bool SB, int S>
hipError_t launch_states(const ScanParams &p, hipStream_t s) {
    const int need = p.N / S;
    if (need <= 1) return launch_lanes<1, SB, S>(p, s);
    if (need <= 2) return launch_lanes<2, SB, S>(p, s);
    if (need <= 4) return launch_lanes<4, SB, S>(p, s);
    if (need <= 8) return launch_lanes<8, SB, S>(p, s);
    if constexpr (S == 4) return launch_lanes<16, SB, S>(p, s);
    return hipErrorInvalidValue;  // (no more than 64 states)
}
}  // namespace

// 16 bytes of states a lane where they allow it (512 sequences of bf16 states 50 us with 8 bytes, 35 with 16; of fp32
// states 57 us with 16, 64 with 32)
hipError_t launch_scan_step(const ScanParams &p, hipStream_t s) {
    if (!p.state_bf16) return launch_states<false, 4>(p, s);
    return p.N % 8 == 0 ? launch_states<true, 8>(p, s) : launch_states<true, 4>(p, s);
}

}  // namespace layer
}  // namespace ssd
