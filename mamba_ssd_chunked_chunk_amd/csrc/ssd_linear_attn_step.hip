// Linear attention, one token per sequence, by the recurrence itself:
//     S = lambda S + v k^T,   o = scale S q
// Each thread holds 8 consecutive key channels of kRows rows of the state
// (16-byte loads and stores; the lanes of a row cover it contiguously), so
// the state is read once and written once.  That is the bound: 8 K V bytes a
// head in fp32 against 4 K V flop (512 tokens of 128 heads of 64 x 128: 845 us,
// 5.1 TB/s, as fast as a copy).  A block takes at most 64 rows of a 128-channel
// state, so that a single token of 16 heads still spreads over 32 of them (4.4
// us).
#include "ssd_linear_attn.hpp"

namespace ssd {
namespace la {
namespace {
constexpr int kThreads = 256;
constexpr int kRows = 4;  // state rows of a thread

// sum over each aligned group of LANES (8, 16 or 32) lanes; every lane receives it
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    v = dpp_add_all<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_add_all<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_add_all<0x141>(v);  // row_half_mirror
    if constexpr (LANES >= 16) v = dpp_add_all<0x140>(v);  // row_mirror
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16, 64);
    return v;
}

template <int LANES, bool SB>
__global__ __launch_bounds__(kThreads) void la_step(StepParams p) {
    constexpr int RP = kThreads / LANES;  // rows side by side
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int64_t slot = p.cache_idx[b];
    if (slot >= p.max_slots) return;  // padding
    const int r0 = blockIdx.y * (RP * kRows) + threadIdx.x / LANES;
    const int c = (threadIdx.x % LANES) * 8;
    const bool in = c < p.K;
    const bool init = p.has_init != nullptr && p.has_init[b] != 0;
    const int64_t at = (slot * p.H + h) * p.K * p.V + (int64_t)r0 * p.K + c;

    float S[kRows][8], v[kRows], q[8] = {}, k[8] = {};
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const bool row = r0 + n * RP < p.V;
#pragma unroll
        for (int e = 0; e < 8; ++e) S[n][e] = 0.f;
        if (init && in && row) load_state8<SB>(p.pool, at + (int64_t)n * RP * p.K, S[n]);
        v[n] = row ? bf16_bits_to_float(p.v[b * p.vs + (int64_t)h * p.V + r0 + n * RP]) : 0.f;
    }
    if (in) {
        load_state8<true>(p.q, b * p.qs + (int64_t)(h / p.div) * p.K + c, q);
        load_state8<true>(p.k, b * p.ks + (int64_t)(h / p.div) * p.K + c, k);
    }
    const float decay = init ? expf(p.log_decay[h]) : 0.f;  // no state, nothing to decay: lambda may be infinite
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const bool row = r0 + n * RP < p.V;
        float o = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            S[n][e] = S[n][e] * decay + v[n] * k[e];
            o += S[n][e] * q[e];
        }
        o = lanes_sum<LANES>(o) * p.scale;
        if (!row) continue;
        if (in) store_state8<SB>(p.pool, at + (int64_t)n * RP * p.K, S[n]);
        if (threadIdx.x % LANES == 0)
            p.o[((int64_t)b * p.H + h) * p.V + r0 + n * RP] = float_to_bf16_bits(o);
    }
}

template <int LANES>
hipError_t launch_lanes(const StepParams &p, hipStream_t s) {
    constexpr int rows = kThreads / LANES * kRows;
    const dim3 grid((unsigned)((int64_t)p.batch * p.H), (unsigned)((p.V + rows - 1) / rows));
    if (p.state_bf16)
        la_step<LANES, true><<<grid, kThreads, 0, s>>>(p);
    else
        la_step<LANES, false><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_step(const StepParams &p, hipStream_t s) {
    if (p.K <= 64) return launch_lanes<8>(p, s);
    if (p.K <= 128) return launch_lanes<16>(p, s);
    return launch_lanes<32>(p, s);
}

}  // namespace la
}  // namespace ssd
