// Root-mean-square norm with the residual's addition, its 8-bit outputs and
// its backward pass.  A row lies in the registers of 64 to 1024 threads, 8
// consecutive elements each and up to 4 times, so it is read once; the sums over
// it are fp32.  Memory bounds both directions: 16384 rows of 4096 with an fp32
// residual, 806 MB, 150 us (5.4 TB/s), and to 8 bits, 738 MB, 136 us either way; the
// backward pass of 5001 rows of 2560 in bf16, 102 MB, 22 us (4.7 TB/s), and 6.5 us
// for the sum over the blocks' shares.  Without a residual 16384 rows of 4096 to e4m3,
// 201 MB, take 41 us, and to int8, whose codes are decided on the remainder of a
// division (32 vector instructions an element for 18), 53.
#include <algorithm>

#include "ssd.h"
#include "ssd_layer.hpp"
#include "ssd_state_cache.hpp"

namespace ssd {
namespace layer {
namespace {

// ROWS rows of TPR threads each in a block
template <int TPR>
struct Team {
    static constexpr int kRows = TPR == 64 ? 4 : 1;
    static constexpr int kThreads = TPR * kRows;
    static constexpr int kWaves = TPR / 64;
};

// sums over the threads of a row, in all of them; `buf` holds a float a wave
// (for each of the sums), and a barrier has to pass before it is used again
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *buf) {
    v.x = wave_sum(v.x);
    v.y = wave_sum(v.y);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x / 64] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) {
            v.x += buf[w].x;
            v.y += buf[w].y;
        }
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *buf) {
    v = wave_max_u32(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x / 64] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) v = v > buf[w] ? v : buf[w];
    }
    return v;
}

__device__ __forceinline__ void load8(const void *base, int64_t at, bool bf16, float (&o)[8]) {
    if (bf16)
        load_state8<true>(base, at, o);
    else
        load_state8<false>(base, at, o);
}

template <int TPR, int VPT>
__global__ __launch_bounds__(Team<TPR>::kThreads) void rms_norm(NormParams p) {
    __shared__ float2 sums[16];
    __shared__ uint32_t tops[16];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * Team<TPR>::kRows + threadIdx.x / TPR;
    const bool live = row < p.rows;
    float r[VPT][8];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * TPR) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] = 0.f;
        if (live && c < p.width) load_state8<true>(p.x, row * p.xs + c, r[v]);
    }
    if (p.res != nullptr) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * TPR) * 8;
            if (!live || c >= p.width) continue;
            const int64_t at = row * p.width + c;
            float a[8];
            load8(p.res, at, p.res_bf16, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] += a[e];
            if (p.res_bf16) {
                // the stream is held in bf16: what is normed is what is held
                const u32x4 w = narrow8(r[v]);
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.res_out) + at) = w;
                widen8(w, r[v]);
            } else {
                store_state8<false>(p.res_out, at, r[v]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(r[v][e], r[v][e], sum);
    sum = row_sum<TPR>(make_float2(sum, 0.f), sums).x;
    const float s = 1.f / sqrtf(sum / (float)p.width + p.eps);
    uint32_t top = 0;  // magnitudes order as their bits, infinities and NaN last
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * TPR) * 8;
        if (c >= p.width) continue;
        float w[8];
        load_state8<false>(p.weight, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[v][e] *= s * w[e];
            const uint32_t m = __float_as_uint(r[v][e]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
    }
    if (p.out == SSD_OUT_BF16) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * TPR) * 8;
            if (live && c < p.width)
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.y) + row * p.width + c) = narrow8(r[v]);
        }
        return;
    }
    top = row_max<TPR>(top, tops);
    const bool finite = top < 0x7F800000u;
    float scale, inv;
    if (p.out == SSD_CODE_E4M3) {
        const int k = e4m3_scale_exponent(top);
        scale = top == 0 ? 0.f : __uint_as_float((uint32_t)k << 23);
        inv = __uint_as_float((uint32_t)(254 - k) << 23);  // exact
    } else {
        scale = code_scale(__uint_as_float(top));
        if (scale < 1.17549435e-38f) scale = 0.f;
        inv = __builtin_amdgcn_rcpf(scale);
    }
    const bool codes = scale > 0.f && finite;
    if (!finite) scale = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * TPR) * 8;
        if (!live || c >= p.width) continue;
        uint32_t q[2] = {};
        if (codes && p.out == SSD_CODE_E4M3) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(r[v][4 * i] * inv, r[v][4 * i + 1] * inv, 0, false);
                q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(r[v][4 * i + 2] * inv, r[v][4 * i + 3] * inv, q[i], true);
            }
        } else if (codes) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e / 4] |= (uint32_t)(nearest_code(r[v][e], scale, inv) & 0xFF) << (8 * (e % 4));
        }
        *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(p.y) + row * p.width + c) = u32x2{q[0], q[1]};
    }
    if (live && t == 0) p.scales[row] = scale;
}

// Gradient: with u = w dy, d = s u - s^3 r mean(u r) + d_r, formed as
// s (u - (s r) (s mean(u r))), whose factors stay near u and 1 (s^3 alone leaves the
// range of fp32 where r is above 2^43 or below 2^-43).  Each row's team walks over
// rows and keeps its share of sum s r dy in registers.
template <int TPR, int VPT>
__global__ __launch_bounds__(Team<TPR>::kThreads) void rms_norm_grad(NormGradParams p) {
    __shared__ float2 sums[2][16];
    const int t = threadIdx.x % TPR;
    const int team = blockIdx.x * Team<TPR>::kRows + threadIdx.x / TPR;
    const int teams = gridDim.x * Team<TPR>::kRows;
    // rows of 4 vectors a thread leave no registers for the weights, which they read again from L2 (3000 rows of 24576:
    // 251 -> 187 us)
    constexpr bool kKeep = VPT < 4 || TPR < 1024;
    float w[VPT][8], dw[VPT][8];
    auto weight = [&](int v) {
        const int c = (t + v * TPR) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[v][e] = 0.f;
        if (c < p.width) load_state8<false>(p.weight, c, w[v]);
    };
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
        if (kKeep) weight(v);
    }
    const float share = 1.f / (float)p.width;
    // every team of a block takes as many turns (they share barriers)
    const int64_t turns = (p.rows + teams - 1) / teams;
    for (int64_t n = 0; n < turns; ++n) {
        const int64_t row = n * teams + team;
        const bool live = row < p.rows;
        float r[VPT][8], u[VPT][8];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * TPR) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = u[v][e] = 0.f;
            if (live && c < p.width) {
                load8(p.r, row * p.width + c, p.res_bf16, r[v]);
                load_state8<true>(p.dy, row * p.width + c, u[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!kKeep) weight(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum.x = __builtin_fmaf(r[v][e], r[v][e], sum.x);
                sum.y = __builtin_fmaf(u[v][e] * w[v][e], r[v][e], sum.y);
            }
        }
        sum = row_sum<TPR>(sum, sums[n & 1]);
        const float s = 1.f / sqrtf(sum.x * share + p.eps);
        const float k = s * (sum.y * share);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * TPR) * 8;
            if (!live || c >= p.width) continue;
            const int64_t at = row * p.width + c;
            float d[8] = {};
            if (p.d_r != nullptr) load8(p.d_r, at, p.res_bf16, d);
            if (!kKeep) weight(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = s * r[v][e];
                dw[v][e] = __builtin_fmaf(n, u[v][e], dw[v][e]);
                d[e] = __builtin_fmaf(s, __builtin_fmaf(-k, n, u[v][e] * w[v][e]), d[e]);
            }
            *reinterpret_cast<u32x4 *>(p.dx + at) = narrow8(d);
            if (p.d_res != nullptr) {
                if (p.res_bf16)
                    store_state8<true>(p.d_res, at, d);
                else
                    store_state8<false>(p.d_res, at, d);
            }
        }
    }
    // the teams of a block are one part, added by the first (5001 rows of 512: 24.6 -> 14.5 us with the sums behind)
    constexpr int kOthers = Team<TPR>::kRows - 1;
    if constexpr (kOthers > 0) {
        __shared__ float others[kOthers][VPT * 8][TPR];
        const int i = threadIdx.x / TPR - 1;
        if (i >= 0)
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) others[i][v * 8 + e][t] = dw[v][e];
        __syncthreads();
        if (i >= 0) return;
#pragma unroll
        for (int k = 0; k < kOthers; ++k)
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[v][e] += others[k][v * 8 + e][t];
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * TPR) * 8;
        if (c < p.width) store_state8<false>(p.part, (int64_t)blockIdx.x * p.width + c, dw[v]);
    }
}

__global__ __launch_bounds__(kSumThreads) void sum_parts(Sums sums) {
    add_parts<32>(sums, blockIdx.x);
}

template <int TPR, int VPT>
hipError_t norm_as(const NormParams &p, hipStream_t s) {
    constexpr int rows = Team<TPR>::kRows;
    rms_norm<TPR, VPT><<<dim3((unsigned)((p.rows + rows - 1) / rows)), Team<TPR>::kThreads, 0, s>>>(p);
    return hipGetLastError();
}
template <int TPR, int VPT>
hipError_t norm_grad_as(const NormGradParams &p, hipStream_t s) {
    rms_norm_grad<TPR, VPT><<<dim3((unsigned)p.parts), Team<TPR>::kThreads, 0, s>>>(p);
    return hipGetLastError();
}

constexpr int kWide = 2048;  // up to this width a row has 64 threads, above it 256, 512 or 1024
}  // namespace

int64_t norm_threads(int64_t rows, int width) {
    if (rows > UINT32_MAX) return rows;
    return rows * (width <= kWide ? 64 : width <= 4096 ? 256 : width <= 8192 ? 512 : 1024) + 255;
}

// Rows of more than 8192 elements in 1024 threads, 2 vectors each (12000 rows of 16384: 342 us in 256 threads, 297 in
// 512, 268 in 1024), of more than 4096 in 512 (20000 of 5120: 153 us in 256, 147 in 512, 159 in 1024).
hipError_t launch_norm(const NormParams &p, hipStream_t s) {
    if (p.width <= 512) return norm_as<64, 1>(p, s);
    if (p.width <= 1024) return norm_as<64, 2>(p, s);
    if (p.width <= kWide) return norm_as<64, 4>(p, s);
    if (p.width <= 4096) return norm_as<256, 2>(p, s);
    if (p.width <= 8192) return norm_as<512, 2>(p, s);
    if (p.width <= 16384) return norm_as<1024, 2>(p, s);
    return norm_as<1024, 4>(p, s);
}

int norm_grad_parts(int64_t rows, int width) {
    const int per_block = width <= 1024 ? 4 : 1;
    const int64_t most = width <= 4096 ? 1024 : 256;  // blocks that are resident (of 1024 threads one a unit)
    return (int)std::clamp<int64_t>((rows + per_block - 1) / per_block, 1, most);
}

// (12000 rows of 8192: 226 us in 1024 blocks of 256 threads, 166 in 256 of 1024)
hipError_t launch_norm_grad(const NormGradParams &p, hipStream_t s) {
    hipError_t e;
    if (p.width <= 512) e = norm_grad_as<64, 1>(p, s);
    else if (p.width <= 1024) e = norm_grad_as<64, 2>(p, s);
    else if (p.width <= 2048) e = norm_grad_as<256, 1>(p, s);
    else if (p.width <= 4096) e = norm_grad_as<256, 2>(p, s);
    else if (p.width <= 8192) e = norm_grad_as<1024, 1>(p, s);
    else if (p.width <= 16384) e = norm_grad_as<1024, 2>(p, s);
    else e = norm_grad_as<1024, 4>(p, s);
    if (e != hipSuccess) return e;
    return launch_sums(Sums{{Sum{p.part, p.parts, p.width, p.width, p.dweight}}}, s);
}

hipError_t launch_sums(const Sums &sums, hipStream_t s) {
    sum_parts<<<dim3((unsigned)sum_blocks<32>(sums)), kSumThreads, 0, s>>>(sums);
    return hipGetLastError();
}

}  // namespace layer
}  // namespace ssd
