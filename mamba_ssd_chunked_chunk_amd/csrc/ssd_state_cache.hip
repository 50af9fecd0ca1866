// Pool states in 8 bits: rows of N elements quantised with one scale each,
// and read back.  A row lies across the lanes that hold 8 elements of it
// each; a thread takes kRows rows so that enough loads are in flight.  Both
// directions are bound by HBM: 4 (or 2) + 1 bytes an element.
#include "ssd_common.hpp"
#include "ssd_linear_attn.hpp"

namespace ssd {
namespace {
constexpr int kThreads = 256;
constexpr int kRows = 4;

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, d, 64);
        v = v > o ? v : o;
    }
    return v;
}

// x / s to the nearest integer, ties to even, decided on the true quotient:
// the product with the rounded reciprocal is within one of it, and the
// remainder x - c s is exact in fp32 (a multiple of half a unit of s's last
// place, below s in size).
__device__ __forceinline__ int nearest_code(float x, float s, float inv) {
    float c = rintf(x * inv);
    const float r = 2.f * __builtin_fmaf(-c, s, x);
    const float a = fabsf(r);
    const bool odd = ((int)c & 1) != 0;
    if (a > s || (a == s && odd)) c += r > 0.f ? 1.f : -1.f;
    return (int)c;
}

// Where block `blk` works: the pair it moves (or none) and its first row.
template <int LANES>
struct Span {
    int64_t pool_row, entry_row;  // of the pair's first row
    int64_t first;
    bool live;
    __device__ Span(const CacheParams &p, int64_t blocks_per_pair) {
        const int64_t i = blockIdx.x / blocks_per_pair;
        const uint32_t a = p.pool_idx[i], b = p.entry_idx[i];
        live = a < p.max_slots && b < p.max_entries;
        pool_row = (int64_t)a * p.rows_per_slot;
        entry_row = (int64_t)b * p.rows_per_slot;
        first = (blockIdx.x - i * blocks_per_pair) * (kThreads / LANES * kRows) + threadIdx.x / LANES;
    }
};

template <int LANES, bool SB, bool E4M3>
__global__ __launch_bounds__(kThreads) void state_quantize(CacheParams p, const void *pool, uint8_t *codes,
                                                           float *scales, int blocks_per_pair) {
    constexpr int RP = kThreads / LANES;
    const Span<LANES> w(p, blocks_per_pair);
    if (!w.live) return;
    const int c = (threadIdx.x % LANES) * 8;
    const bool in = c < p.N;
    float x[kRows][8];
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[n][e] = 0.f;
        const int64_t row = w.first + n * RP;
        if (in && row < p.rows_per_slot) load_state8<SB>(pool, (w.pool_row + row) * p.N + c, x[n]);
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int64_t row = w.first + n * RP;
        uint32_t top = 0;  // magnitudes order as their bits, infinities and NaN last
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = __float_as_uint(x[n][e]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
        top = lanes_max<LANES>(top);
        if (row >= p.rows_per_slot) continue;
        const bool finite = top < 0x7F800000u;
        float s;
        uint32_t lo = 0, hi = 0;
        if constexpr (E4M3) {
            // top = m 2^e: 448 = 1.75 2^8 holds m <= 1.75 with 2^(e-8)
            int k = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
            k = k < 1 ? 1 : k;
            s = top == 0 ? 0.f : __uint_as_float((uint32_t)k << 23);
            if (top != 0 && finite) {
                const float inv = __uint_as_float((uint32_t)(254 - k) << 23);  // exact
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][0] * inv, x[n][1] * inv, 0, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][2] * inv, x[n][3] * inv, lo, true);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][4] * inv, x[n][5] * inv, 0, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][6] * inv, x[n][7] * inv, hi, true);
            }
        } else {
            s = __uint_as_float(top) / 127.f;
            if (s < 1.17549435e-38f) s = 0.f;
            if (s > 0.f && finite) {
                const float inv = 1.f / s;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo |= (uint32_t)(nearest_code(x[n][e], s, inv) & 0xFF) << (8 * e);
                    hi |= (uint32_t)(nearest_code(x[n][4 + e], s, inv) & 0xFF) << (8 * e);
                }
            }
        }
        if (!finite) s = __uint_as_float(0x7FC00000u);
        const int64_t at = w.entry_row + row;
        if (in) *reinterpret_cast<u32x2 *>(codes + at * p.N + c) = u32x2{lo, hi};
        if (c == 0) scales[at] = s;
    }
}

template <int LANES, bool SB, bool E4M3>
__global__ __launch_bounds__(kThreads) void state_dequantize(CacheParams p, void *pool, const uint8_t *codes,
                                                             const float *scales, int blocks_per_pair) {
    constexpr int RP = kThreads / LANES;
    const Span<LANES> w(p, blocks_per_pair);
    const int c = (threadIdx.x % LANES) * 8;
    if (!w.live || c >= p.N) return;
    u32x2 q[kRows];
    float s[kRows];
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int64_t row = w.first + n * RP;
        if (row >= p.rows_per_slot) continue;
        q[n] = *reinterpret_cast<const u32x2 *>(codes + (w.entry_row + row) * p.N + c);
        s[n] = scales[w.entry_row + row];
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int64_t row = w.first + n * RP;
        if (row >= p.rows_per_slot) continue;
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = q[n][i];
            if constexpr (E4M3) {
                const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(v, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
                x[4 * i] = a[0] * s[n];
                x[4 * i + 1] = a[1] * s[n];
                x[4 * i + 2] = b[0] * s[n];
                x[4 * i + 3] = b[1] * s[n];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * i + e] = (float)(int8_t)(v >> (8 * e)) * s[n];
            }
        }
        store_state8<SB>(pool, (w.pool_row + row) * p.N + c, x);
    }
}

template <typename F>
hipError_t by_lanes(const CacheParams &p, bool bf16, bool e4m3, F f) {
    const int lanes = p.N <= 64 ? 8 : p.N <= 128 ? 16 : 32;
    const int64_t rows = kThreads / lanes * kRows;
    const int64_t bpp = (p.rows_per_slot + rows - 1) / rows;
    const dim3 grid((unsigned)(bpp * p.count));
    auto pick = [&](auto l) {
        constexpr int L = decltype(l)::value;
        if (bf16)
            e4m3 ? f(l, std::true_type{}, std::true_type{}, grid, (int)bpp)
                 : f(l, std::true_type{}, std::false_type{}, grid, (int)bpp);
        else
            e4m3 ? f(l, std::false_type{}, std::true_type{}, grid, (int)bpp)
                 : f(l, std::false_type{}, std::false_type{}, grid, (int)bpp);
        (void)L;
    };
    if (lanes == 8)
        pick(std::integral_constant<int, 8>{});
    else if (lanes == 16)
        pick(std::integral_constant<int, 16>{});
    else
        pick(std::integral_constant<int, 32>{});
    return hipGetLastError();
}
}  // namespace

hipError_t launch_state_quantize(const CacheParams &c, const void *pool, bool bf16, bool e4m3, void *codes,
                                 float *scales, hipStream_t s) {
    return by_lanes(c, bf16, e4m3, [&](auto l, auto sb, auto e4, dim3 grid, int bpp) {
        state_quantize<decltype(l)::value, decltype(sb)::value, decltype(e4)::value>
            <<<grid, kThreads, 0, s>>>(c, pool, static_cast<uint8_t *>(codes), scales, bpp);
    });
}
hipError_t launch_state_dequantize(const CacheParams &c, void *pool, bool bf16, bool e4m3, const void *codes,
                                   const float *scales, hipStream_t s) {
    return by_lanes(c, bf16, e4m3, [&](auto l, auto sb, auto e4, dim3 grid, int bpp) {
        state_dequantize<decltype(l)::value, decltype(sb)::value, decltype(e4)::value>
            <<<grid, kThreads, 0, s>>>(c, pool, static_cast<const uint8_t *>(codes), scales, bpp);
    });
}
}  // namespace ssd
