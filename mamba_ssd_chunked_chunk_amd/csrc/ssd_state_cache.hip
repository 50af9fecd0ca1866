// Pool states in 8 bits: rows of N elements quantised with one scale each,
// and read back.  A row lies across the lanes that hold 16 bytes of its state
// each (4 elements in fp32, 8 in bf16), so every state access of a wavefront is
// one run of memory; a thread takes several rows so that enough of them are in
// flight.  Both directions are bound by memory: 4 (or 2) + 1 bytes an element.
// 268 MB of fp32 state to int8: 87 us (338 MB counted, 3.9 TB/s); back: 57 us (338
// MB, 5.9 TB/s: four bytes of five are written, and the codes, 67 MB and just
// written, fit the 256 MB cache, so a copy's 5.1 is no bound here); 1.07 GB from
// e4m3: 256 us (1.35 GB, 5.3 TB/s; medians).  Lanes of 8 elements of
// fp32 and 4 rows a thread: 88 us, and 77 back; 16 rows a thread to int8: 103.
#include <algorithm>

#include "ssd_common.hpp"
#include "ssd_linear_attn.hpp"

namespace ssd {
namespace {
constexpr int kThreads = 256;
constexpr int kRowsIn = 4, kRowsOut = 8;  // of a thread, quantising and reading back

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}
// largest over each aligned group of LANES lanes; every lane receives it
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_max<0x141>(v);  // row_half_mirror: groups of 8
    if constexpr (LANES >= 16) v = dpp_max<0x140>(v);  // row_mirror: rows of 16
#pragma unroll
    for (int d = 16; d < LANES; d <<= 1) {
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

// top / 127, correctly rounded: by Markstein's theorem one step from a product
// with the rounded reciprocal gives it, away from the subnormal range.
__device__ __forceinline__ float code_scale(float top) {
    constexpr float inv = 1.f / 127.f;
    if (top < 0x1p-100f) return top / 127.f;
    const float q = top * inv;
    return __builtin_fmaf(__builtin_fmaf(-127.f, q, top), inv, q);
}

// Where a block works: the pair it moves (or none) and its first row.
template <int LANES, int ROWS>
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
        first = (blockIdx.x - i * blocks_per_pair) * (kThreads / LANES * ROWS) + threadIdx.x / LANES;
    }
};

// E consecutive elements of a state (16 bytes) as floats, and back
template <bool SB, int E>
__device__ __forceinline__ void load_elements(const void *base, int64_t idx, float (&f)[E]) {
    if constexpr (SB) {
        load_state8<true>(base, idx, f);
    } else {
        const f32x4 v = load_state4<false>(base, idx);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = v[e];
    }
}
template <bool SB, int E>
__device__ __forceinline__ void store_elements(void *base, int64_t idx, const float (&f)[E]) {
    if constexpr (SB)
        store_state8<true>(base, idx, f);
    else
        store_state4<false>(base, idx, f32x4{f[0], f[1], f[2], f[3]});
}

template <int LANES, bool SB, bool E4M3>
__global__ __launch_bounds__(kThreads) void state_quantize(CacheParams p, const void *pool, uint8_t *codes,
                                                           float *scales, int blocks_per_pair) {
    constexpr int RP = kThreads / LANES, E = SB ? 8 : 4;
    const Span<LANES, kRowsIn> w(p, blocks_per_pair);
    if (!w.live) return;
    const int c = (threadIdx.x % LANES) * E;
    const bool in = c < p.N;
    float x[kRowsIn][E];
#pragma unroll
    for (int n = 0; n < kRowsIn; ++n) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[n][e] = 0.f;
        const int64_t row = w.first + n * RP;
        if (in && row < p.rows_per_slot) load_elements<SB, E>(pool, (w.pool_row + row) * p.N + c, x[n]);
    }
#pragma unroll
    for (int n = 0; n < kRowsIn; ++n) {
        const int64_t row = w.first + n * RP;
        uint32_t top = 0;  // magnitudes order as their bits, infinities and NaN last
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t m = __float_as_uint(x[n][e]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
        top = lanes_max<LANES>(top);
        if (row >= p.rows_per_slot) continue;
        const bool finite = top < 0x7F800000u;
        float s;
        uint32_t q[E / 4] = {};
        if constexpr (E4M3) {
            // top = m 2^e: 448 = 1.75 2^8 holds m <= 1.75 with 2^(e-8)
            int k = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
            k = k < 1 ? 1 : k;
            s = top == 0 ? 0.f : __uint_as_float((uint32_t)k << 23);
            if (top != 0 && finite) {
                const float inv = __uint_as_float((uint32_t)(254 - k) << 23);  // exact
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][4 * i] * inv, x[n][4 * i + 1] * inv, 0, false);
                    q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[n][4 * i + 2] * inv, x[n][4 * i + 3] * inv, q[i], true);
                }
            }
        } else {
            s = code_scale(__uint_as_float(top));
            if (s < 1.17549435e-38f) s = 0.f;
            if (s > 0.f && finite) {
                // adding 1.5 2^23 rounds to a whole number, whose low byte is the code
                const float inv = __builtin_amdgcn_rcpf(s);
                float far = 0.f;  // the largest remainder
                uint32_t y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float m = __builtin_fmaf(x[n][e], inv, 0x1.8p23f);
                    y[e] = __float_as_uint(m);
                    far = fmaxf(far, fabsf(__builtin_fmaf(0x1.8p23f - m, s, x[n][e])));
                }
                if (2.f * far >= s) {  // a quotient at (or misjudged by the reciprocal near) a half: seldom
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = (uint32_t)nearest_code(x[n][e], s, inv);
                }
#pragma unroll
                for (int i = 0; i < E / 4; ++i)
                    q[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(y[4 * i + 3], y[4 * i + 2], 0x0C0C0400),
                                                 __builtin_amdgcn_perm(y[4 * i + 1], y[4 * i], 0x0C0C0400), 0x05040100);
            }
        }
        if (!finite) s = __uint_as_float(0x7FC00000u);
        const int64_t at = w.entry_row + row;
        if (in) {
            if constexpr (SB)
                *reinterpret_cast<u32x2 *>(codes + at * p.N + c) = u32x2{q[0], q[1]};
            else
                *reinterpret_cast<uint32_t *>(codes + at * p.N + c) = q[0];
        }
        if (c == 0) scales[at] = s;
    }
}

template <int LANES, bool SB, bool E4M3>
__global__ __launch_bounds__(kThreads) void state_dequantize(CacheParams p, void *pool, const uint8_t *codes,
                                                             const float *scales, int blocks_per_pair) {
    constexpr int RP = kThreads / LANES, E = SB ? 8 : 4;
    const Span<LANES, kRowsOut> w(p, blocks_per_pair);
    const int c = (threadIdx.x % LANES) * E;
    if (!w.live || c >= p.N) return;
    uint32_t q[kRowsOut][E / 4];
    float s[kRowsOut];
#pragma unroll
    for (int n = 0; n < kRowsOut; ++n) {
        const int64_t row = w.first + n * RP;
        if (row >= p.rows_per_slot) continue;
        const uint32_t *at = reinterpret_cast<const uint32_t *>(codes + (w.entry_row + row) * p.N + c);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) q[n][i] = at[i];
        s[n] = scales[w.entry_row + row];
    }
#pragma unroll
    for (int n = 0; n < kRowsOut; ++n) {
        const int64_t row = w.first + n * RP;
        if (row >= p.rows_per_slot) continue;
        float x[E];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
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
        store_elements<SB, E>(pool, (w.pool_row + row) * p.N + c, x);
    }
}

int lanes_of(const CacheParams &p, bool bf16) {
    const int need = p.N / (bf16 ? 8 : 4);
    return need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : 64;
}
int64_t blocks_per_pair(const CacheParams &p, int lanes, int thread_rows) {
    const int64_t rows = kThreads / lanes * thread_rows;
    return (p.rows_per_slot + rows - 1) / rows;
}

template <typename F>
hipError_t by_lanes(const CacheParams &p, int thread_rows, bool bf16, bool e4m3, F f) {
    const int lanes = lanes_of(p, bf16);
    const int64_t bpp = blocks_per_pair(p, lanes, thread_rows);
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
    else if (lanes == 32)
        pick(std::integral_constant<int, 32>{});
    else
        pick(std::integral_constant<int, 64>{});
    return hipGetLastError();
}
}  // namespace

int64_t state_cache_threads(const CacheParams &c, bool bf16) {
    return blocks_per_pair(c, lanes_of(c, bf16), std::min(kRowsIn, kRowsOut)) * c.count * kThreads;
}

hipError_t launch_state_quantize(const CacheParams &c, const void *pool, bool bf16, bool e4m3, void *codes,
                                 float *scales, hipStream_t s) {
    return by_lanes(c, kRowsIn, bf16, e4m3, [&](auto l, auto sb, auto e4, dim3 grid, int bpp) {
        state_quantize<decltype(l)::value, decltype(sb)::value, decltype(e4)::value>
            <<<grid, kThreads, 0, s>>>(c, pool, static_cast<uint8_t *>(codes), scales, bpp);
    });
}
hipError_t launch_state_dequantize(const CacheParams &c, void *pool, bool bf16, bool e4m3, const void *codes,
                                   const float *scales, hipStream_t s) {
    return by_lanes(c, kRowsOut, bf16, e4m3, [&](auto l, auto sb, auto e4, dim3 grid, int bpp) {
        state_dequantize<decltype(l)::value, decltype(sb)::value, decltype(e4)::value>
            <<<grid, kThreads, 0, s>>>(c, pool, static_cast<const uint8_t *>(codes), scales, bpp);
    });
}
}  // namespace ssd
