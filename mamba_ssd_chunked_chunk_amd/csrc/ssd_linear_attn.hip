// Linear attention with a fixed decay per head: the chunked form, forward
// and (as three recurrences with exchanged roles) backward.
//
// A workgroup walks one sequence for one head and 32 * NW value channels, in
// chunks of 64 tokens.  With i, j the places in a chunk, S the state that
// enters it and lambda the head's decay,
//     out_i = lambda^(i+1) S q_i + sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j
//     S    <- lambda^len S + sum_j lambda^(len-1-j) v_j k_j^T
// Each wavefront owns 32 value channels and keeps S of them (32 x kd, fp32)
// in registers for the whole walk, so the state never moves; the wavefronts
// share only the chunk's q, k, v rows and its 64 x 64 matrix of weighted
// scores, in LDS.  Every product is computed transposed (channels x tokens):
// a lane then holds one token and 8 consecutive channels, so its decay is a
// scalar and its result is written 16 bytes at a time, and the state
// registers are, as they are, the operand of the next product.
//
// Operands that run along tokens (v and k of the state update) come from LDS
// with the transposing read, whose lanes take columns in groups of four; the
// groups are ordered so that the accumulator's 8 registers of a lane are 8
// consecutive channels (channel() below).
//
// Rounding: scores and the state are rounded to bf16 once as operands of the
// output, which is bf16 itself.  The weighted v of the state update is split
// into three bf16 parts that carry its 24 bits, so states are those of fp32
// sums.
#include "ssd_linear_attn.hpp"

namespace ssd {
namespace la {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;

__device__ __forceinline__ f32x16 mfma32_bf16(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Channel (or token) that operand lane l % 32 stands for, so that accumulator
// register e of lane half hh belongs to channel 16 (e / 8) + 8 hh + e % 8:
// bits 2 and 3 exchanged.
__device__ __forceinline__ int channel(int l) { return (l & 19) | ((l & 4) << 1) | ((l & 8) >> 1); }

// LDS place (in 16-byte units) of unit c of row r, rows of U units: the units
// of a row are permuted so that both a column of 16-byte reads down
// consecutive rows and the transposing reads (4 rows x 4 units) touch every
// bank once.
template <int U>
__device__ __forceinline__ int place(int r, int c) {
    if constexpr (U == 8)
        return r * U + (c ^ ((((r >> 1) & 1) << 2) | ((r >> 2) & 3)));
    else
        return r * U + (c ^ (((r & 3) << 2) | ((r >> 2) & 3)));
}

template <int U>
__device__ __forceinline__ bf16x8 row_read(const uint16_t *s, int r, int c) {
    return *reinterpret_cast<const bf16x8 *>(s + place<U>(r, c) * 8);
}

// 8 tokens (t0 + 8 (lane / 32) ..) of the column c0 + channel(lane % 32)
template <int U>
__device__ __forceinline__ bf16x8 column_read(const uint16_t *s, int t0, int c0, int lane) {
    const int x = lane & 15;
    const int r = t0 + 8 * (lane >> 5) + (x >> 2);
    const int col = c0 + (lane & 16) + 4 * (((x & 1) << 1) | ((x >> 1) & 1));
    const int c = col >> 3, half = col & 4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + place<U>(r, c) * 8 + half));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + place<U>(r + 4, c) * 8 + half));
    const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ bf16x8 pack8(const float (&f)[8]) {
    const u32x4 w = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7])};
    return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void unpack8(const bf16x8 &b, float (&f)[8]) {
    const u32x4 w = __builtin_bit_cast(u32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16x2_lo(w[i]);
        f[2 * i + 1] = bf16x2_hi(w[i]);
    }
}

// 8 state elements (v channel i, k channels j .. j+7) at base
template <bool SB>
__device__ __forceinline__ void read_state(const void *base, int64_t at, int64_t sk, float (&f)[8]) {
    if (sk == 1) {
        load_state8<SB>(base, at, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (SB)
                f[e] = bf16_bits_to_float(static_cast<const uint16_t *>(base)[at + e * sk]);
            else
                f[e] = static_cast<const float *>(base)[at + e * sk];
        }
    }
}
template <bool SB>
__device__ __forceinline__ void write_state(void *base, int64_t at, int64_t sk, const float (&f)[8]) {
    if (sk == 1) {
        store_state8<SB>(base, at, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (SB)
                static_cast<uint16_t *>(base)[at + e * sk] = float_to_bf16_bits(f[e]);
            else
                static_cast<float *>(base)[at + e * sk] = f[e];
        }
    }
}

// KD: channels of k and q the kernel holds (kd rounded up; the rest is zero)
template <int KD, int NW, bool SB>
__global__ __launch_bounds__(64 * NW) void la_walk(Params p) {
    constexpr int NTH = 64 * NW;
    constexpr int UK = KD / 8;       // 16-byte units of a q or k row
    constexpr int VT = 32 * NW;      // value channels of the workgroup
    constexpr int UV = VT / 8;
    constexpr int NT = KD / 32;      // 32 x 32 tiles of a wavefront's state
    constexpr int LK = kTok * UK / NTH, LV = kTok * UV / NTH;  // 16-byte loads of a thread
    __shared__ __attribute__((aligned(16))) uint16_t s_q[kTok * KD];
    __shared__ __attribute__((aligned(16))) uint16_t s_k[kTok * KD];
    __shared__ __attribute__((aligned(16))) uint16_t s_v[kTok * VT];
    __shared__ __attribute__((aligned(16))) uint16_t s_p[kTok * kTok];

    const Op &op = p.op[blockIdx.z];
    const int v0 = blockIdx.y * VT;
    if (v0 >= op.vd) return;
    const int h = blockIdx.x % p.H, b = blockIdx.x / p.H;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hh = lane >> 5, l32 = lane & 31;

    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[b] : (int64_t)b;
    if (slot >= p.max_slots) return;  // padding
    const int64_t begin = min(max((int64_t)p.qsl[b], (int64_t)0), p.T);
    const int64_t end = max(min((int64_t)p.qsl[b + 1], p.T), begin);
    const bool rev = op.reverse != 0;
    // log2 of the decay; -infinity as a finite number, so that times 0 it is 0
    const float ld = p.log_decay[h] * kLog2e;
    const float l2 = ld < -1e30f ? -1e30f : ld;
    const float shift = rev ? 1.f : 0.f;

    // ---- the state: registers e of tile t hold (v channel sv_i, k channel
    // 32 t + 16 (e / 8) + 8 hh + e % 8)
    const int vch = v0 + 32 * wave + channel(l32);
    const bool vch_in = vch < op.vd;
    const int64_t state_at = (slot * p.H + h) * p.state_size + (int64_t)vch * op.sv;
    f32x16 S[NT];
    const bool init = op.state_in != nullptr && (p.init_all != 0 || (p.has_init != nullptr && p.has_init[b] != 0));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int kc = 32 * t + 16 * x + 8 * hh;
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (init && vch_in && kc < op.kd) read_state<SB>(op.state_in, state_at + kc * op.sk, op.sk, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) S[t][8 * x + e] = f[e];
        }

    const uint16_t *gq = op.q.p + (int64_t)(h / op.q.div) * op.kd;
    const uint16_t *gk = op.k.p + (int64_t)(h / op.k.div) * op.kd;
    const uint16_t *gv = op.v.p + (int64_t)(h / op.v.div) * op.vd + v0;

#pragma unroll 1
    for (int64_t c0 = 0; c0 < end - begin; c0 += kTok) {
        const int len = (int)min((int64_t)kTok, end - begin - c0);
        // place r of the chunk is token first + r * dir
        const int64_t first = rev ? end - 1 - c0 : begin + c0;
        const int dir = rev ? -1 : 1;
        __syncthreads();  // the previous chunk's rows are no longer read
#pragma unroll
        for (int n = 0; n < LK; ++n) {
            const int r = (tid + n * NTH) / UK, c = (tid + n * NTH) % UK;
            u32x4 wq = {0, 0, 0, 0}, wk = {0, 0, 0, 0};
            if (r < len && 8 * c < op.kd) {
                const int64_t t = first + r * dir;
                wq = *reinterpret_cast<const u32x4 *>(gq + t * op.q.stride + 8 * c);
                wk = *reinterpret_cast<const u32x4 *>(gk + t * op.k.stride + 8 * c);
            }
            *reinterpret_cast<u32x4 *>(s_q + place<UK>(r, c) * 8) = wq;
            *reinterpret_cast<u32x4 *>(s_k + place<UK>(r, c) * 8) = wk;
        }
#pragma unroll
        for (int n = 0; n < LV; ++n) {
            const int r = (tid + n * NTH) / UV, c = (tid + n * NTH) % UV;
            u32x4 wv = {0, 0, 0, 0};
            if (r < len && v0 + 8 * c < op.vd)
                wv = *reinterpret_cast<const u32x4 *>(gv + (first + r * dir) * op.v.stride + 8 * c);
            *reinterpret_cast<u32x4 *>(s_v + place<UV>(r, c) * 8) = wv;
        }
        __syncthreads();

        // ---- weighted scores, 32 x 32 tiles (rt, ct) with ct <= rt: lane =
        // token i, registers = tokens j (as channels of the state)
#pragma unroll
        for (int tile = 0; tile < 3; ++tile) {
            if (tile % NW != wave) continue;
            const int rt = tile == 0 ? 0 : 1, ct = tile == 2 ? 1 : 0;
            f32x16 a = {};
#pragma unroll
            for (int u = 0; u < KD / 16; ++u)
                a = mfma32_bf16(row_read<UK>(s_k, 32 * ct + channel(l32), 2 * u + hh),
                                row_read<UK>(s_q, 32 * rt + l32, 2 * u + hh), a);
            const int i = 32 * rt + l32;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float f[8];
                const int j0 = 32 * ct + 16 * x + 8 * hh;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = i - (j0 + e);
                    f[e] = d >= 0 ? a[8 * x + e] * (op.scale_pair * fast_exp2(l2 * (float)d)) : 0.f;
                }
                *reinterpret_cast<bf16x8 *>(s_p + place<8>(i, j0 / 8) * 8) = pack8(f);
            }
        }

        // ---- output from the state, out^T = S q^T (channels x tokens)
        f32x16 O[2] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = S[t][8 * x + e];
                const bf16x8 a = pack8(f);
#pragma unroll
                for (int rt = 0; rt < 2; ++rt)
                    O[rt] = mfma32_bf16(a, row_read<UK>(s_q, 32 * rt + l32, 4 * t + 2 * x + hh), O[rt]);
            }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
            O[rt] *= op.scale_state * fast_exp2(l2 * ((float)(32 * rt + l32) + 1.f - shift));
        __syncthreads();  // scores complete

        // ---- output from the chunk, and the state update, 16 tokens at a time
        const float keep = fast_exp2(l2 * (float)len);
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] *= keep;
#pragma unroll
        for (int u = 0; u < kTok / 16; ++u) {
            const bf16x8 v = column_read<UV>(s_v, 16 * u, 32 * wave, lane);
            if (u < 2) O[0] = mfma32_bf16(v, row_read<8>(s_p, l32, 2 * u + hh), O[0]);
            O[1] = mfma32_bf16(v, row_read<8>(s_p, 32 + l32, 2 * u + hh), O[1]);
            float f[8], r[8];
            unpack8(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = max(len - 1 - (16 * u + 8 * hh + e), 0);
                f[e] *= op.scale_update * fast_exp2(l2 * ((float)d + shift));
            }
            const bf16x8 w1 = pack8(f);
            unpack8(w1, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= r[e];
            const bf16x8 w2 = pack8(f);
            unpack8(w2, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= r[e];
            const bf16x8 w3 = pack8(f);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bf16x8 k = column_read<UK>(s_k, 16 * u, 32 * t, lane);
                S[t] = mfma32_bf16(k, w3, S[t]);
                S[t] = mfma32_bf16(k, w2, S[t]);
                S[t] = mfma32_bf16(k, w1, S[t]);
            }
        }

        // ---- 16-byte stores: token 32 rt + l32, channels 16 x + 8 hh ..
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const int r = 32 * rt + l32;
            if (r >= len) continue;
            const int64_t row = ((first + r * dir) * p.H + h) * op.vd;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int vc = v0 + 32 * wave + 16 * x + 8 * hh;
                if (vc >= op.vd) continue;
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = O[rt][8 * x + e];
                if (op.out_f32)
                    store_state8<false>(op.out, row + vc, f);
                else
                    store_state8<true>(op.out, row + vc, f);
            }
        }
    }

    if (op.state_out == nullptr || !vch_in) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int kc = 32 * t + 16 * x + 8 * hh;
            if (kc >= op.kd) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = S[t][8 * x + e];
            write_state<SB>(op.state_out, state_at + kc * op.sk, op.sk, f);
        }
}

// One thread per 8 channels of a (token, group); the sequences' rows only.
__global__ __launch_bounds__(256) void la_group_sum(const float *src, uint16_t *dst, const int32_t *qsl, int batch,
                                                    int64_t n8, int G, int div, int w8) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const int64_t tg = i / w8, t = tg / G;
    if (t < qsl[0] || t >= qsl[batch]) return;
    const int c = (int)(i - tg * w8) * 8;
    float s[8] = {};
    for (int d = 0; d < div; ++d) {
        float f[8];
        load_state8<false>(src, (tg * div + d) * (int64_t)w8 * 8 + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += f[e];
    }
    store_state8<true>(dst, i * 8, s);
}

template <int KD, int NW>
hipError_t launch_kd(const Params &p, int nops, int tiles, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.batch * p.H), (unsigned)tiles, (unsigned)nops), block(64 * NW);
    if (p.state_bf16)
        la_walk<KD, NW, true><<<grid, block, 0, s>>>(p);
    else
        la_walk<KD, NW, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}
template <int KD>
hipError_t launch_nw(const Params &p, int nops, int vd, hipStream_t s) {
    if (vd <= 64) return launch_kd<KD, 2>(p, nops, 1, s);
    return launch_kd<KD, 4>(p, nops, (vd + 127) / 128, s);
}
}  // namespace

hipError_t launch_walk(const Params &p, int nops, hipStream_t s) {
    int kd = 0, vd = 0;
    for (int i = 0; i < nops; ++i) {
        kd = std::max(kd, p.op[i].kd);
        vd = std::max(vd, p.op[i].vd);
    }
    if (kd <= 64) return launch_nw<64>(p, nops, vd, s);
    if (kd <= 128) return launch_nw<128>(p, nops, vd, s);
    return launch_nw<256>(p, nops, vd, s);
}

hipError_t launch_group_sum(const float *src, uint16_t *dst, const Params &p, int div, int width, hipStream_t s) {
    const int G = p.H / div;
    const int64_t n8 = p.T * G * (width / 8);
    la_group_sum<<<dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s>>>(src, dst, p.qsl, p.batch, n8, G, div,
                                                                         width / 8);
    return hipGetLastError();
}

}  // namespace la
}  // namespace ssd
