// Linear attention with a fixed decay per head: the chunked form, forward
// and (as three recurrences with exchanged roles) backward.
//
// A workgroup walks one segment of a sequence for one head and 16 * NW value
// channels, in chunks of 64 tokens.  With i, j the places in a chunk, S the
// state that enters it and lambda the head's decay,
//     out_i = lambda^(i+1) S q_i + sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j
//     S    <- lambda^len S + sum_j lambda^(len-1-j) v_j k_j^T
// Each wavefront owns 16 value channels and keeps S of them (16 x kd, fp32)
// in registers for the whole walk, so the state never moves; the wavefronts
// share only the chunk's q, k, v rows and its 64 x 64 matrix of weighted
// scores, in LDS.  Every product is computed transposed (channels x tokens):
// a lane then holds one token and consecutive channels, so its decay is a
// scalar, and the state registers are, as they are, the operand of the next
// product.
//
// Operands that run along tokens (v and k of the state update) come from LDS
// with the transposing read, whose lanes take columns in groups of four.  For
// k (and for the rows of k in the scores) two tiles of 16 channels are taken
// from 32, channels 8 g + 0..3 to the one and 8 g + 4..7 to the other, so
// that the two accumulators of a lane together are 8 consecutive channels:
// one 16-byte operand of the next product.
//
// Rounding: scores and the state are rounded to bf16 once as operands of the
// output, which is bf16 itself.  The weighted v of the state update is split
// into three bf16 parts that carry its 24 bits where the state is returned in
// fp32, so it is that of fp32 sums; into two, 2.4e-6 off in norm, where it
// only enters bf16 values (outputs, bf16 states).
#include "ssd_linear_attn.hpp"

namespace ssd {
namespace la {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;

// LDS layout of a chunk's rows: unit c (16 bytes, 8 channels) of row r at
// byte c kUnit + 16 r.  16 consecutive rows of a unit are 256 bytes (every
// bank once), and units lie 16 banks apart (kUnit = 1024 + 64), so 4 rows x 4
// units, which the transposing reads and the stores touch at a time, do not
// meet either.  Every place is a lane's base plus a constant, which is the
// offset field of the instruction: one register serves a whole phase.
constexpr int kUnit = kTok * 16 + 64;

__device__ __forceinline__ bf16x8 read_unit(const char *s, int at) {
    return *reinterpret_cast<const bf16x8 *>(s + at);
}

// Transposing read: lane l gets 8 tokens (`at` of lane l is 4 channels of token
// 8 (l / 16) + l % 16 / 4; the lanes' 16 columns are those 4 of lanes 0 .. 3 of
// its 16 in turn).
__device__ __forceinline__ bf16x8 read_columns(const char *s, int at) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + at + 4 * 16));
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

__device__ __forceinline__ int clamp_row(const Params &p, int t) { return min(max(t, 0), (int)p.T); }

// whether sequence b of an operation starts from a stored state
__device__ __forceinline__ bool resumes(const Params &p, const Op &op, int b) {
    return op.state_in != nullptr && (p.init_all != 0 || (p.has_init != nullptr && p.has_init[b] != 0));
}

// The segment a workgroup takes.  Sequences are cut into segments of `seg`
// tokens counted in walking order; slot w of the launch is segment w - first
// of the last sequence whose first slot, qsl / seg + b, is at most w.  (A
// sequence of n tokens has at most n / seg + 1 segments, so their slots never
// meet the next sequence's; slots in between are empty.)  Every lane tests one
// sequence at a time, so 64-ary search finds it in one or two steps.
struct Segment {
    int b, index, count;  // sequence, segment of it, its number of segments (0: an empty slot)
    int begin, len;       // the sequence's first token and length
};
__device__ __forceinline__ Segment find_segment(const Params &p, int w) {
    const int lane = threadIdx.x & 63;
    Segment g;
    int lo = 0, first = 0;
    if (p.seg == 0) {  // one segment per sequence
        lo = w;
        first = w;
    } else {
        int n = p.batch;
        while (true) {
            const int step = (n + 63) / 64;
            const int i = lane * step;
            bool at = false;
            if (i < n) at = clamp_row(p, p.qsl[lo + i]) / p.seg + lo + i <= w;
            const int k = __popcll(__ballot(at)) - 1;
            if (k < 0) return Segment{0, 0, 0, 0, 0};
            lo += k * step;
            n = min(step, n - k * step);
            if (n <= 1) break;
        }
    }
    g.b = __builtin_amdgcn_readfirstlane(lo);
    g.begin = __builtin_amdgcn_readfirstlane(clamp_row(p, p.qsl[g.b]));
    g.len = max(__builtin_amdgcn_readfirstlane(clamp_row(p, p.qsl[g.b + 1])) - g.begin, 0);
    if (p.seg == 0) {
        g.index = 0;
        g.count = 1;
    } else {
        g.index = w - (g.begin / p.seg + g.b);
        g.count = max((g.len + p.seg - 1) / p.seg, 1);
        if (g.index >= g.count) g.count = 0;
    }
    return g;
}

// Raw buffer over the rows of one chunk: rows past it read as zero and are
// not stored.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, kBufferFormat32);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every such buffer

// Wavefronts per SIMD that the registers of a variant allow.
constexpr int waves_of(int KD, int NW) { return KD > 128 ? 2 : NW == 8 ? 4 : 3; }

// KD: channels of k and q the kernel holds (kd rounded up; the rest is zero).
// LOCAL: only the state a segment leaves when it starts from zero.
template <int KD, int NW, bool SB, bool LOCAL>
__global__ __launch_bounds__(64 * NW, waves_of(KD, NW)) void la_walk(Params p) {
    constexpr int NTH = 64 * NW;
    constexpr int UK = KD / 8;       // 16-byte units of a q or k row
    constexpr int VT = 16 * NW;      // value channels of the workgroup
    constexpr int UV = VT / 8;
    constexpr int NT = KD / 32;      // blocks of 32 k channels of a wavefront's state
    constexpr int LK = kTok * UK / NTH, LV = kTok * UV / NTH;  // 16-byte loads of a thread
    constexpr int RK = NTH / UK, RV = NTH / UV;                // rows between them
    __shared__ __attribute__((aligned(16))) char s_q[LOCAL ? 16 : UK * kUnit];
    __shared__ __attribute__((aligned(16))) char s_k[UK * kUnit];
    __shared__ __attribute__((aligned(16))) char s_v[UV * kUnit];
    __shared__ __attribute__((aligned(16))) char s_p[LOCAL ? 16 : kTok / 8 * kUnit];
    __shared__ float s_pair[96], s_lead[32];

    // Consecutive workgroups go to the 8 XCDs in turn.  The workgroups that
    // read the same rows (a group's heads, their blocks of channels, the
    // recurrences) stay on one XCD, and its L2.
    const int together = p.share * p.tiles * p.nops;
    const int run = (int)blockIdx.x / 8;
    int id = (run / together * 8 + (int)(blockIdx.x % 8)) * together + run % together;
    if (id >= p.slots * p.H * p.tiles * p.nops) return;
    const int which = id % p.nops;
    id /= p.nops;
    const int v0 = (id % p.tiles) * VT;
    id /= p.tiles;
    const int h = id % p.H, w = id / p.H;
    const Op &op = p.op[which];
    if (v0 >= op.vd) return;
    const int tid = threadIdx.x;
    const int lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const Segment g = find_segment(p, w);
    if (g.count == 0 || (LOCAL && g.index == g.count - 1)) return;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[g.b] : (int64_t)g.b;
    if (slot >= p.max_slots) return;  // padding
    // the segment's tokens: n of them, from t0 upwards
    const int skip = p.seg == 0 ? 0 : g.index * p.seg;
    const int n = p.seg == 0 ? g.len : min(p.seg, g.len - skip);
    const bool rev = op.reverse != 0;
    const int64_t t0 = rev ? g.begin + g.len - skip - n : g.begin + skip;
    // log2 of the decay; -infinity as a finite number, so that times 0 it is 0
    const float ld = p.log_decay[h] * kLog2e;
    const float l2 = ld < -1e30f ? -1e30f : ld;
    const float shift = rev ? 1.f : 0.f;

    // ---- the state: register 4 y + e (y 0, 1) of block t holds v channel vch
    // and k channel 32 t + 8 q4 + 4 y + e
    const int vch = v0 + 16 * wave + l16;
    const bool vch_in = vch < op.vd;
    const int64_t state_at = (slot * p.H + h) * p.state_size + (int64_t)vch * op.sv;
    // the wavefront's part of the segment's slot in the workspace
    f32x4 *const part = reinterpret_cast<f32x4 *>(
        p.parts + ((((int64_t)which * p.slots + w) * p.H + h) * p.tiles * VT + v0 + 16 * wave) * KD) + lane;
    f32x4 S[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t][0] = S[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!LOCAL) {
        if (g.count > 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < 2; ++y) S[t][y] = part[(t * 2 + y) * 64];
        } else if (resumes(p, op, g.b) && vch_in) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int kc = 32 * t + 8 * q4;
                if (kc >= op.kd) continue;
                float f[8];
                read_state<SB>(op.state_in, state_at + kc * op.sk, op.sk, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[t][e / 4][e % 4] = f[e];
            }
        }
    }

    // ---- constants of the walk.  Place r of a chunk of len tokens is its
    // token r - pad (pad = 64 - len), or in reverse 63 - r: a short chunk ends
    // at the last place, where the weights of the state update are the full
    // chunk's, and starts with rows of zeros.
    // In LDS: weights of the scores by distance i - j (0 above the diagonal),
    // from distance -31 on, and of the last 32 tokens in the state update.
    if (tid < 64 + 31) {
        const int d = tid - 31;
        s_pair[tid] = d >= 0 ? op.scale_pair * fast_exp2(l2 * (float)d) : 0.f;
        if (tid < 32) s_lead[tid] = op.scale_update * fast_exp2(l2 * ((float)tid + shift));
    }
    const bool fine = !SB && op.state_out != nullptr;  // three parts of the weighted v, or two
    const float by32 = fast_exp2(l2 * 32.f);

    const int64_t qs = op.q.stride, ks = op.k.stride, vs = op.v.stride, os = (int64_t)p.H * op.vd;
    const uint16_t *gq = op.q.p + (int64_t)(h / op.q.div) * op.kd;
    const uint16_t *gk = op.k.p + (int64_t)(h / op.k.div) * op.kd;
    const uint16_t *gv = op.v.p + (int64_t)(h / op.v.div) * op.vd;
    // A thread's unit and row of the loads: 16 lanes take 4 rows of 4 units.
    // The thread number is made opaque wherever they are used, so that they are
    // formed again instead of held in some ten registers across the chunk.
    auto unit_of = [](int t, int U) { return (t >> 4) % (U / 4) * 4 + (t & 3); };
    auto row_of = [](int t, int U) { return (t >> 4) / (U / 4) * 4 + (t >> 2) % 4; };
    auto opaque = [](int t) {
        asm volatile("" : "+v"(t));
        return t;
    };

    u32x4 fq[LOCAL ? 1 : LK], fk[LK], fv[LV];
    auto fetch = [&](int c0) {  // the chunk's rows, lowest token first, into registers
        const int len = min(kTok, n - c0);
        const int64_t first = rev ? t0 + n - c0 - len : t0 + c0;
        const auto bk = rows_buffer(gk + first * ks, (uint32_t)((len - 1) * ks + op.kd) * 2);
        const auto bv = rows_buffer(gv + first * vs, (uint32_t)((len - 1) * vs + op.vd) * 2);
        const int t = opaque(tid), ck = unit_of(t, UK), rk = row_of(t, UK), cv = unit_of(t, UV), rv = row_of(t, UV);
        const uint32_t ok = 8 * ck < op.kd ? (uint32_t)(rk * (int)ks + 8 * ck) * 2 : kNowhere;
        const uint32_t ov = v0 + 8 * cv < op.vd ? (uint32_t)(rv * (int)vs + v0 + 8 * cv) * 2 : kNowhere;
#pragma unroll
        for (int i = 0; i < LK; ++i)
            fk[i] = __builtin_amdgcn_raw_buffer_load_b128(bk, ok + i * RK * (uint32_t)ks * 2, 0, 0);
#pragma unroll
        for (int i = 0; i < LV; ++i)
            fv[i] = __builtin_amdgcn_raw_buffer_load_b128(bv, ov + i * RV * (uint32_t)vs * 2, 0, 0);
        if constexpr (!LOCAL) {
            const auto bq = rows_buffer(gq + first * qs, (uint32_t)((len - 1) * qs + op.kd) * 2);
            const uint32_t oq = 8 * ck < op.kd ? (uint32_t)(rk * (int)qs + 8 * ck) * 2 : kNowhere;
#pragma unroll
            for (int i = 0; i < LK; ++i)
                fq[i] = __builtin_amdgcn_raw_buffer_load_b128(bq, oq + i * RK * (uint32_t)qs * 2, 0, 0);
        }
    };
    if (n > 0) fetch(0);

    f32x4 O[4] = {};
    // Stores the outputs of the chunk at c0: place 16 rt + l16, 4 channels from
    // 4 q4.  A chunk's outputs leave behind the barriers of the next one, ahead
    // of its loads: waiting for loads then never waits for younger stores.
    auto emit = [&](int c0) {
        const int len = min(kTok, n - c0), pad = kTok - len;
        const int64_t first = rev ? t0 + n - c0 - len : t0 + c0;
        const int eb = op.out_f32 ? 4 : 2;
        const auto bo = rows_buffer(static_cast<char *>(op.out) + (first * os + (int64_t)h * op.vd) * eb,
                                    (uint32_t)((len - 1) * os + op.vd) * eb);
        const int vc = v0 + 16 * wave + 4 * q4;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const int r = 16 * rt + l16;
            const int tok = rev ? 63 - r : r - pad;
            const uint32_t at =
                vc < op.vd && (uint32_t)tok < (uint32_t)len ? (uint32_t)(tok * (int)os + vc) * eb : kNowhere;
            if (op.out_f32)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[rt]), bo, at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2{pack_bf16x2(O[rt][0], O[rt][1]), pack_bf16x2(O[rt][2], O[rt][3])}, bo, at, 0, 0);
        }
    };

    // a lane's places: rows l16 of unit q4; rows of k as two tiles; columns
    const int at_row = q4 * kUnit + l16 * 16;
    const int at_key = q4 * kUnit + (8 * (l16 >> 2) + (l16 & 3)) * 16;
    const int at_col = (8 * q4 + (l16 >> 2)) * 16;
    const int at_kcol = at_col + (l16 & 3) * kUnit;
    const int at_vcol = at_col + (2 * wave + ((l16 & 3) >> 1)) * kUnit + (l16 & 1) * 8;
    const float *const w_pair = s_pair + 31 + 16 * (wave & 3) + l16 - 8 * q4, *const w_lead = s_lead + 31 - 8 * q4;

#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += kTok) {
        const int len = min(kTok, n - c0), pad = kTok - len;
        __syncthreads();  // the previous chunk's rows are no longer read
        // token i of the chunk to its place; tokens past it (zeros) wrap to the places before it
        const int ft = opaque(tid), ck = unit_of(ft, UK), rk = row_of(ft, UK), cv = unit_of(ft, UV),
                  rv = row_of(ft, UV);
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const int r = rev ? 63 - (rk + i * RK) : (rk + i * RK + pad) & 63;
            *reinterpret_cast<u32x4 *>(s_k + ck * kUnit + r * 16) = fk[i];
            if constexpr (!LOCAL) *reinterpret_cast<u32x4 *>(s_q + ck * kUnit + r * 16) = fq[i];
        }
#pragma unroll
        for (int i = 0; i < LV; ++i) {
            const int r = rev ? 63 - (rv + i * RV) : (rv + i * RV + pad) & 63;
            *reinterpret_cast<u32x4 *>(s_v + cv * kUnit + r * 16) = fv[i];
        }
        __syncthreads();
        if (!LOCAL && c0 > 0) emit(c0 - kTok);
        if (c0 + kTok < n) fetch(c0 + kTok);

        if constexpr (!LOCAL) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) O[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
            // ---- weighted scores in blocks of 16 tokens i (lanes) x 32 tokens
            // j (8 consecutive ones a lane): blocks (rt, c) = (0,0) (1,0) (2,0)
            // (3,0) (2,1) (3,1).  Wavefront m takes block m, and with four
            // of them 0 and 1 also 4 and 5, which lie as far below the diagonal
#pragma unroll
            for (int m = 0; m < 6; ++m) {
                if (m % NW != wave) continue;
                const int rt = m < 4 ? m : m - 2, c = m < 4 ? 0 : 1;
                f32x4 a[2] = {};
#pragma unroll
                for (int u = 0; u < KD / 32; ++u) {
                    const bf16x8 q = read_unit(s_q, at_row + 16 * rt * 16 + 4 * u * kUnit);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        a[y] = mfma_bf16(read_unit(s_k, at_key + (32 * c + 4 * y) * 16 + 4 * u * kUnit), q, a[y]);
                }
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = a[e / 4][e % 4] * w_pair[-e];
                *reinterpret_cast<bf16x8 *>(s_p + at_row + 16 * rt * 16 + 4 * c * kUnit) = pack8(f);
            }
            // ---- output from the state, out^T = S q^T (channels x tokens)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = S[t][e / 4][e % 4];
                const bf16x8 a = pack8(f);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt)
                    O[rt] = mfma_bf16(a, read_unit(s_q, at_row + 16 * rt * 16 + 4 * t * kUnit), O[rt]);
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                O[rt] *= op.scale_state * fast_exp2(l2 * ((float)(16 * rt + l16 - pad + 1) - shift));
            __syncthreads();  // scores complete
        }

        // ---- output from the chunk, and the state update, 32 tokens at a time
        const float keep = fast_exp2(l2 * (float)len);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            S[t][0] *= keep;
            S[t][1] *= keep;
        }
#pragma unroll
        for (int u = 0; u < kTok / 32; ++u) {
            const bf16x8 v = read_columns(s_v, at_vcol + 32 * u * 16);
            if constexpr (!LOCAL) {
#pragma unroll
                for (int rt = 2 * u; rt < 4; ++rt)
                    O[rt] = mfma_bf16(v, read_unit(s_p, at_row + 16 * rt * 16 + 4 * u * kUnit), O[rt]);
            }
            float f[8], r[8];
            unpack8(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= w_lead[-e] * (u == 0 ? by32 : 1.f);
            const bf16x8 w1 = pack8(f);
            unpack8(w1, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= r[e];
            const bf16x8 w2 = pack8(f);
            bf16x8 w3;
            if (fine) {
                unpack8(w2, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] -= r[e];
                w3 = pack8(f);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bf16x8 k0 = read_columns(s_k, at_kcol + 32 * u * 16 + 4 * t * kUnit);
                const bf16x8 k1 = read_columns(s_k, at_kcol + 32 * u * 16 + 4 * t * kUnit + 8);
                if (fine) {
                    S[t][0] = mfma_bf16(k0, w3, S[t][0]);
                    S[t][1] = mfma_bf16(k1, w3, S[t][1]);
                }
                S[t][0] = mfma_bf16(k0, w2, S[t][0]);
                S[t][1] = mfma_bf16(k1, w2, S[t][1]);
                S[t][0] = mfma_bf16(k0, w1, S[t][0]);
                S[t][1] = mfma_bf16(k1, w1, S[t][1]);
            }
        }
    }
    if (!LOCAL && n > 0) emit((n - 1) / kTok * kTok);

    if constexpr (LOCAL) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) part[(t * 2 + y) * 64] = S[t][y];
    } else {
        if (g.index != g.count - 1 || op.state_out == nullptr || !vch_in) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int kc = 32 * t + 8 * q4;
            if (kc >= op.kd) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = S[t][e / 4][e % 4];
            write_state<SB>(op.state_out, state_at + kc * op.sk, op.sk, f);
        }
    }
}

// The segments' own states into the states that enter them, in place: one
// thread per 4 state elements of a (sequence, head), in the order of the
// walk's registers.  Sequences of one segment are left to the walk.
template <bool SB>
__global__ __launch_bounds__(256) void la_chain(Params p, int KD, int VT) {
    const int per_head = p.tiles * VT * KD / 4;  // groups of 4
    const int blocks = (per_head + 255) / 256;
    int id = blockIdx.x;
    const int i = (id % blocks) * 256 + (int)threadIdx.x;
    id /= blocks;
    const int h = id % p.H, b = id / p.H;
    const int which = blockIdx.y;
    const Op &op = p.op[which];
    if (i >= per_head) return;
    const int begin = clamp_row(p, p.qsl[b]), len = max(clamp_row(p, p.qsl[b + 1]) - begin, 0);
    const int count = (len + p.seg - 1) / p.seg;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[b] : (int64_t)b;
    if (count <= 1 || slot >= p.max_slots) return;
    const int lane = i & 63, y = (i >> 6) & 1, t = (i >> 7) % (KD / 32), wave = (i >> 7) / (KD / 32);
    const int vch = 16 * wave + (lane & 15), kc = 32 * t + 8 * (lane >> 4) + 4 * y;
    const bool in = vch < op.vd && kc < op.kd;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (in && resumes(p, op, b)) {
        const int64_t at = (slot * p.H + h) * p.state_size + (int64_t)vch * op.sv + kc * op.sk;
        if (op.sk == 1) {
            S = load_state4<SB>(op.state_in, at);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[e] = SB ? bf16_bits_to_float(static_cast<const uint16_t *>(op.state_in)[at + e * op.sk])
                          : static_cast<const float *>(op.state_in)[at + e * op.sk];
        }
    }
    const float ld = p.log_decay[h] * kLog2e;
    const float keep = fast_exp2((ld < -1e30f ? -1e30f : ld) * (float)p.seg);
    const int64_t step = (int64_t)p.H * per_head;
    f32x4 *part = reinterpret_cast<f32x4 *>(p.parts) +
                  ((int64_t)which * p.slots + begin / p.seg + b) * step + (int64_t)h * per_head + i;
    for (int s = 0; s < count - 1; ++s, part += step) {
        const f32x4 own = *part;
        *part = S;
        S = S * keep + own;
    }
    *part = S;
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

template <int KD, int NW, bool SB>
hipError_t launch_kd(const Params &p, hipStream_t s) {
    const int64_t n = (int64_t)p.slots * p.H * p.tiles * p.nops;
    const int64_t run = (int64_t)8 * p.share * p.tiles * p.nops;
    const dim3 grid((unsigned)((n + run - 1) / run * run)), block(64 * NW);
    if (p.seg != 0) {
        la_walk<KD, NW, SB, true><<<grid, block, 0, s>>>(p);
        const int blocks = (p.tiles * 16 * NW * KD / 4 + 255) / 256;
        const dim3 cg((unsigned)(p.batch * p.H * blocks), (unsigned)p.nops);
        la_chain<SB><<<cg, dim3(256), 0, s>>>(p, KD, 16 * NW);
    }
    la_walk<KD, NW, SB, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}
template <int KD>
hipError_t launch_nw(const Params &p, const Shape &h, hipStream_t s) {
    if (h.nw == 4) return p.state_bf16 ? launch_kd<KD, 4, true>(p, s) : launch_kd<KD, 4, false>(p, s);
    return p.state_bf16 ? launch_kd<KD, 8, true>(p, s) : launch_kd<KD, 8, false>(p, s);
}
}  // namespace

// Segments: a walk is a chain of chunks, so a launch needs enough of them
// side by side: kTarget workgroups, two per compute unit, each of at least
// kLeast tokens.  Sequences no longer than a segment are not cut.
Shape shape_of(int64_t T, int batch, int H, int kd, int vd, int nops) {
    constexpr int64_t kTarget = 512, kLeast = 256;
    Shape h;
    h.kd = kd <= 64 ? 64 : kd <= 128 ? 128 : 256;
    h.nw = vd <= 64 ? 4 : 8;
    h.tiles = (vd + 16 * h.nw - 1) / (16 * h.nw);
    const int64_t want = T * H * h.tiles * nops / kTarget;  // tokens
    const int64_t seg = std::max((want + kTok - 1) / kTok * kTok, kLeast);
    h.seg = T > seg ? (int)seg : 0;
    h.slots = h.seg != 0 ? (int)(T / seg) + batch : batch;
    h.bytes = h.seg != 0 ? (size_t)nops * h.slots * H * h.tiles * 16 * h.nw * h.kd * sizeof(float) : 0;
    return h;
}

hipError_t launch_walk(Params &p, const Shape &h, int nops, hipStream_t s) {
    p.nops = nops;
    p.tiles = h.tiles;
    p.seg = h.seg;
    p.slots = h.slots;
    if (h.kd == 64) return launch_nw<64>(p, h, s);
    if (h.kd == 128) return launch_nw<128>(p, h, s);
    return launch_nw<256>(p, h, s);
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
