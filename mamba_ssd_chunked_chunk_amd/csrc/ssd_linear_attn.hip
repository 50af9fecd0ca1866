// Linear attention with a fixed decay per head: the chunked form, forward
// and (as three recurrences with exchanged roles) backward.
//
// A workgroup walks one segment of a sequence, in chunks of 64 tokens, for one
// head and VT value channels, or for HP heads that share q and k.  With i, j
// the places in a chunk, S the state that enters it and lambda the head's decay,
//     out_i = lambda^(i+1) S q_i + sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j
//     S    <- lambda^len S + sum_j lambda^(len-1-j) v_j k_j^T
// Each wavefront owns 16 DT value channels and keeps S of them (fp32) in
// registers for the whole walk, so the state never moves; the wavefronts share
// only the chunk's q, k, v rows and its 64 x 64 matrix of weighted scores, in
// LDS.  Every product is computed transposed (channels x tokens): a lane then
// holds one token and consecutive channels, so its decay is a scalar, and the
// state registers are, as they are, the operand of the next product.
//
// LDS is what a wavefront of 16 channels is bound by (32 ragged prompts of 128
// heads: active 64% of a compute unit's cycles, 42% of those in conflicts), since
// all of them read all of q and k; 32 channels (DT 2) and the orders below bring
// that to 38%, 24% of those in conflicts.  The orders
// below let every large read touch each bank once:
//   - rows lie unit by unit (16 bytes, 8 channels), units 16 banks apart;
//   - operands along tokens come from the transposing read, 4 rows of 4 half
//     units at a time, two such tiles for 32 channels (the lane groups then use
//     the same half of the banks: half rate, cheaper than exchanging halves in
//     registers);
//   - of the 32 tokens of a product, lane group q4 takes 4 q4 .. + 3 and 16 + 4 q4 .. + 3
//     (k, v and the scores alike: a sum's order is free);
//   - of 32 rows of q or scores, the first 16-row tile takes 0 .. 3, 8 .. 11,
//     .., the second the others.
//
// What bounds it: 65536 tokens of 16 heads of 128 x 128: the walk 233 us (1.11 GB
// counted, 4.8 TB/s, a copy's being 5.1), the pass for segments' states 132 us
// (0.55 GB, 4.2 TB/s): memory; the call takes 393 us, 370 with most products left
// out and 241 with no rows moved after the first.  32 ragged prompts of 128 heads
// that share q and k by 16: 538 us (1.76 GB), 402 with most products left out, 328
// with no rows moved: with two workgroups a compute unit the two overlap only in
// part (matrix cores busy 35% of the cycles, LDS 38%).
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

// LDS layout of a chunk's CT rows: unit c of row r at byte c unit_bytes + 16 r.
// Every place is a lane's base plus a constant, which is the offset field of
// the instruction: one register serves a whole phase.
constexpr int unit_bytes(int CT) { return CT * 16 + 64; }

__device__ __forceinline__ bf16x8 read_unit(const char *s, int at) {
    return *reinterpret_cast<const bf16x8 *>(s + at);
}

// Transposing read: lane l gets the tokens r .. r + 3 and r + 16 .. r + 19 of one
// of 16 columns; `at` of lane l is row r + l % 16 / 4 of the four columns that
// lanes 4 (l % 4) .. + 3 of its 16 get.
__device__ __forceinline__ bf16x8 read_columns(const char *s, int at) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s + at + 16 * 16));
    const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// the 32 channels of two tiles: lane l of tile y (0, 1) of 16 columns
__device__ __forceinline__ int column(int l, int y) { return 8 * (l >> 2) + 4 * y + (l & 3); }

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
__device__ __forceinline__ int clamp_row(const Params &p, int t) { return min(max(t, 0), (int)p.T); }

// log2 of a head's decay; -infinity as a finite number, so that times 0 it is 0
__device__ __forceinline__ float log2_decay(const Params &p, int h) {
    const float ld = p.log_decay[h] * kLog2e;
    return ld < -1e30f ? -1e30f : ld;
}

// a uniform value as one the compiler has to keep
__device__ __forceinline__ int held(int x) {
    x = __builtin_amdgcn_readfirstlane(x);
    asm volatile("" : "+s"(x));
    return x;
}
__device__ __forceinline__ float held(float x) { return __int_as_float(held(__float_as_int(x))); }

// whether sequence b of an operation starts from a stored state
__device__ __forceinline__ bool resumes(const Params &p, const Op &op, int b) {
    return op.state_in != nullptr && (p.init_all != 0 || (p.has_init != nullptr && p.has_init[b] != 0));
}

// Only sequences of more than a segment are cut, and only those have states in
// the workspace.  Ahead of a sequence that starts at row `begin` there are at most
// begin / (seg + 1) of them (and at most b sequences at all): its number among
// those that could be, which is less than p.cuts and another for each cut one.
__device__ __forceinline__ int cut_number(const Params &p, int begin, int b) { return min(b, begin / (p.seg + 1)); }

// The workspace's slot of a cut sequence's first part.  floor(begin / sub) grows by
// at least its number of parts less one up to the next cut sequence and cut_number
// by one, so their slots never meet; p.sub_slots holds them whatever the table says.
__device__ __forceinline__ int first_slot(const Params &p, int begin, int b) {
    return begin / p.sub + cut_number(p, begin, b);
}

// The last sequence b with number(b, its first row) <= w, or -1, for numbers that
// never decrease: every lane tests one sequence at a time, a 64-ary search.
template <typename F>
__device__ __forceinline__ int last_up_to(const Params &p, int w, F number) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = p.batch;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int i = lane * step;
        bool at = false;
        if (i < n) at = number(lo + i, clamp_row(p, p.qsl[lo + i])) <= w;
        const int k = __popcll(__ballot(at)) - 1;
        if (k < 0) return -1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The segment a workgroup takes: sequences are cut into segments of `seg`
// tokens (0: not cut), counted in walking order, and number w of the launch is
// one of them or none.  LOCAL: a part, p.seg / seg of which make a segment; of up
// to 64 sequences only the parts of segments that another follows are numbered,
// and one vote finds that there are none (the ragged prompts below, where no
// sequence is cut: 6 us for the pass instead of 30; 4 x 4096 tokens of 16 heads,
// backward: 236 -> 224 for the call).
struct Segment {
    int b, index, count;  // sequence, segment of it, its number of segments (0: none)
    int begin, len;       // the sequence's first token and length
};
template <bool LOCAL>
__device__ __forceinline__ Segment find_segment(const Params &p, int w, int seg) {
    const int lane = threadIdx.x & 63;
    const Segment none = {0, 0, 0, 0, 0};
    Segment g;
    if (p.batch <= 64) {
        // Longest sequences first, since what starts last must not be long (32
        // ragged prompts of 128 heads, 18 to 7975 tokens, the last of 5032: 601 ->
        // 531 us).  Lane b holds sequence b and counts the segments ahead of its own.
        int begin = 0, len = -1, count = 0, first = 0;
        if (lane < p.batch) {
            begin = clamp_row(p, p.qsl[lane]);
            len = max(clamp_row(p, p.qsl[lane + 1]) - begin, 0);
            if (LOCAL)
                count = len > p.seg ? (len - 1) / p.seg * (p.seg / seg) : 0;
            else
                count = seg == 0 ? 1 : max((len + seg - 1) / seg, 1);
        }
        if (LOCAL && __ballot(count != 0) == 0) return none;  // no sequence is cut
        for (int j = 0; j < p.batch; ++j) {
            const int l = __builtin_amdgcn_readlane(len, j), c = __builtin_amdgcn_readlane(count, j);
            first += l > len || (l == len && j < lane) ? c : 0;
        }
        const uint64_t at = __ballot(first <= w && w < first + count);
        if (at == 0) return none;
        g.b = (int)__builtin_ctzll(at);
        g.begin = __builtin_amdgcn_readlane(begin, g.b);
        g.len = __builtin_amdgcn_readlane(len, g.b);
        g.count = LOCAL ? (g.len + seg - 1) / seg : __builtin_amdgcn_readlane(count, g.b);
        g.index = w - __builtin_amdgcn_readlane(first, g.b);
        return g;
    }
    // Many sequences: in their order.  Sequence b's numbers start at qsl / seg +
    // b (a sequence of n tokens has at most n / seg + 1 segments, so they never
    // meet the next one's; those in between are nobody's), a cut one's parts at
    // their slot.
    auto number = [&](int b, int begin) { return LOCAL ? first_slot(p, begin, b) : begin / seg + b; };
    const int b = seg == 0 ? w : last_up_to(p, w, number);
    if (b < 0) return none;
    g.b = __builtin_amdgcn_readfirstlane(b);
    g.begin = __builtin_amdgcn_readfirstlane(clamp_row(p, p.qsl[g.b]));
    g.len = max(__builtin_amdgcn_readfirstlane(clamp_row(p, p.qsl[g.b + 1])) - g.begin, 0);
    if (seg == 0) {
        g.index = 0;
        g.count = 1;
    } else {
        if (LOCAL && g.len <= p.seg) return none;
        g.index = w - number(g.b, g.begin);
        g.count = max((g.len + seg - 1) / seg, 1);
        if (g.index < 0 || g.index >= g.count) g.count = 0;
    }
    return g;
}

// Raw buffer over the rows of one chunk: rows past it read as zero and are
// not stored.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, kBufferFormat32);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every such buffer

// KD: channels of k and q the kernel holds (kd rounded up; the rest is zero);
// CT: tokens of a chunk; NW wavefronts of DT tiles of 16 value channels, for HP
// heads.
// LOCAL: only the state a segment leaves when it starts from zero.
template <int KD, int CT, int NW, int DT, int HP, bool SB, bool LOCAL>
__global__ __launch_bounds__(64 * NW, CT == 64 ? 2 : 3) void la_walk(Params p) {
    constexpr int kUnit = unit_bytes(CT);
    constexpr int RT = CT / 16;      // 16-token tiles of a chunk
    constexpr int NTH = 64 * NW;
    constexpr int WH = NW / HP;      // wavefronts of a head
    constexpr int VT = 16 * DT * WH; // value channels of the workgroup, of each head
    constexpr int UK = KD / 8;       // units of a q or k row
    constexpr int UV = HP * VT / 8;  // and of the heads' v rows together
    constexpr int NT = KD / 32;      // blocks of 32 k channels of a wavefront's state
    constexpr int LK = CT * UK / NTH, LV = CT * UV / NTH;  // 16-byte loads of a thread
    constexpr int RK = NTH / UK, RV = NTH / UV;                // rows between them
    constexpr int kScores = CT / 8 * kUnit;
    static_assert(VT % 32 == 0, "pairs of tiles");
    __shared__ __attribute__((aligned(16))) char s_q[LOCAL ? 16 : UK * kUnit];
    __shared__ __attribute__((aligned(16))) char s_k[UK * kUnit];
    __shared__ __attribute__((aligned(16))) char s_v[UV * kUnit];
    __shared__ __attribute__((aligned(16))) char s_p[LOCAL ? 16 : HP * kScores];
    __shared__ float s_pair[HP][CT + 32], s_lead[HP][CT];

    // Consecutive workgroups go to the 8 XCDs in turn.  The workgroups that
    // read the same rows (a group's heads, their blocks of channels, the
    // recurrences) stay on one XCD, and its L2.
    const int together = p.share / HP * p.tiles * p.nops;
    const int run = (int)blockIdx.x / 8;
    int id = (run / together * 8 + (int)(blockIdx.x % 8)) * together + run % together;
    if (id >= (LOCAL ? p.sub_slots : p.slots) * (p.H / HP) * p.tiles * p.nops) return;
    const int which = id % p.nops;
    id /= p.nops;
    const int v0 = (id % p.tiles) * VT;
    id /= p.tiles;
    const int h0 = id % (p.H / HP) * HP, w = id / (p.H / HP);
    const Op &op = p.op[which];
    // what the walk needs of it, held in scalar registers (a scalar load inside
    // the walk would wait for every LDS read before it)
    const int kd = held(op.kd), vd = held(op.vd), out_f32 = held(op.out_f32);
    const int qs = held((int)op.q.stride), ks = held((int)op.k.stride), vs = held((int)op.v.stride);
    const bool rev = held(op.reverse) != 0;
    const float scale_state = held(op.scale_state);
    if (v0 >= vd) return;
    const int tid = threadIdx.x;
    const int lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hw = wave / WH, h = h0 + hw;  // the wavefront's head

    if (LOCAL && op.twin != 0) return;  // la_chain makes its states from the twin's
    const int seg = LOCAL ? p.sub : p.seg;
    const Segment g = find_segment<LOCAL>(p, w, seg);
    if (g.count == 0) return;
    // nothing follows the last segment
    if (LOCAL && g.index * p.sub >= (g.len - 1) / p.seg * p.seg) return;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[g.b] : (int64_t)g.b;
    if (slot >= p.max_slots) return;  // padding
    // the segment's tokens: n of them, from t0 upwards
    const int skip = g.index * seg;
    const int n = seg == 0 ? g.len : min(seg, g.len - skip);
    const int64_t t0 = rev ? g.begin + g.len - skip - n : g.begin + skip;
    const float l2 = log2_decay(p, h);
    const float shift = rev ? 1.f : 0.f;

    // ---- the state: register e of S[t][y][d] holds k channel 32 t + 8 q4 + 4 y
    // + e and v channel vch(d)
    const int tile0 = wave % WH * DT;  // the wavefront's first tile of the head's value channels
    auto vch = [&](int d) { return v0 + 32 * ((tile0 + d) >> 1) + column(l16, (tile0 + d) & 1); };
    const int64_t state_at = (slot * p.H + h) * p.state_size;
    // the wavefront's part of the slot of the segment's (first) states in the workspace
    const int64_t part_slot =
        g.count > 1 ? first_slot(p, g.begin, g.b) + (LOCAL ? g.index : (int64_t)g.index * (p.seg / p.sub)) : 0;
    f32x4 *const part = reinterpret_cast<f32x4 *>(
        p.parts + ((((int64_t)which * p.sub_slots + part_slot) * p.H + h) * p.tiles * VT + v0 + 16 * tile0) * KD) + lane;
    f32x4 S[NT][2][DT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < DT; ++d) S[t][0][d] = S[t][1][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    bool zero = true;  // no state enters the first chunk
    if constexpr (!LOCAL) {
        if (g.count > 1) {
            zero = false;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int y = 0; y < 2; ++y) S[t][y][d] = part[((d * NT + t) * 2 + y) * 64];
        } else if (resumes(p, op, g.b)) {
            zero = false;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int kc = 32 * t + 8 * q4;
                    if (kc >= op.kd || vch(d) >= op.vd) continue;
                    float f[8];
                    read_state<SB>(op.state_in, state_at + vch(d) * op.sv + kc * op.sk, op.sk, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) S[t][e / 4][d][e % 4] = f[e];
                }
        }
    }

    // ---- constants of the walk.  Place r of a chunk of len tokens is its
    // token r - pad (pad = CT - len), or in reverse CT - 1 - r: a short chunk ends
    // at the last place, where the weights of the state update are the full
    // chunk's, and starts with rows of zeros.
    // In LDS: weights of the scores by distance i - j (0 above the diagonal),
    // from distance -31 on, and of the tokens in the state update, last first.
    // Both stop at the segment's tokens: where lambda > 1 a power of the padded
    // rows may be infinite, and rows of zeros would make it NaN.
    if (tid < HP * 128) {
        const int i = tid & 127, d = i - 31;
        const float l2h = HP == 1 ? l2 : log2_decay(p, h0 + (tid >> 7));
        if (i < CT + 31) s_pair[tid >> 7][i] = d >= 0 && d < n ? op.scale_pair * fast_exp2(l2h * (float)d) : 0.f;
        if (i < CT) s_lead[tid >> 7][i] = i < n ? op.scale_update * fast_exp2(l2h * ((float)i + shift)) : 0.f;
    }
    const bool fine = !SB && op.state_out != nullptr;  // three parts of the weighted v, or two

    const int os = p.H * vd;
    const uint16_t *gq = op.q.p + (int64_t)(h0 / op.q.div) * kd;
    const uint16_t *gk = op.k.p + (int64_t)(h0 / op.k.div) * kd;
    const uint16_t *gv = op.v.p + (int64_t)(h0 / op.v.div) * vd;
    // A thread's unit and row of the loads: 8 lanes take 4 rows of 2 units (the
    // stores to LDS use 32 banks at a time).  The thread number is made opaque
    // wherever they are used, so that they are formed again instead of held in
    // some ten registers across the chunk.
    auto unit_of = [](int t, int U) { return (t >> 3) % (U / 2) * 2 + (t & 1); };
    auto row_of = [](int t, int U) { return (t >> 3) / (U / 2) * 4 + (t >> 1) % 4; };
    auto opaque = [](int t) {
        asm volatile("" : "+v"(t));
        return t;
    };

    u32x4 fq[LOCAL ? 1 : LK], fk[LK], fv[LV];
    auto fetch = [&](int c0) {  // the chunk's rows, lowest token first, into registers
        const int len = min(CT, n - c0);
        const int64_t first = rev ? t0 + n - c0 - len : t0 + c0;
        const auto bk = rows_buffer(gk + first * ks, (uint32_t)((len - 1) * ks + kd) * 2);
        const auto bv = rows_buffer(gv + first * vs, (uint32_t)((len - 1) * vs + HP * vd) * 2);
        const int t = opaque(tid), ck = unit_of(t, UK), rk = row_of(t, UK), cv = unit_of(t, UV), rv = row_of(t, UV);
        const int hv = cv / (VT / 8), vc = v0 + cv % (VT / 8) * 8;  // head and channel of the v unit
        const uint32_t ok = 8 * ck < kd ? (uint32_t)(rk * ks + 8 * ck) * 2 : kNowhere;
        const uint32_t ov = vc < vd ? (uint32_t)(rv * vs + hv * vd + vc) * 2 : kNowhere;
#pragma unroll
        for (int i = 0; i < LK; ++i)
            fk[i] = __builtin_amdgcn_raw_buffer_load_b128(bk, ok + i * RK * (uint32_t)ks * 2, 0, 0);
#pragma unroll
        for (int i = 0; i < LV; ++i)
            fv[i] = __builtin_amdgcn_raw_buffer_load_b128(bv, ov + i * RV * (uint32_t)vs * 2, 0, 0);
        if constexpr (!LOCAL) {
            const auto bq = rows_buffer(gq + first * qs, (uint32_t)((len - 1) * qs + kd) * 2);
            const uint32_t oq = 8 * ck < kd ? (uint32_t)(rk * qs + 8 * ck) * 2 : kNowhere;
#pragma unroll
            for (int i = 0; i < LK; ++i)
                fq[i] = __builtin_amdgcn_raw_buffer_load_b128(bq, oq + i * RK * (uint32_t)qs * 2, 0, 0);
        }
    };
    if (n > 0) fetch(0);

    // in 16-row tile rt of q, scores and outputs, lane l16 is token place0 + row_tile(rt)
    auto row_tile = [](int rt) { return 32 * (rt >> 1) + 4 * (rt & 1); };
    const int place0 = 8 * (l16 >> 2) + (l16 & 3);
    f32x4 O[RT][DT] = {};
    // Stores the outputs of the chunk at c0: a token a tile, channels 8 q4 .. of
    // a pair of tiles (half of them with one tile).  A chunk's outputs leave behind
    // the barriers of the next one, ahead of its loads: waiting for loads then
    // never waits for younger stores.
    auto emit = [&](int c0) {
        const int len = min(CT, n - c0), pad = CT - len;
        const int64_t first = rev ? t0 + n - c0 - len : t0 + c0;
        const int eb = out_f32 ? 4 : 2;
        const auto bo = rows_buffer(static_cast<char *>(op.out) + (first * os + (int64_t)h * vd) * eb,
                                    (uint32_t)((len - 1) * os + vd) * eb);
        const int vc = v0 + 32 * (tile0 >> 1) + 8 * q4 + 4 * (tile0 & 1);
        const int tok0 = rev ? CT - 1 - place0 : place0 - pad;
        const uint32_t at0 = (uint32_t)((tok0 * os + vc) * eb);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int more = row_tile(rt);
            const int tok = rev ? tok0 - more : tok0 + more;
            const uint32_t at = vc < vd && (uint32_t)tok < (uint32_t)len
                                    ? at0 + (uint32_t)((rev ? -more : more) * os * eb)
                                    : kNowhere;
            if constexpr (DT == 2) {
                const f32x4 lo = O[rt][0], hi = O[rt][1];
                if (out_f32) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), bo, at, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), bo, at + 16, 0, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(
                        u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                              pack_bf16x2(hi[2], hi[3])},
                        bo, at, 0, 0);
                }
            } else {
                const f32x4 x = O[rt][0];
                if (out_f32)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), bo, at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b64(
                        u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, bo, at, 0, 0);
            }
        }
    };

    // a lane's places: row l16 of unit q4; row place0; columns of k and v tiles
    const int at_row = q4 * kUnit + l16 * 16;
    const int at_place = q4 * kUnit + place0 * 16;
    const int at_col = (4 * q4 + (l16 >> 2)) * 16 + (l16 & 3) * kUnit;
    const int v_units = (hw * (VT / 8) + 4 * (tile0 >> 1)) * kUnit;
    const float *const w_pair = s_pair[0] + 31 + place0 - 4 * q4;
    const float *const w_lead = s_lead[hw] + CT - 1 - 4 * q4;
    const int scores = hw * kScores;

    // the chunk's v columns, kept for the scores' product
    bf16x8 vcol[CT / 32][DT];
    // out^T += v^T scores^T of the chunk whose scores are complete
    auto add_scores = [&]() {
#pragma unroll
        for (int u = 0; u < CT / 32; ++u)
#pragma unroll
            for (int rt = 2 * u; rt < RT; ++rt) {
                const bf16x8 x = read_unit(s_p, scores + at_place + row_tile(rt) * 16 + 4 * u * kUnit);
#pragma unroll
                for (int d = 0; d < DT; ++d) O[rt][d] = mfma_bf16(vcol[u][d], x, O[rt][d]);
            }
    };

    // Two barriers a chunk: between them lie (A to B) the rows' way into LDS
    // and the scores' product of the chunk before, and (B to A) everything else.
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += CT) {
        const int len = min(CT, n - c0), pad = CT - len;
        // a state of zeros stays one, also where lambda^len is infinite
        const float l2s = !LOCAL && zero && c0 == 0 ? -1e30f : l2;
        __syncthreads();  // A: the previous chunk's rows are read, its scores written
        // token i of the chunk to its place; tokens past it (zeros) wrap to the places before it
        const int ft = opaque(tid), ck = unit_of(ft, UK), rk = row_of(ft, UK), cv = unit_of(ft, UV),
                  rv = row_of(ft, UV);
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const int r = rev ? CT - 1 - (rk + i * RK) : (rk + i * RK + pad) & (CT - 1);
            *reinterpret_cast<u32x4 *>(s_k + ck * kUnit + r * 16) = fk[i];
            if constexpr (!LOCAL) *reinterpret_cast<u32x4 *>(s_q + ck * kUnit + r * 16) = fq[i];
        }
#pragma unroll
        for (int i = 0; i < LV; ++i) {
            const int r = rev ? CT - 1 - (rv + i * RV) : (rv + i * RV + pad) & (CT - 1);
            *reinterpret_cast<u32x4 *>(s_v + cv * kUnit + r * 16) = fv[i];
        }
        if (!LOCAL && c0 > 0) {
            add_scores();
            emit(c0 - CT);
        }
        __syncthreads();  // B
        if (c0 + CT < n) fetch(c0 + CT);

        if constexpr (!LOCAL) {
            // ---- weighted scores, for all heads, in blocks of 16 RB tokens i
            // (lanes) x 32 tokens j (8 a lane): of 64 tokens (rt, c) = (0, 0) (2, 0)
            // (2, 1), of 32 (0, 0) (1, 0)
            constexpr int RB = CT == 64 ? 2 : 1;
            static_assert(NW >= 3, "a wavefront for each block");
#pragma unroll
            for (int m = 0; m < (CT == 64 ? 3 : 2); ++m) {
                if (m != wave) continue;
                const int c = m == 2 ? 1 : 0, rt = RB * (m - c);
                f32x4 a[RB][2] = {};
#pragma unroll
                for (int u = 0; u < KD / 32; ++u) {
                    if (NT > 4 && 32 * u >= kd) break;
                    bf16x8 q[RB];
#pragma unroll
                    for (int i = 0; i < RB; ++i)
                        q[i] = read_unit(s_q, at_place + row_tile(rt + i) * 16 + 4 * u * kUnit);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const bf16x8 k = read_unit(s_k, at_row + (32 * c + 16 * y) * 16 + 4 * u * kUnit);
#pragma unroll
                        for (int i = 0; i < RB; ++i) a[i][y] = mfma_bf16(k, q[i], a[i][y]);
                    }
                }
#pragma unroll
                for (int x = 0; x < HP; ++x)
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = a[i][e / 4][e % 4] *
                                   w_pair[(CT + 32) * x + row_tile(rt + i) - 32 * c - 16 * (e / 4) - e % 4];
                        *reinterpret_cast<bf16x8 *>(s_p + x * kScores + at_place + row_tile(rt + i) * 16 +
                                                    4 * c * kUnit) = pack8(f);
                    }
            }
            // ---- output from the state, out^T = S q^T (channels x tokens)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (NT > 4 && 32 * t >= kd) break;  // a wide launch may hold narrower operations
                bf16x8 a[DT];
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = S[t][e / 4][d][e % 4];
                    a[d] = pack8(f);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const bf16x8 q = read_unit(s_q, at_place + row_tile(rt) * 16 + 4 * t * kUnit);
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        O[rt][d] = mfma_bf16(a[d], q, t == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : O[rt][d]);
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float x = scale_state * fast_exp2(l2s * ((float)(place0 + row_tile(rt) - pad + 1) - shift));
#pragma unroll
                for (int d = 0; d < DT; ++d) O[rt][d] *= x;
            }
        }

        // ---- the state update, 32 tokens at a time
        const float keep = fast_exp2(l2s * (float)len);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (NT > 4 && 32 * t >= kd) break;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                S[t][0][d] *= keep;
                S[t][1][d] *= keep;
            }
        }
#pragma unroll
        for (int u = 0; u < CT / 32; ++u) {
            bf16x8 part3[DT][3];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                vcol[u][d] = read_columns(s_v, at_col + v_units + 8 * ((tile0 + d) & 1) + 32 * u * 16);
                float f[8], r[8];
                unpack8(vcol[u][d], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= w_lead[-32 * u - 16 * (e / 4) - e % 4];
                part3[d][0] = pack8(f);
                unpack8(part3[d][0], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] -= r[e];
                part3[d][1] = pack8(f);
                if (fine) {
                    unpack8(part3[d][1], r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] -= r[e];
                    part3[d][2] = pack8(f);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (NT > 4 && 32 * t >= kd) break;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const bf16x8 k = read_columns(s_k, at_col + 8 * y + 32 * u * 16 + 4 * t * kUnit);
                    if (fine) {
#pragma unroll
                        for (int d = 0; d < DT; ++d) S[t][y][d] = mfma_bf16(k, part3[d][2], S[t][y][d]);
                    }
#pragma unroll
                    for (int d = 0; d < DT; ++d) S[t][y][d] = mfma_bf16(k, part3[d][1], S[t][y][d]);
#pragma unroll
                    for (int d = 0; d < DT; ++d) S[t][y][d] = mfma_bf16(k, part3[d][0], S[t][y][d]);
                }
            }
        }
    }
    if (!LOCAL && n > 0) {
        __syncthreads();
        add_scores();
        emit((n - 1) / CT * CT);
    }

    if constexpr (LOCAL) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < 2; ++y) part[((d * NT + t) * 2 + y) * 64] = S[t][y][d];
    } else {
        if (g.index != g.count - 1 || op.state_out == nullptr) return;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int kc = 32 * t + 8 * q4;
                if (kc >= op.kd || vch(d) >= op.vd) continue;
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = S[t][e / 4][d][e % 4];
                store_state8<SB>(op.state_out, state_at + vch(d) * op.sv + kc, f);
            }
    }
}

// The states of the segments' parts (of `sub` tokens) into the states that
// enter the segments, in place of their first parts': a block takes one head of the
// cut sequence of number c, a thread 4 state elements at a time, in the order of the
// walk's registers.  Sequences of one segment are left to the walk.  With
// `mirror` the states are those of another operation too, transposed (its k
// channels are this one's v channels and the reverse), and are written there
// as well.
template <bool SB>
__global__ __launch_bounds__(256) void la_chain(Params p, int KD, int VT) {
    constexpr int kAhead = 4;
    const int per_head = p.tiles * VT * KD / 4;  // groups of 4
    const int h = blockIdx.x % p.H, c = blockIdx.x / p.H;
    const int which = blockIdx.y;
    const Op &op = p.op[which];
    if (op.twin != 0) return;
    int b, begin, len;
    if (p.batch <= 64) {  // one load: lane l looks at sequence l
        const int lane = threadIdx.x & 63;
        begin = len = 0;
        if (lane < p.batch) {
            begin = clamp_row(p, p.qsl[lane]);
            len = clamp_row(p, p.qsl[lane + 1]) - begin;
        }
        const uint64_t at = __ballot(len > p.seg && cut_number(p, begin, lane) == c);
        if (at == 0) return;
        b = (int)__builtin_ctzll(at);
        begin = __builtin_amdgcn_readlane(begin, b);
        len = __builtin_amdgcn_readlane(len, b);
    } else {
        b = last_up_to(p, c, [&](int i, int first) { return cut_number(p, first, i); });
        if (b < 0) return;
        begin = clamp_row(p, p.qsl[b]);
        len = clamp_row(p, p.qsl[b + 1]) - begin;
        if (len <= p.seg || cut_number(p, begin, b) != c) return;
    }
    const int count = (len + p.seg - 1) / p.seg, parts = p.seg / p.sub;  // segments, and parts of one
    const int last = (count - 1) * parts;
    const int64_t slot = p.cache_idx != nullptr ? (int64_t)p.cache_idx[b] : (int64_t)b;
    if (slot >= p.max_slots) return;
    for (int i = blockIdx.z * 256 + (int)threadIdx.x; i < per_head; i += gridDim.z * 256) {
        const int lane = i & 63, y = (i >> 6) & 1, t = (i >> 7) % (KD / 32), tile = (i >> 7) / (KD / 32);
        const int vch = 32 * (tile >> 1) + column(lane & 15, tile & 1);
        const int kc = 32 * t + 8 * (lane >> 4) + 4 * y;
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
        const float keep = fast_exp2(log2_decay(p, h) * (float)p.sub);
        const int64_t step = (int64_t)p.H * per_head;
        const int64_t head = first_slot(p, begin, b) * step + (int64_t)h * per_head;
        f32x4 *part = reinterpret_cast<f32x4 *>(p.parts) + (int64_t)which * p.sub_slots * step + head + i;
        // (v channel kc, k channel vch) of the mirror: element vch % 4 of the group of its
        // lane (a backward launch holds as many v channels as k channels)
        const bool mirrored = op.mirror != 0;
        const int mtile = kc / 32 * 2 + (kc >> 2) % 2, mt = vch / 32, my = (vch >> 2) % 2;
        const int mlane = vch % 32 / 8 * 16 + kc % 32 / 8 * 4;
        float *twin = p.parts + 4 * ((int64_t)op.mirror * p.sub_slots * step + head +
                                     ((mtile * (KD / 32) + mt) * 2 + my) * 64 + mlane) + vch % 4;
        int rest = 0;  // parts until the next segment starts
        for (int s = 0; s <= last; s += kAhead) {
            f32x4 own[kAhead];  // loaded ahead of the chain
#pragma unroll
            for (int a = 0; a < kAhead; ++a) own[a] = in && s + a < last ? part[a * step] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (s + a <= last && rest == 0) {
                    part[a * step] = S;
                    if (mirrored) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) twin[4 * (a * step + e)] = S[e];
                    }
                }
                rest = rest == 0 ? parts - 1 : rest - 1;
                S = S * keep + own[a];
            }
            part += kAhead * step;
            twin += 4 * kAhead * step;
        }
    }
}

// One thread per 8 channels of a (token, group); the sequences' rows only.
__global__ __launch_bounds__(256) void la_group_sum(GroupSum a, const int32_t *qsl, int batch, int64_t n8, int G,
                                                    int div, int w8) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const int64_t tg = i / w8, t = tg / G;
    if (t < qsl[0] || t >= qsl[batch]) return;
    const int c = (int)(i - tg * w8) * 8;
    const float *src = a.src[blockIdx.y];
    float s[8] = {};
    for (int d = 0; d < div; ++d) {
        float f[8];
        load_state8<false>(src, (tg * div + d) * (int64_t)w8 * 8 + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += f[e];
    }
    store_state8<true>(a.dst[blockIdx.y], i * 8, s);
}

template <int KD, int CT, int NW, int DT, int HP, bool SB>
hipError_t launch_variant(const Params &p, hipStream_t s) {
    constexpr int VT = 16 * DT * NW / HP;
    const int64_t each = (int64_t)(p.H / HP) * p.tiles * p.nops, run = (int64_t)8 * (p.share / HP) * p.tiles * p.nops;
    auto grid = [&](int slots) { return dim3((unsigned)((slots * each + run - 1) / run * run)); };
    const dim3 block(64 * NW);
    if (p.seg != 0) {
        la_walk<KD, CT, NW, DT, HP, SB, true><<<grid(p.batch <= 64 ? p.sub_slots - p.cuts : p.sub_slots), block, 0, s>>>(p);
        // blocks for the card, or one for each head
        const int64_t heads = (int64_t)p.cuts * p.H;
        const int most = p.tiles * VT * KD / 1024, split = (int)std::min<int64_t>(most, (4096 + heads - 1) / heads);
        const dim3 cg((unsigned)heads, (unsigned)p.nops, (unsigned)split);
        la_chain<SB><<<cg, dim3(256), 0, s>>>(p, KD, VT);
    }
    la_walk<KD, CT, NW, DT, HP, SB, false><<<grid(p.slots), block, 0, s>>>(p);
    return hipGetLastError();
}
template <int KD, bool SB>
hipError_t launch_kd(const Params &p, const Shape &h, hipStream_t s) {
    if (h.vt == 128) return launch_variant<KD, 64, 4, 2, 1, SB>(p, s);
    if (h.heads == 2) return launch_variant<KD, 64, 4, 2, 2, SB>(p, s);
    return launch_variant<KD, 64, 4, 1, 1, SB>(p, s);
}
template <bool SB>
hipError_t launch_any(const Params &p, const Shape &h, hipStream_t s) {
    if (h.kd == 64) return launch_kd<64, SB>(p, h, s);
    if (h.kd == 128) return launch_kd<128, SB>(p, h, s);
    if (h.vt == 128) return launch_variant<256, 64, 8, 1, 1, SB>(p, s);
    return launch_variant<256, 32, 4, 1, 1, SB>(p, s);
}
}  // namespace

// A walk is a chain of chunks, so a launch needs many walks side by side: the
// card holds kAtOnce workgroups (two on each of 256 compute units, one or three
// with wide keys).  Sequences are cut into segments of as many tokens as let their
// number, T / seg and half a segment for each sequence's end, fill the card
// once; cut sequences cost a pass over their k and v for the segments' states,
// so more of them only cost (65536 tokens of 16 heads: kAtOnce 512 391 us, 768
// 424, 1024 421).  Where the sequences alone fill it, only those of more than
// twice a workgroup's share of the tokens are cut, which would end alone (32
// ragged prompts of 128 heads, longest 7975 tokens: 531 us, from one share on
// 547, from half a share 667).
// A segment shorter than the mean sequence is made to divide it.
Shape shape_of(int64_t T, int batch, int H, int share, int kd, const int *vds, int nops, int nlocal) {
    constexpr int64_t kLeast = 128;
    const int vd = *std::max_element(vds, vds + nops);
    Shape h;
    h.kd = kd <= 64 ? 64 : kd <= 128 ? 128 : 256;
    const int64_t mean = (T + batch - 1) / batch;
    // Wide keys: one workgroup of 8 wavefronts and 128 value channels fills a
    // compute unit's LDS; where sequences are short, and their states most of the
    // traffic, three with 64 channels and chunks of 32 tokens move them faster.
    // The border depends on the widths too (us with 64 / 128 channels for everything):
    //   mean length                        27        66       ~200  265-282   ~1100
    //   96 x 200, 12 heads, backward  1319/1371   809/761   562/487  564/455  484/392
    //   256 x 256, 12 heads, backward 1911/2693 1134/1423   754/857  704/779  598/618
    //   192 x 128, 4 heads, backward   136/227    96/128     66/92    69/92
    //   200 x 128, 12 heads, prompts   468/609   262/301    170/190  171/176  200/173
    // 256 tokens lose up to 15% below it (96 x 200) and a third above it (192 x 128).
    h.vt = vd <= 64 || (h.kd == 256 && mean <= 256) ? 64 : 128;
    h.heads = h.vt == 64 && h.kd < 256 && share % 2 == 0 && nops == 1 ? 2 : 1;
    const int64_t kAtOnce = h.kd < 256 ? 512 : h.vt == 64 ? 768 : 256;
    auto tiles = [&](int n) {
        int sum = 0;
        for (int i = 0; i < n; ++i) sum += (vds[i] + h.vt - 1) / h.vt;
        return (int64_t)(H / h.heads) * sum;
    };
    // with states handed on transposed (la_chain), as many v channels as k channels
    h.tiles = (nlocal < nops ? h.kd : vd) / h.vt + ((nlocal < nops ? 0 : vd) % h.vt != 0);
    const int64_t walks = tiles(nops);  // workgroups of a token
    const int64_t room = kAtOnce - batch * walks / 2;
    int64_t seg = 2 * T * walks / kAtOnce;
    if (room > 0) seg = std::min(seg, T * walks / room);
    seg = std::max(seg, kLeast);
    if (seg < mean) {
        const int64_t n = (mean + seg / 2) / seg;
        seg = (mean + n - 1) / n;
    }
    seg = std::max((seg + kTok - 1) / kTok * kTok, kLeast);
    // parts: the pass for the states has no output to wait for and walks fewer
    // segments (none of them the last), so it may be cut finer
    const int64_t local = tiles(nlocal) * std::max<int64_t>(T / seg - batch / 2, 1);
    const int64_t parts = std::max<int64_t>(1, std::min((kAtOnce + local - 1) / local, seg / kLeast));
    const int64_t sub = (seg + parts * kTok - 1) / (parts * kTok) * kTok;
    seg = sub * parts;
    // (512 tokens: the longest walk that takes no longer than the two more launches)
    const bool cut = T > std::max<int64_t>(seg, 512);
    h.seg = cut ? (int)seg : 0;
    h.sub = cut ? (int)sub : 0;
    h.slots = cut ? (int)(T / seg) + batch : batch;
    h.cuts = cut ? (int)std::min<int64_t>(batch, T / (seg + 1)) : 0;
    h.sub_slots = cut ? (int)(T / sub) + h.cuts : 0;
    h.bytes = (size_t)nops * h.sub_slots * H * h.tiles * h.vt * h.kd * sizeof(float);
    // (in whole runs of the workgroups that share rows, on 8 XCDs)
    const int64_t each = (int64_t)(H / h.heads) * h.tiles * nops, run = (int64_t)8 * (share / h.heads) * h.tiles * nops;
    const int64_t blocks = (std::max(h.slots, h.sub_slots) * each + run - 1) / run * run;
    h.threads = std::max(blocks * (h.kd == 256 && h.vt == 128 ? 512 : 256), (int64_t)h.cuts * H * 256);
    return h;
}

hipError_t launch_walk(Params &p, const Shape &h, int nops, hipStream_t s) {
    p.nops = nops;
    p.tiles = h.tiles;
    p.seg = h.seg;
    p.sub = h.sub;
    p.slots = h.slots;
    p.sub_slots = h.sub_slots;
    p.cuts = h.cuts;
    return p.state_bf16 ? launch_any<true>(p, h, s) : launch_any<false>(p, h, s);
}

hipError_t launch_group_sum(const GroupSum &a, const Params &p, int div, int width, hipStream_t s) {
    const int G = p.H / div;
    const int64_t n8 = p.T * G * (width / 8);
    la_group_sum<<<dim3((unsigned)((n8 + 255) / 256), 2), dim3(256), 0, s>>>(a, p.qsl, p.batch, n8, G, div, width / 8);
    return hipGetLastError();
}

}  // namespace la
}  // namespace ssd
