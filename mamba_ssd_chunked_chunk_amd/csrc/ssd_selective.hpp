// What the kernels of the selective scan share.
#pragma once

#include "ssd_layer.hpp"

namespace ssd {
namespace layer {

constexpr int kTile = 16;  // tokens between two hand-overs of a walk

// What a workgroup works on.
struct Span {
    int g, c0, ch0;  // group, first channel in it and in all
    int nch;         // channels, up to 64
};
__device__ __forceinline__ Span span_of(const ScanParams &p, int block) {
    const int per = p.blocks / p.G;
    Span w;
    w.g = block / per;
    w.c0 = (block % per) * 64;
    w.ch0 = w.g * p.Dg + w.c0;
    w.nch = min(64, p.Dg - w.c0);
    return w;
}

__device__ __forceinline__ void widen4(const u32x2 &v, float (&o)[4]) {
    o[0] = bf16x2_lo(v[0]);
    o[1] = bf16x2_hi(v[0]);
    o[2] = bf16x2_lo(v[1]);
    o[3] = bf16x2_hi(v[1]);
}

// softplus without a branch or a division: with z = e^-|v| and u = 1 + z
// rounded, log1p(z) = log(u) + (z - (u - 1)) / u but for terms of the second
// order, and the quotient by u in [1, 2] moves the last summand, at most half a
// unit of u's last place, by less than 2^-24 z.
__device__ __forceinline__ float softplus_fast(float v) {
    const float z = fast_exp2(-fabsf(v) * kLog2e);  // in (0, 1]
    const float u = 1.f + z;
    const float l = __builtin_fmaf(__builtin_amdgcn_logf(u), kLn2, z - (u - 1.f));
    return __builtin_amdgcn_fmed3f(v, 0.f, __builtin_inff()) + l;
}
__device__ __forceinline__ float time_step(const ScanParams &p, float raw) {
    return p.softplus ? softplus_fast(raw) : raw;
}

// First place of a cut sequence's segments among those of all cut sequences: at
// most begin / (cut + 1) of them lie ahead of it, each with at most one partial
// segment.
__device__ __forceinline__ int64_t cut_place(const ScanParams &p, const Seq &q) {
    return q.begin / p.seg + min(q.b, q.begin / (p.cut + 1));
}

// What a workgroup works on: segment s of nseg of a sequence, and the number
// that no other segment of any sequence has.
struct Piece {
    Seq q;
    int s, nseg, number;
};
__device__ __forceinline__ int segments_of(const ScanParams &p, int len) {
    return len > p.cut ? (len + p.seg - 1) / p.seg : 1;
}

// The piece at a place of the grid; false where there is none.  With CUT, of the
// places of cut sequences alone.
//
// Sequences are numbered one behind the other, 64 of them at a time, a sequence a
// lane: whole ones in classes of their length, the longest first, and the segments
// of cut ones in the middle, where their length belongs.  Gaps between them would
// leave whole rows of compute units without work, as they come in step with the
// units that the workgroups are given to (states of 8 x 2048 tokens 430 -> 350 us),
// and a long one at the end all but one (backward pass of 65 ragged prompts of 186
// tokens on average 632 -> 436 us).  Where that is not worth the search (`listed`)
// they have the places of find_piece and cut_place, with gaps.
constexpr int kClasses = 14;
template <bool CUT>
__device__ __forceinline__ bool piece_at(const ScanParams &p, int place, Piece &w) {
    const int lane = threadIdx.x & 63;
    if (p.batch == 1) {  // (300 tokens, with and without the search, 27.4 and 25.0 us)
        w.q = seq_at(p.qsl, 0, p.T);
        w.nseg = segments_of(p, w.q.len);
        w.s = w.number = place;
        return place < w.nseg && !(CUT && w.nseg == 1);
    }
    if (p.listed) {
        struct Lane {
            int begin, len, n, cls;  // n: pieces, 0 behind the last sequence; cls: of a whole one, else -1
        };
        const float per_class = (float)kClasses / ((float)p.cut + 1.f);
        auto lane_of = [&](int j) {
            Lane v{0, 0, 0, -1};
            const int b = j * 64 + lane;
            if (b >= p.batch) return v;
            v.begin = clamp_row(p.qsl[b], p.T);
            const int end = clamp_row(p.qsl[b + 1], p.T);
            v.len = end > v.begin ? end - v.begin : 0;
            v.n = segments_of(p, v.len);
            if (v.n == 1) v.cls = min((int)((float)(p.cut - v.len) * per_class), kClasses - 1);
            return v;
        };
        constexpr int kLong = kClasses / 2;  // classes of more than a segment's length
        const int chunks = (p.batch + 63) / 64;
        Lane v;
        int cut = 0, longer = 0, whole[kClasses] = {};  // segments, long sequences, sequences of each class
        for (int j = 0; j < chunks; ++j) {
            v = lane_of(j);
            if (__ballot(v.n > 1) != 0) cut += __builtin_amdgcn_readlane(wave_incl_scan(v.n > 1 ? v.n : 0), 63);
            longer += __builtin_popcountll(__ballot(v.cls >= 0 && v.cls < kLong));
            if (!CUT)
#pragma unroll
                for (int c = 0; c < kClasses; ++c) whole[c] += __builtin_popcountll(__ballot(v.cls == c));
        }
        w.number = CUT ? place + longer : place;
        if (w.number >= p.places) return false;  // (where a wrong table lets sequences overlap)
        const bool among_cut = w.number >= longer && w.number < longer + cut;
        if (CUT && !among_cut) return false;
        int rest = w.number, cls = -1;
        if (among_cut) {
            rest -= longer;
        } else {
            rest -= rest < longer ? 0 : cut;
#pragma unroll
            for (int c = 0; c < kClasses; ++c) {
                if (cls < 0 && rest < whole[c]) cls = c;
                if (cls < 0) rest -= whole[c];
            }
            if (cls < 0) return false;
        }
        for (int j = 0; j < chunks; ++j) {
            if (chunks > 1) v = lane_of(j);
            // pieces of this chunk's lanes, and those ahead of each
            int all, ahead;
            const bool some = among_cut ? v.n > 1 : v.cls == cls;
            if (among_cut) {
                const int upto = wave_incl_scan(some ? v.n : 0);
                all = __builtin_amdgcn_readlane(upto, 63);
                ahead = upto - v.n;
            } else {
                const uint64_t m = __ballot(some);
                all = __builtin_popcountll(m);
                ahead = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
            }
            if (rest < all) {
                const int at = __builtin_ctzll(__ballot(some && ahead <= rest && rest < ahead + v.n));
                w.q = Seq{j * 64 + at, __builtin_amdgcn_readlane(v.begin, at), __builtin_amdgcn_readlane(v.len, at)};
                w.nseg = __builtin_amdgcn_readlane(v.n, at);
                w.s = rest - __builtin_amdgcn_readlane(ahead, at);
                return true;
            }
            rest -= all;
        }
        return false;
    }
    if (!CUT) {
        const bool found = find_piece(p.qsl, p.batch, p.T, p.seg, place, w.q, w.s);
        w.nseg = segments_of(p, w.q.len);
        w.number = place;
        return found && w.s < w.nseg;
    }
    // (places of cut sequences never meet, so the owner is the last sequence whose first place is not behind this one)
    int lo = 0, hi = p.batch - 1;
    while (hi > lo) {
        const int step = (hi - lo + 63) / 64;
        const int b = lo + (lane + 1) * step;
        bool ahead = b <= hi;
        if (ahead) {
            const int begin = clamp_row(p.qsl[b], p.T);
            ahead = begin / p.seg + min(b, begin / (p.cut + 1)) <= place;
        }
        const uint64_t m = __ballot(ahead);
        const int k = ~m == 0 ? 64 : __builtin_ctzll(~m);
        lo += k * step;
        hi = hi < lo + step - 1 ? hi : lo + step - 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    w.q = seq_at(p.qsl, lo, p.T);
    w.nseg = segments_of(p, w.q.len);
    w.s = place - (int)cut_place(p, w.q);
    w.number = w.q.begin / p.seg + w.q.b + w.s;
    return w.nseg > 1 && w.s >= 0 && w.s < w.nseg;
}

// The state that enters segment s > 0 from the states that the segments ahead
// of it leave (all but the first from zero).  A: times log2(e).
__device__ __forceinline__ void chain_states(const ScanParams &p, int64_t first, int s, int64_t at, int ch,
                                             const float (&A)[4], float (&h)[4]) {
    const float *part = p.parts + first * p.D * p.N + at;
    const float *steps = p.steps + first * p.D + ch;
    const int64_t row = (int64_t)p.D * p.N;
#pragma unroll 4
    for (int j = 0; j < s; ++j) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(part + j * row);
        const float d = steps[(int64_t)j * p.D];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = j == 0 ? v[i] : __builtin_fmaf(fast_exp2(d * A[i]), h[i], v[i]);
    }
}

// Where the state ahead of token t (a multiple of kGradTile) of a sequence is
// kept for the backward pass, 4 states of a channel together.
__device__ __forceinline__ float *mark_at(const ScanParams &p, const Seq &q, int t, int n0, int ch) {
    const int64_t tile = q.begin / kGradTile + q.b + t / kGradTile;
    return p.marks + ((tile * (p.N / 4) + n0 / 4) * p.D + ch) * 4;
}

// wavefronts that hold N states, 4 each
inline int waves_of(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
template <typename F>
void by_waves(int n, F f) {
    switch (n) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return f(std::integral_constant<int, 16>{});
    }
}

int grad_waves_of(int N);  // and in the backward pass
hipError_t launch_scan_marks(const ScanParams &p, hipStream_t s);

}  // namespace layer
}  // namespace ssd
