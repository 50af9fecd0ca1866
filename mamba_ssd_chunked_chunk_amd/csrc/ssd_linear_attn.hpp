// Shared definitions of the linear-attention kernels (fixed decay per head).
#pragma once

#include "ssd_common.hpp"

namespace ssd {
namespace la {

constexpr int kTok = 64;  // tokens of a chunk

// A [total_len, n, width] bf16 tensor as the kernels read it: `stride`
// elements between tokens, and head h reads row h / div of the n.
struct Rows {
    const uint16_t *p;
    int64_t stride;
    int div;
};

// One recurrence over the tokens of each sequence, forward or in reverse:
//     S = lambda S + c v_t k_t^T        out_t = S q_t
// with kd channels of k and q, vd channels of v and out.  The forward
// operation is one of these and its backward pass is three of them with the
// roles exchanged:
//     o:  (q, k, v)     dq: (d_o, v, k)
//     dk: (v, d_o, q) and dv: (k, q, d_o), in reverse
// Reversed, the state enters the first (the last of the sequence) token
// undecayed and leaves decayed once more: exponents shift by one.
struct Op {
    Rows q, k, v;
    void *out;           // [T][H][vd]: bf16, or fp32 where heads are summed afterwards
    int out_f32;
    int kd, vd;
    int reverse;
    float scale_pair;    // on q . k within a chunk
    float scale_state;   // on out from the state that enters the chunk
    float scale_update;  // on v k^T as it enters the state
    // state element (v channel i, k channel j) of slot s, head h at
    // ((s H + h) state_size + i sv + j sk); null in: zero, null out: dropped (sk
    // is 1 where there is an out)
    const void *state_in;
    void *state_out;
    int64_t sv, sk;
    // dk and dv walk with the same states, transposed: the segments' are made
    // for `dv` alone (mirror: the other's number), and handed to dk (twin: 1)
    int mirror, twin;
};

constexpr int kMaxOps = 3;

struct Params {
    Op op[kMaxOps];
    int64_t T;
    int batch, H;
    int share;            // heads of a group
    int state_size;       // V * K
    int state_bf16;
    const float *log_decay;
    const int32_t *qsl;
    const uint8_t *has_init;    // null: see init_all
    const uint32_t *cache_idx;  // null: slot b
    int init_all;
    uint32_t max_slots;
    // the launch (set by launch_walk)
    int nops, tiles;  // tiles: workgroups along the value channels
    int seg, slots;   // tokens of a segment (0: whole sequences) and slots of segments
    int sub, sub_slots;  // the same of the parts of segments (seg is a multiple of sub), of cut sequences alone
    int cuts;         // most sequences of more than a segment
    float *parts;     // [nops][sub_slots][H][tiles * VT][KD] states of the parts, in register order
};

// What a launch takes of kd x vd channels (the largest of its operations').
struct Shape {
    int kd, vt, tiles;  // kd rounded up; value channels of a workgroup, and workgroups along vd
    int heads;          // heads of a workgroup
    int seg, slots, sub, sub_slots, cuts;
    size_t bytes;       // of `parts`
    int64_t threads;    // of its largest grid, which 32 bits have to hold
};
// vds: the value channels of its nops operations, of which the first nlocal have segments' states of their own
Shape shape_of(int64_t T, int batch, int H, int share, int kd, const int *vds, int nops, int nlocal);
hipError_t launch_walk(Params &p, const Shape &h, int nops, hipStream_t s);

// sums the heads of each group, twice: dst[t][g][w] = sum_i src[t][g * div + i][w]
struct GroupSum {
    const float *src[2];
    uint16_t *dst[2];
};
hipError_t launch_group_sum(const GroupSum &a, const Params &p, int div, int width, hipStream_t s);

struct StepParams {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;
    uint16_t *o;
    const float *log_decay;
    void *pool;
    const uint8_t *has_init;
    const uint32_t *cache_idx;
    int batch, H, div, K, V;
    uint32_t max_slots;
    int state_bf16;
    float scale;
};
hipError_t launch_step(const StepParams &p, hipStream_t s);

}  // namespace la

struct CacheParams {
    const uint32_t *pool_idx, *entry_idx;
    int64_t rows_per_slot;  // H * P
    int count, N;
    uint32_t max_slots, max_entries;
};
// threads of the larger of the two launches, which 32 bits have to hold
int64_t state_cache_threads(const CacheParams &c, bool bf16);
hipError_t launch_state_quantize(const CacheParams &c, const void *pool, bool bf16, bool e4m3, void *codes,
                                 float *scales, hipStream_t s);
hipError_t launch_state_dequantize(const CacheParams &c, void *pool, bool bf16, bool e4m3, const void *codes,
                                   const float *scales, hipStream_t s);
}  // namespace ssd
