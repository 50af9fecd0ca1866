// Shared definitions of the operators around and beside the scan: the norm,
// the short convolution and the selective scan.
#pragma once

#include <type_traits>

#include "ssd_common.hpp"

namespace ssd {
namespace layer {

// ---------------------------------------------------------------- pieces

// 8 consecutive bf16 as floats, and back (16 bytes)
__device__ __forceinline__ void widen8(const u32x4 &v, float (&o)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        o[2 * k] = bf16x2_lo(v[k]);
        o[2 * k + 1] = bf16x2_hi(v[k]);
    }
}
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// 1 / (1 + e^-x) with the hardware's exponential and reciprocal: 0 and 1 at the
// ends of the range.
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * x));
}

// sums over a wavefront, in every lane
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add_all<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_add_all<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_add_all<0x141>(v);  // row_half_mirror
    v = dpp_add_all<0x140>(v);  // row_mirror
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    return v;
}

// Adds to a pointer that is the same in all lanes.
template <typename T>
__device__ __forceinline__ T *moved(T *base, int64_t bytes) {
    typedef std::conditional_t<std::is_const<T>::value, const char, char> Byte;
    return reinterpret_cast<T *>(reinterpret_cast<Byte *>(base) + bytes);
}
// Such a pointer into global memory that stays in scalar registers: a loop that
// adds to it and to a lane's offset would else be turned into one that adds to
// 64 lanes' sums.  (hold() where all lanes are, at() and put() anywhere.)
template <typename T>
struct Scalar {
    __attribute__((address_space(1))) T *ptr;
    __device__ explicit Scalar(T *p) : ptr((__attribute__((address_space(1))) T *)p) {}
    __device__ __forceinline__ void hold() { asm volatile("" : "+s"(ptr)); }
    template <typename V>
    __device__ __forceinline__ V at(uint32_t bytes) const {
        typedef __attribute__((address_space(1))) const char *Bytes;
        return *reinterpret_cast<const __attribute__((address_space(1))) V *>(reinterpret_cast<Bytes>(ptr) + bytes);
    }
    template <typename V>
    __device__ __forceinline__ void put(uint32_t bytes, const V &v) const {
        typedef __attribute__((address_space(1))) char *Bytes;
        *reinterpret_cast<__attribute__((address_space(1))) V *>(reinterpret_cast<Bytes>(ptr) + bytes) = v;
    }
    // the same past the caches
    template <typename V>
    __device__ __forceinline__ void put_past(uint32_t bytes, const V &v) const {
        typedef __attribute__((address_space(1))) char *Bytes;
        __builtin_nontemporal_store(
            v, reinterpret_cast<__attribute__((address_space(1))) V *>(reinterpret_cast<Bytes>(ptr) + bytes));
    }
};
// ... and reads or writes at a lane's own offset from it, in bytes.
template <typename V, typename T>
__device__ __forceinline__ V at_offset(const T *base, uint32_t bytes) {
    return *reinterpret_cast<const V *>(reinterpret_cast<const char *>(base) + bytes);
}
template <typename V, typename T>
__device__ __forceinline__ void put_offset(T *base, uint32_t bytes, const V &v) {
    *reinterpret_cast<V *>(reinterpret_cast<char *>(base) + bytes) = v;
}

// ---------------------------------------------------------------- ragged batches

// Where a sequence lies, the same in all lanes: rows begin .. begin + len - 1.  Boundaries are clamped
// to 0 .. T, so a wrong table never leads outside the tensors.
struct Seq {
    int b, begin, len;
};
__device__ __forceinline__ int clamp_row(int v, int T) { return v < 0 ? 0 : v > T ? T : v; }
__device__ __forceinline__ Seq seq_at(const int32_t *qsl, int b, int T) {
    const int begin = __builtin_amdgcn_readfirstlane(clamp_row(qsl[b], T));
    const int end = __builtin_amdgcn_readfirstlane(clamp_row(qsl[b + 1], T));
    return Seq{b, begin, end > begin ? end - begin : 0};
}

// Sequences are cut into pieces of `piece` tokens.  Piece s of sequence b has
// the place begin / piece + b + s: begin / piece bounds the whole pieces ahead
// and b the partial ones, so places never meet, and T / piece + batch of them
// hold all (some stay empty).  Finds the sequence and the piece of a place;
// false where it is empty (a sequence without tokens has one piece, 0).  All
// lanes of a wavefront search together, 64 boundaries at a time.
__device__ __forceinline__ bool find_piece(const int32_t *qsl, int batch, int T, int piece, int place, Seq &seq,
                                           int &s) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = batch - 1;  // the last b with begin / piece + b <= place
    while (hi > lo) {
        const int step = (hi - lo + 63) / 64;
        const int b = lo + (lane + 1) * step;
        const bool ahead = b <= hi && clamp_row(qsl[b], T) / piece + b <= place;
        const uint64_t m = __ballot(ahead);
        const int k = ~m == 0 ? 64 : __builtin_ctzll(~m);
        lo += k * step;
        hi = hi < lo + step - 1 ? hi : lo + step - 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    seq = seq_at(qsl, lo, T);
    s = place - (seq.begin / piece + lo);
    return s >= 0 && (s == 0 || (int64_t)s * piece < seq.len);
}

// ---------------------------------------------------------------- norm

struct NormParams {
    int64_t rows, xs;
    int width;
    float eps;
    int res_bf16, out;  // out: SSD_OUT_BF16, SSD_CODE_I8 or SSD_CODE_E4M3
    void *y;
    float *scales;
    void *res_out;
    const uint16_t *x;
    const void *res;
    const float *weight;
};
// threads of the launch, which 32 bits have to hold
int64_t norm_threads(int64_t rows, int width);
hipError_t launch_norm(const NormParams &p, hipStream_t s);

struct NormGradParams {
    int64_t rows;
    int width;
    float eps;
    int res_bf16;
    uint16_t *dx;
    void *d_res;
    const void *r;
    const float *weight;
    const uint16_t *dy;
    const void *d_r;
    float *part;  // [parts][width]
    float *dweight;
    int parts;
};
int norm_grad_parts(int64_t rows, int width);
hipError_t launch_norm_grad(const NormGradParams &p, hipStream_t s);

// out[j] = sum over i < n of part[i * stride + j], j < width (a multiple of 4,
// as is the stride), or nothing where out is null.
struct Sum {
    const float *part;
    int n;
    int64_t stride, width;
    float *out;
};
struct Sums {
    Sum s[3];
};
constexpr int kSumThreads = 256;
// Blocks of COLS columns each
template <int COLS>
inline __host__ __device__ int64_t sum_blocks(const Sum &s) {
    return s.out == nullptr ? 0 : (s.width + COLS - 1) / COLS;
}
template <int COLS>
inline __host__ int64_t sum_blocks(const Sums &a) {
    return sum_blocks<COLS>(a.s[0]) + sum_blocks<COLS>(a.s[1]) + sum_blocks<COLS>(a.s[2]);
}
// The block-th of them, a thread 4 columns of every kSumThreads 4 / COLS-th part.
// (Many parts of few columns want narrow blocks, 1024 of 2560 columns 6.4 us with
// 32, 8.4 with 64; few of many do not, beside the sums of the scan's backward
// pass 39 us and 33.)
template <int COLS>
__device__ __forceinline__ void add_parts(const Sums &all, int64_t block) {
    constexpr int kRows = kSumThreads * 4 / COLS, kAtOnce = 8;
    __shared__ f32x4 buf[kRows][COLS / 4];
    int k = 0;
    while (k < 2 && block >= sum_blocks<COLS>(all.s[k])) block -= sum_blocks<COLS>(all.s[k++]);
    const Sum &a = all.s[k];
    const int col = threadIdx.x % (COLS / 4), first = threadIdx.x / (COLS / 4);
    const int64_t j = block * COLS + col * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (j < a.width)
        for (int i = first; i < a.n; i += kAtOnce * kRows) {
            f32x4 v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (i + u * kRows < a.n)
                    v[u] = *reinterpret_cast<const f32x4 *>(a.part + (i + u * kRows) * a.stride + j);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) s += v[u];
        }
    buf[first][col] = s;
    __syncthreads();
    if (first == 0 && j < a.width) {
#pragma unroll
        for (int i = 1; i < kRows; ++i) s += buf[i][col];
        *reinterpret_cast<f32x4 *>(a.out + j) = s;
    }
}
hipError_t launch_sums(const Sums &sums, hipStream_t s);

// ---------------------------------------------------------------- convolution

struct ConvParams {
    int T, batch, D;
    int64_t xs;
    int silu;
    uint16_t *y;
    const uint16_t *x;
    const float *weight, *bias;
    const uint16_t *state_in;
    uint16_t *state_out;
    const int32_t *qsl;
    const uint8_t *has_init;
    const uint32_t *cache_idx;
    int init_all;
    uint32_t max_slots;
    // backward
    const uint16_t *dy, *d_final;
    uint16_t *dx, *d_init;
    float *part;  // [parts][width + 1][D]
    float *dweight, *dbias;
    int tile;        // tokens of a piece
    int64_t places;  // of pieces
};
// Tokens of a piece and places, of either direction
void conv_shape(ConvParams &p, int width, bool backward);
int64_t conv_parts(const ConvParams &p);
int64_t conv_threads(const ConvParams &p);
hipError_t launch_conv(const ConvParams &p, int width, hipStream_t s);
hipError_t launch_conv_step(const ConvParams &p, int width, hipStream_t s);
hipError_t launch_conv_grad(const ConvParams &p, int width, hipStream_t s);

// ---------------------------------------------------------------- selective scan

struct ScanParams {
    int T, batch, D, G, N, Dg;  // Dg: channels of a group
    int blocks;                 // of 64 channels: G times those of a group
    int64_t xs, dts, zs, bs, cs;
    int softplus;
    uint16_t *y;
    const uint16_t *x, *dt, *z, *B, *C;
    const float *A, *Dskip, *bias;
    const void *state_in;
    void *state_out;
    int state_bf16;
    const int32_t *qsl;
    const uint8_t *has_init;
    const uint32_t *cache_idx;
    int init_all;
    uint32_t max_slots;
    // sequences of more than `cut` tokens are cut into segments of `seg`
    int seg, cut;
    int listed;      // sequences are numbered without gaps
    int64_t places;  // of segments
    int64_t cut_places, cuts;  // of segments of cut sequences; most of those sequences
    float *parts;    // [cut_places][D][N]: the states that segments leave, from zero but the first
    float *steps;    // [cut_places][D]: sums of their time steps
    // backward
    const uint16_t *dy;
    const void *d_final;
    uint16_t *dx, *ddt, *dz, *dB, *dC;
    void *d_init;
    float *dA, *dD, *dbias;
    float *adj;      // [cut_places][D][N]: the same of the gradient, backwards, from zero but the last
    float *marks;    // [tiles][N / 4][D][4]: the state ahead of each tile of kGradTile tokens
    float *bc;       // [blocks][T][2][N]: dC and dB of 64 channels
    float *dA_part, *dD_part;  // [places][D][N], [places][2][D]
};
constexpr int kGradTile = 8;
void scan_shape(ScanParams &p, bool backward);
int64_t scan_threads(const ScanParams &p, bool backward);
hipError_t launch_scan(const ScanParams &p, hipStream_t s);
hipError_t launch_scan_grad(const ScanParams &p, hipStream_t s);
hipError_t launch_scan_step(const ScanParams &p, hipStream_t s);

}  // namespace layer
}  // namespace ssd
