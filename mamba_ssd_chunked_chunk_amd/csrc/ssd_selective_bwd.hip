// Backward pass of the selective scan.  With a = exp(dts A), e = dy silu(z) and U
// the gradient of the state,
//     U_t = C_t e_t + a_{t+1} U_{t+1}
// runs against the tokens and needs every token's state, so a forward walk
// first leaves the state ahead of each tile of 8 tokens, and the backward walk
// goes from tile to tile, makes its 8 states again (and keeps them and their
// decays in registers) and then turns round.  As in the forward pass a
// workgroup takes 64 channels, a wavefront 4 states of them, a channel a lane;
// sums over states go through LDS.  Sums over channels (dB and dC) are formed
// by exchanging halves: 64 values a lane, of 8 tokens, 4 states and the two
// gradients, become one a lane in 6 steps, each of which adds what two lanes
// hold of half the values.  They leave as fp32 for each 64 channels, and a last
// kernel adds the blocks of a group, in their order.
#include "ssd_selective.hpp"

namespace ssd {
namespace layer {
namespace {

// One step of the exchange: lanes whose bit is clear keep a and get their
// partner's a, the others b.
__device__ __forceinline__ float fold32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the partner by a DPP pattern, which flips the bit
template <int CTRL>
__device__ __forceinline__ float fold_dpp(float a, float b, bool bit) {
    const float keep = bit ? b : a, give = bit ? a : b;
    return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), CTRL, 0xF, 0xF, false));
}

// 4 bf16 of a token, or zeros where there is none
__device__ __forceinline__ Quad quad_or_zero(const uint16_t *row0, int64_t stride, int t, int last) {
    Quad r = quad_at(row0 + (int64_t)min(t, last) * stride);
    if (t > last) r = Quad{{0.f, 0.f, 0.f, 0.f}};
    return r;
}

// The gradient of the state that leaves segment s, from what the segments
// behind it pass on from zero (the last one from d_final).
__device__ __forceinline__ void chain_back(const ScanParams &p, int64_t first, int s, int nseg, int64_t at, int ch,
                                           const float (&A)[4], float (&u)[4]) {
    const int64_t row = (int64_t)p.D * p.N;
#pragma unroll 4
    for (int j = nseg - 1; j > s; --j) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(p.adj + (first + j) * row + at);
        const float d = j < nseg - 1 ? p.steps[(first + j) * p.D + ch] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = j == nseg - 1 ? v[i] : __builtin_fmaf(fast_exp2(d * A[i]), u[i], v[i]);
    }
}

__device__ __forceinline__ f32x4 final_grad(const ScanParams &p, int64_t at) {
    if (p.d_final == nullptr) return f32x4{0.f, 0.f, 0.f, 0.f};
    return p.state_bf16 ? load_state4<true>(p.d_final, at) : load_state4<false>(p.d_final, at);
}

// What the segments of cut sequences pass on to those ahead of them, from zero
// but the last: U_t = (U_{t+1} + C_t e_t) a_t down to their first tokens.
template <int NW>
__global__ __launch_bounds__(NW * 64) void scan_adjoint(ScanParams p) {
    constexpr int NT = NW * 64, kItems = (kTile * 16 + NT - 1) / NT;
    __shared__ float2 sin[kTile][64];  // time step and e
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    Seq q;
    int s;
    if (!find_piece(p.qsl, p.batch, p.T, p.seg, blockIdx.x / p.blocks, q, s)) return;
    const int nseg = q.len > p.seg ? (q.len + p.seg - 1) / p.seg : 1;
    if (s == 0) return;
    const Span w = span_of(p, blockIdx.x % p.blocks);
    const int t0 = s * p.seg, t1 = min(q.len, t0 + p.seg), n0 = wave * 4;
    const bool mine = lane < w.nch && n0 < p.N;
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    const int64_t at = (int64_t)ch * p.N + n0;
    float A[4] = {}, u[4] = {};
    if (mine) {
        const f32x4 v = s == nseg - 1 ? final_grad(p, (int64_t)q.b * p.D * p.N + at) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            A[i] = p.A[at + i] * kLog2e;
            u[i] = v[i];
        }
    }
    const uint16_t *Cp = p.C + (int64_t)q.begin * p.cs + w.g * p.N + n0;
    for (int t = t0 + (t1 - 1 - t0) / kTile * kTile; t >= t0; t -= kTile) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = i / 16, c = (i % 16) * 4;
            if (i >= kTile * 16 || t + r >= t1 || c >= w.nch) continue;
            const int64_t row = q.begin + t + r;
            float d[4], e[4], z[4];
            widen4(*reinterpret_cast<const u32x2 *>(p.dt + row * p.dts + w.ch0 + c), d);
            widen4(*reinterpret_cast<const u32x2 *>(p.dy + row * p.D + w.ch0 + c), e);
            if (p.z != nullptr) {
                widen4(*reinterpret_cast<const u32x2 *>(p.z + row * p.zs + w.ch0 + c), z);
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] *= z[j] * sigmoid_f(z[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sin[r][c + j] = make_float2(time_step(p, d[j], w.ch0 + c + j), e[j]);
        }
        __syncthreads();
        if (n0 >= p.N) continue;
        for (int i = min(kTile, t1 - t) - 1; i >= 0; --i) {
            const float2 e = sin[i][lane];
            const Quad C = quad_at(Cp + (int64_t)(t + i) * p.cs);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __builtin_fmaf(C.v[j], e.y, u[j]) * fast_exp2(e.x * A[j]);
        }
    }
    if (mine)
        *reinterpret_cast<f32x4 *>(p.adj + (cut_place(p, q) + s) * p.D * p.N + at) = f32x4{u[0], u[1], u[2], u[3]};
}

template <int NW>
__global__ __launch_bounds__(NW * 64) void scan_grad(ScanParams p) {
    constexpr int NT = NW * 64, K = kGradTile, kItems = (K * 32 + NT - 1) / NT;
    constexpr int kTeams = NT < 256 ? NT / 32 : 8;  // threads that finish the same channels
    __shared__ float4 sin[K][64];        // time step, times x, e, x
    __shared__ float part[3][NW][K][64];  // a wavefront's shares of C.h, U.B and q.A
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int place = blockIdx.x / p.blocks, block = blockIdx.x % p.blocks;
    const Span w = span_of(p, block);
    const int n0 = wave * 4;
    const bool mine = lane < w.nch && n0 < p.N;
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    const int64_t at = (int64_t)ch * p.N + n0;
    float *dA_to = p.dA_part + (int64_t)place * p.D * p.N + at;
    float *dD_to = p.dD_part + (int64_t)place * 2 * p.D + w.ch0;
    Seq q;
    int s;
    if (!find_piece(p.qsl, p.batch, p.T, p.seg, place, q, s)) {  // an empty place adds nothing
        if (mine) *reinterpret_cast<f32x4 *>(dA_to) = f32x4{0.f, 0.f, 0.f, 0.f};
        if (threadIdx.x < w.nch) dD_to[threadIdx.x] = dD_to[p.D + threadIdx.x] = 0.f;
        return;
    }
    const int nseg = q.len > p.seg ? (q.len + p.seg - 1) / p.seg : 1;
    const int t0 = s * p.seg, t1 = min(q.len, t0 + p.seg), last = q.len - 1;
    const int64_t state = (int64_t)q.b * p.D * p.N + at;

    float A[4] = {}, u[4] = {}, dA[4] = {};  // u: the gradient of the state behind the walk
    if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = p.A[at + i] * kLog2e;
        if (s == nseg - 1) {
            const f32x4 v = final_grad(p, state);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = v[i];
        } else {
            chain_back(p, cut_place(p, q), s, nseg, at, ch, A, u);
        }
    }
    // the tokens and channels this thread prepares and finishes: 2 channels of a token an item
    const int c = (threadIdx.x % 32) * 2;
    const int64_t row0 = q.begin;
    const bool in = c < w.nch;
    float bias[2] = {}, skip[2] = {}, dD[2] = {}, db[2] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (in && p.bias != nullptr) bias[e] = p.bias[w.ch0 + c + e];
        if (in && p.Dskip != nullptr) skip[e] = p.Dskip[w.ch0 + c + e];
    }
    const uint16_t *Bp = p.B + row0 * p.bs + w.g * p.N + n0, *Cp = p.C + row0 * p.cs + w.g * p.N + n0;
    uint32_t nx[kItems], nd[kItems], nz[kItems], ny[kItems];
    f32x4 mark = {0.f, 0.f, 0.f, 0.f};
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int r = t + (threadIdx.x + k * NT) / 32;
            nx[k] = nd[k] = nz[k] = ny[k] = 0;
            if (r >= t + K || r >= t1 || !in) continue;
            const int64_t row = row0 + r;
            nx[k] = *reinterpret_cast<const uint32_t *>(p.x + row * p.xs + w.ch0 + c);
            nd[k] = *reinterpret_cast<const uint32_t *>(p.dt + row * p.dts + w.ch0 + c);
            ny[k] = *reinterpret_cast<const uint32_t *>(p.dy + row * p.D + w.ch0 + c);
            if (p.z != nullptr) nz[k] = *reinterpret_cast<const uint32_t *>(p.z + row * p.zs + w.ch0 + c);
        }
        if (mine) mark = *reinterpret_cast<const f32x4 *>(mark_at(p, q, t, n0, ch));
    };
    const int tiles = (t1 - t0 + K - 1) / K;
    if (tiles > 0) fetch(t0 + (tiles - 1) * K);
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int t = t0 + tile * K, n = min(K, t1 - t);
        uint32_t rd[kItems], rz[kItems], ry[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = i / 32;
            rd[k] = nd[k];
            rz[k] = nz[k];
            ry[k] = ny[k];
            if (i >= K * 32) continue;
            const bool live = r < n && in;  // elsewhere nothing happens: no step, no gradient
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = e ? bf16x2_hi(nx[k]) : bf16x2_lo(nx[k]), z = e ? bf16x2_hi(nz[k]) : bf16x2_lo(nz[k]);
                const float raw = (e ? bf16x2_hi(nd[k]) : bf16x2_lo(nd[k])) + bias[e];
                const float step = p.softplus ? softplus_f(raw) : raw;
                float g = e ? bf16x2_hi(ny[k]) : bf16x2_lo(ny[k]);
                if (p.z != nullptr) g *= z * sigmoid_f(z);
                sin[r][c + e] = live ? make_float4(step, step * x, g, x) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        const f32x4 h0 = mark;
        if (tile > 0) fetch(t - K);
        __syncthreads();
        if (n0 < p.N) {
            float h[K][4], a[K][4];
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const float4 v = sin[i][lane];
                const Quad B = quad_or_zero(Bp, p.bs, t + i, last), C = quad_or_zero(Cp, p.cs, t + i, last);
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[i][j] = fast_exp2(v.x * A[j]);
                    h[i][j] = __builtin_fmaf(a[i][j], i > 0 ? h[i > 0 ? i - 1 : 0][j] : h0[j], v.y * B.v[j]);
                    y = __builtin_fmaf(C.v[j], h[i][j], y);
                }
                part[0][wave][i][lane] = y;
            }
            float dAt[4] = {}, f[K][4];
#pragma unroll
            for (int i = K - 1; i >= 0; --i) {
                const float4 v = sin[i][lane];
                const Quad B = quad_or_zero(Bp, p.bs, t + i, last), C = quad_or_zero(Cp, p.cs, t + i, last);
                float uB = 0.f, qA = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = __builtin_fmaf(C.v[j], v.z, u[j]);
                    // (lanes without a channel hold zeros: no share in the sums over channels)
                    f[i][j] = fold32(v.z * h[i][j], u[j] * v.y);
                    uB = __builtin_fmaf(u[j], B.v[j], uB);
                    u[j] *= a[i][j];
                    const float qq = u[j] * (i > 0 ? h[i > 0 ? i - 1 : 0][j] : h0[j]);
                    qA = __builtin_fmaf(qq, A[j], qA);
                    dAt[j] = __builtin_fmaf(qq, v.x, dAt[j]);
                }
                part[1][wave][i][lane] = uB;
                part[2][wave][i][lane] = qA;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dA[j] += dAt[j];
            // value (gradient, token, state) of lane bits (5), (4, 3, 2), (1, 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = fold16(f[i][j], f[i + 4][j]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = fold_dpp<0x128>(f[i][j], f[i + 2][j], lane & 8);  // row_ror:8
#pragma unroll
            for (int j = 0; j < 4; ++j) f[0][j] = fold_dpp<0x141>(f[0][j], f[1][j], lane & 4);  // row_half_mirror
            f[0][0] = fold_dpp<0x4E>(f[0][0], f[0][2], lane & 2);  // quad_perm [2,3,0,1]
            f[0][1] = fold_dpp<0x4E>(f[0][1], f[0][3], lane & 2);
            f[0][0] = fold_dpp<0xB1>(f[0][0], f[0][1], lane & 1);  // quad_perm [1,0,3,2]
            const int i = (lane >> 2) & 7;
            if (i < n) {
                const int64_t row = (int64_t)block * p.T + row0 + t + i;
                p.bc[(row * 2 + (lane >> 5)) * p.N + n0 + (lane & 3)] = f[0][0];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = i / 32;
            if (i >= K * 32 || r >= n || !in) continue;
            float2 y = make_float2(0.f, 0.f), uB = y, qA = y;
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                if (v * 4 >= p.N) continue;
                const float2 a = *reinterpret_cast<const float2 *>(&part[0][v][r][c]);
                const float2 b = *reinterpret_cast<const float2 *>(&part[1][v][r][c]);
                const float2 d = *reinterpret_cast<const float2 *>(&part[2][v][r][c]);
                y.x += a.x;
                y.y += a.y;
                uB.x += b.x;
                uB.y += b.y;
                qA.x += d.x;
                qA.y += d.y;
            }
            float dx[2], ddt[2], dz[2] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 v = sin[r][c + e];
                const float b = e ? uB.y : uB.x;
                const float raw = (e ? bf16x2_hi(rd[k]) : bf16x2_lo(rd[k])) + bias[e];
                dx[e] = __builtin_fmaf(v.x, b, skip[e] * v.z);
                ddt[e] = __builtin_fmaf(e ? qA.y : qA.x, kLn2, v.w * b);
                if (p.softplus) ddt[e] *= sigmoid_f(raw);
                dD[e] = __builtin_fmaf(v.z, v.w, dD[e]);
                db[e] += ddt[e];
                if (p.z != nullptr) {
                    const float z = e ? bf16x2_hi(rz[k]) : bf16x2_lo(rz[k]), o = sigmoid_f(z);
                    const float g = e ? bf16x2_hi(ry[k]) : bf16x2_lo(ry[k]);
                    const float out = __builtin_fmaf(skip[e], v.w, e ? y.y : y.x);
                    dz[e] = g * out * __builtin_fmaf(z * o, 1.f - o, o);
                }
            }
            const int64_t to = (row0 + t + r) * p.D + w.ch0 + c;
            *reinterpret_cast<uint32_t *>(p.dx + to) = pack_bf16x2(dx[0], dx[1]);
            *reinterpret_cast<uint32_t *>(p.ddt + to) = pack_bf16x2(ddt[0], ddt[1]);
            if (p.z != nullptr) *reinterpret_cast<uint32_t *>(p.dz + to) = pack_bf16x2(dz[0], dz[1]);
        }
        __syncthreads();
    }
    if (mine) {
        *reinterpret_cast<f32x4 *>(dA_to) = f32x4{dA[0], dA[1], dA[2], dA[3]};
        if (s == 0 && p.d_init != nullptr) {
            const f32x4 v = {u[0], u[1], u[2], u[3]};
            if (p.state_bf16)
                store_state4<true>(p.d_init, state, v);
            else
                store_state4<false>(p.d_init, state, v);
        }
    }
    // sums over tokens of what belongs to channels
    float2 *sums = reinterpret_cast<float2 *>(&sin[0][0]);  // [kTeams][64]
    const int team = threadIdx.x / 32;
    if (team < kTeams)
#pragma unroll
        for (int e = 0; e < 2; ++e) sums[team * 64 + c + e] = make_float2(dD[e], db[e]);
    __syncthreads();
    for (int i = threadIdx.x; i < w.nch; i += NT) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kTeams; ++k) {
            v.x += sums[k * 64 + i].x;
            v.y += sums[k * 64 + i].y;
        }
        dD_to[i] = v.x;
        dD_to[p.D + i] = v.y;
    }
}

// dB and dC: the blocks of a group, added in their order.
__global__ __launch_bounds__(256) void sum_blocks(ScanParams p) {
    const int quads = p.N / 4;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int j = (int)(i % quads);
    i /= quads;
    const int which = (int)(i & 1);
    i >>= 1;
    const int64_t row = i / p.G;
    const int g = (int)(i % p.G);
    if (row >= clamp_row(p.qsl[p.batch], p.T) || row < clamp_row(p.qsl[0], p.T)) return;
    const int per = p.blocks / p.G;
    const float *src = p.bc + (((int64_t)g * per * p.T + row) * 2 + which) * p.N + j * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < per; ++k) v += *reinterpret_cast<const f32x4 *>(src + (int64_t)k * p.T * 2 * p.N);
    uint16_t *to = (which ? p.dB : p.dC) + (row * p.G + g) * p.N + j * 4;
    *reinterpret_cast<u32x2 *>(to) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

}  // namespace

hipError_t launch_scan_grad(const ScanParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.places * p.blocks));
    hipError_t e = launch_scan_states(p, s);
    if (e != hipSuccess) return e;
    if (p.cut_places > 0)
        by_waves(waves_of(p.N), [&](auto n) {
            constexpr int NW = decltype(n)::value;
            scan_adjoint<NW><<<grid, NW * 64, 0, s>>>(p);
        });
    if ((e = launch_scan_marks(p, s)) != hipSuccess) return e;
    by_waves(waves_of(p.N), [&](auto n) {
        constexpr int NW = decltype(n)::value;
        scan_grad<NW><<<grid, NW * 64, 0, s>>>(p);
    });
    const int64_t sums = (int64_t)p.T * p.G * 2 * (p.N / 4);
    if (sums > 0) sum_blocks<<<dim3((unsigned)((sums + 255) / 256)), 256, 0, s>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t DN = (int64_t)p.D * p.N, n = p.places;
    if ((e = launch_sum_parts(p.dA_part, (int)n, DN, DN, p.dA, s)) != hipSuccess) return e;
    if (p.dD != nullptr && (e = launch_sum_parts(p.dD_part, (int)n, 2 * p.D, p.D, p.dD, s)) != hipSuccess) return e;
    if (p.dbias != nullptr) e = launch_sum_parts(p.dD_part + p.D, (int)n, 2 * p.D, p.D, p.dbias, s);
    return e;
}

}  // namespace layer
}  // namespace ssd
