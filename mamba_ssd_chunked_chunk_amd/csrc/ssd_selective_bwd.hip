// Backward pass of the selective scan.  With a = exp(dts A), e = dy silu(z) and U
// the gradient of the state,
//     U_t = C_t e_t + a_{t+1} U_{t+1}
// runs against the tokens and needs every token's state, so a forward walk
// first leaves the state ahead of each tile of 8 tokens, and the backward walk
// goes from tile to tile, makes its 8 states again (and keeps them and their
// decays in registers) and then turns round.  As in the forward pass a
// workgroup takes 64 channels and a wavefront 4 states of them (or two groups of
// 4 in turn), a channel a lane; sums over states go through LDS.  Sums over
// channels (dB and dC) are formed by exchanging halves: 64 values a lane, of 8
// tokens, 4 states and the two gradients, become one a lane in 6 steps, each of
// which adds what two lanes hold of half the values.  They leave as fp32 for each
// 64 channels, and a last kernel adds the blocks of a group, in their order.
//
// 8 x 2048 tokens of 4096 channels and 16 states: states 215 us (of which the
// 537 MB that they write 103), gradients 790, sums 34.  Arithmetic bounds the
// gradients (0.89 vector instructions a cycle and compute unit): a token and state
// costs its decay (an exponential and a product), 5 products, 6 fused adds and two
// exchanges between lanes.
// Tiles of 16 tokens would halve the states (226 -> 213 us) but hold 64 more
// registers a lane, and spill (gradients 857 -> 944 us); three wavefronts a SIMD in
// 168 registers leave the last workgroups alone on their units (857 -> 989 us).
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

// The gradient of the state that leaves segment s, from what the segments
// behind it pass on: the last one in full, the others from zero.
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

// G: groups of 4 states that a wavefront takes one after the other
template <int NW, int G>
union Shared {
    struct {
        float2 sx[kGradTile][64];      // time step, and times x
        f32x4 B[kGradTile][NW * G], C[kGradTile][NW * G];
        float e[kGradTile][64];
        float y[NW][kGradTile][64];    // a wavefront's shares of C.h
        float2 uq[NW][kGradTile][64];  // and of U.B and q.A
    };
    struct {
        float2 step[kTile][64];  // time step and e
        f32x4 adjC[kTile][NW * G];
    };
};

// What a segment between the first and the last passes on to those ahead of it,
// from zero: U_t = (U_{t+1} + C_t e_t) a_t down to its first token.
template <int NW, int G>
__device__ __forceinline__ void adjoint(const ScanParams &p, Shared<NW, G> &lds, const Seq &q, int s, const Span &w) {
    constexpr int NT = NW * 64, kItems = (kTile * 16 + NT - 1) / NT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const int t0 = s * p.seg;
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    float A[G][4] = {}, u[G][4] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int n0 = (g * NW + wave) * 4;
        if (lane < w.nch && n0 < p.N)
#pragma unroll
            for (int i = 0; i < 4; ++i) A[g][i] = p.A[(int64_t)ch * p.N + n0 + i] * kLog2e;
    }
    const int half = p.N / 2, wt = threadIdx.x / half, we = threadIdx.x % half * 2;  // two elements of C, by a thread
    for (int t = t0 + p.seg - kTile; t >= t0; t -= kTile) {  // (a whole number of tiles)
        __syncthreads();
        if (wt < kTile) {
            const uint32_t v =
                *reinterpret_cast<const uint32_t *>(p.C + (int64_t)(q.begin + t + wt) * p.cs + w.g * p.N + we);
            *reinterpret_cast<float2 *>(reinterpret_cast<float *>(&lds.adjC[wt][0]) + we) =
                make_float2(bf16x2_lo(v), bf16x2_hi(v));
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = threadIdx.x + k * NT, r = i / 16, c = (i % 16) * 4;
            if (i >= kTile * 16 || c >= w.nch) continue;
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
            for (int j = 0; j < 4; ++j)
                lds.step[r][c + j] = make_float2(
                    time_step(p, d[j] + (p.bias != nullptr ? p.bias[w.ch0 + c + j] : 0.f)), e[j]);
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if ((g * NW + wave) * 4 >= p.N) continue;
#pragma unroll
            for (int i = kTile - 1; i >= 0; --i) {
                const float2 e = lds.step[i][lane];
                const f32x4 C = lds.adjC[i][g * NW + wave];
#pragma unroll
                for (int j = 0; j < 4; ++j) u[g][j] = __builtin_fmaf(C[j], e.y, u[g][j]) * fast_exp2(e.x * A[g][j]);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int n0 = (g * NW + wave) * 4;
        if (lane < w.nch && n0 < p.N)
            *reinterpret_cast<f32x4 *>(p.adj + ((cut_place(p, q) + s) * p.D + ch) * p.N + n0) =
                f32x4{u[g][0], u[g][1], u[g][2], u[g][3]};
    }
}

// One segment of a sequence (or all of it) and 64 channels.
template <int NW, int G>
__device__ __forceinline__ void grad(const ScanParams &p, Shared<NW, G> &lds, const Piece &piece, int block) {
    const Seq &q = piece.q;
    const int s = piece.s, nseg = piece.nseg;
    constexpr int NT = NW * 64, K = kGradTile, kItems = (K * 32 + NT - 1) / NT, kStep = NT / 32;
    constexpr int kTeams = NT < 256 ? kStep : 8;  // threads that finish the same channels
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const Span w = span_of(p, block);
    const int ch = w.ch0 + (lane < w.nch ? lane : 0);
    const int64_t at = (int64_t)ch * p.N;
    const int t0 = s * p.seg, t1 = nseg > 1 ? min(q.len, t0 + p.seg) : q.len;
    const int64_t state = (int64_t)q.b * p.D * p.N + at;

    bool mine[G];
    float A[G][4] = {}, u[G][4] = {}, dA[G][4] = {};  // u: the gradient of the state behind the walk
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int n0 = (g * NW + wave) * 4;
        mine[g] = lane < w.nch && n0 < p.N;
        if (!mine[g]) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) A[g][i] = p.A[at + n0 + i] * kLog2e;
        if (s == nseg - 1) {
            const f32x4 v = final_grad(p, state + n0);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[g][i] = v[i];
        } else {
            chain_back(p, cut_place(p, q), s, nseg, at + n0, ch, A[g], u[g]);
        }
    }
    if (wave * 4 >= p.N) {  // no states, no share
        for (int i = 0; i < K; ++i) {
            lds.y[wave][i][lane] = 0.f;
            lds.uq[wave][i][lane] = make_float2(0.f, 0.f);
        }
    }
    // the tokens and channels this thread prepares and finishes: 2 channels of a token an item, the same ones in
    // every item
    const int c = (threadIdx.x % 32) * 2, r0 = threadIdx.x / 32;
    const bool in = c < w.nch;
    float bias[2] = {}, skip[2] = {}, dD[2] = {}, db[2] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (in && p.bias != nullptr) bias[e] = p.bias[w.ch0 + c + e];
        if (in && p.Dskip != nullptr) skip[e] = p.Dskip[w.ch0 + c + e];
    }
    // pointers to the first row of the tile that is worked on (or, of inputs, fetched next), and bytes from there
    const int tiles = (t1 - t0 + K - 1) / K;
    const int64_t row = q.begin + t0 + (int64_t)(tiles - 1) * K;
    const bool gate = p.z != nullptr;
    const uint16_t *xp = p.x + row * p.xs + w.ch0, *tp = p.dt + row * p.dts + w.ch0, *yp = p.dy + row * p.D + w.ch0;
    const uint16_t *zp = gate ? p.z + row * p.zs + w.ch0 : nullptr;
    uint16_t *dxp = p.dx + row * p.D + w.ch0, *dtp = p.ddt + row * p.D + w.ch0;
    uint16_t *dzp = gate ? p.dz + row * p.D + w.ch0 : nullptr;
    const int xs = (int)p.xs * 2, ts = (int)p.dts * 2, zs = (int)p.zs * 2, ys = p.D * 2;  // bytes between rows
    const uint32_t xo = r0 * xs + c * 2, to = r0 * ts + c * 2, zo = r0 * zs + c * 2, yo = r0 * ys + c * 2;
    // two elements of B or of C of a token of the tile, by the first K N threads
    const int bt = threadIdx.x / p.N, bj = threadIdx.x % p.N * 2;
    const bool ofC = bj >= p.N;
    const int64_t bcs = ofC ? p.cs : p.bs;
    const uint16_t *Wp = (ofC ? p.C + (bj - p.N) : p.B + bj) + (row + bt) * bcs + w.g * p.N;
    float *Wl = reinterpret_cast<float *>(ofC ? &lds.C[bt < K ? bt : 0][0] : &lds.B[bt < K ? bt : 0][0]) +
                (ofC ? bj - p.N : bj);
    uint32_t nw = 0;
    const int64_t mark0 = q.begin / K + q.b + t0 / K + (int64_t)(tiles - 1);
    const float *mp = p.marks + (mark0 * (p.N / 4) + wave) * p.D * 4;  // (of group 0)
    // value (gradient, token, state) of a lane's bits (5), (4, 3, 2), (1, 0)
    float *bcp = p.bc + ((int64_t)block * p.T + row) * 2 * p.N;
    const int bi = (lane >> 2) & 7;
    const uint32_t bo = ((bi * 2 + (lane >> 5)) * p.N + wave * 4 + (lane & 3)) * 4;

    uint32_t nx[kItems], nd[kItems], nz[kItems], ny[kItems];
    f32x4 mark[G] = {};
    auto fetch = [&](int n) {  // n: tokens of the tile
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            nx[k] = nd[k] = nz[k] = ny[k] = 0;
            if (r0 + k * kStep >= n || !in) continue;
            nx[k] = at_offset<uint32_t>(xp, xo + k * kStep * xs);
            nd[k] = at_offset<uint32_t>(tp, to + k * kStep * ts);
            ny[k] = at_offset<uint32_t>(yp, yo + k * kStep * ys);
            if (gate) nz[k] = at_offset<uint32_t>(zp, zo + k * kStep * zs);
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (mine[g]) mark[g] = at_offset<f32x4>(mp + (int64_t)g * NW * p.D * 4, (uint32_t)ch * 16);
        nw = bt < n ? *reinterpret_cast<const uint32_t *>(Wp) : 0;
        Wp -= K * bcs;
        xp = moved(xp, -(int64_t)K * xs);
        tp = moved(tp, -(int64_t)K * ts);
        yp = moved(yp, -(int64_t)K * ys);
        if (gate) zp = moved(zp, -(int64_t)K * zs);
        mp -= (int64_t)p.N * p.D;
    };
    if (tiles > 0) fetch(t1 - t0 - (tiles - 1) * K);
    const float still = p.softplus ? -__builtin_inff() : 0.f;  // what makes a step of 0
    // (loads that have to be here before the loop: a wait inside it would be for the last tile's stores too)
#pragma unroll
    for (int e = 0; e < 2; ++e) asm volatile("" : "+v"(bias[e]), "+v"(skip[e]));
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(A[g][e]), "+v"(u[g][e]));
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int n = min(K, t1 - t0 - tile * K);
        if (bt < K) *reinterpret_cast<float2 *>(Wl) = make_float2(bf16x2_lo(nw), bf16x2_hi(nw));
        float step[kItems][2], x[kItems][2], e[kItems][2], slope[kItems][2], wz[kItems][2];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int r = r0 + k * kStep;
            if (r >= K) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[k][i] = i ? bf16x2_hi(nx[k]) : bf16x2_lo(nx[k]);
                const float g = i ? bf16x2_hi(ny[k]) : bf16x2_lo(ny[k]);
                float raw = (i ? bf16x2_hi(nd[k]) : bf16x2_lo(nd[k])) + bias[i];
                raw = r < n ? raw : still;
                step[k][i] = raw;
                slope[k][i] = 1.f;
                if (p.softplus) {
                    const float v = fast_exp2(-fabsf(raw) * kLog2e);  // softplus_fast, and its slope beside it
                    const float m = 1.f + v;
                    step[k][i] = __builtin_amdgcn_fmed3f(raw, 0.f, __builtin_inff()) +
                                 __builtin_fmaf(__builtin_amdgcn_logf(m), kLn2, v - (m - 1.f));
                    slope[k][i] = __builtin_amdgcn_rcpf(m) * (raw >= 0.f ? 1.f : v);
                }
                e[k][i] = g;
                wz[k][i] = 0.f;
                if (gate) {
                    const float z = i ? bf16x2_hi(nz[k]) : bf16x2_lo(nz[k]), o = sigmoid_f(z), zo_ = z * o;
                    e[k][i] = g * zo_;
                    wz[k][i] = g * __builtin_fmaf(zo_, 1.f - o, o);
                }
                lds.sx[r][c + i] = make_float2(step[k][i], step[k][i] * x[k][i]);
                lds.e[r][c + i] = e[k][i];
            }
        }
        f32x4 first[G];
#pragma unroll
        for (int g = 0; g < G; ++g) first[g] = mark[g];
        if (tile > 0) fetch(K);
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if ((g * NW + wave) * 4 >= p.N) continue;
            if (g > 0) asm volatile("" ::: "memory");  // (what both groups read is read again, not kept)
            const f32x4 h0 = first[g];
            // a token's numbers are read while the one ahead of it is worked on (the compiler, which takes the stores
            // between for a hindrance, would read and wait)
            struct Token {
                float2 v;
                float e;
                f32x4 B, C;
                float2 share;  // of the groups ahead
            };
            auto read = [&](int i, bool back) {
                const int b = g * NW + wave;
                Token m{lds.sx[i][lane], back ? lds.e[i][lane] : 0.f, lds.B[i][b], lds.C[i][b], make_float2(0.f, 0.f)};
                if (g > 0 && back) m.share = lds.uq[wave][i][lane];
                if (g > 0 && !back) m.share.x = lds.y[wave][i][lane];
                return m;
            };
            float h[K][4], a[K][4];
            Token next = read(0, false);
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const Token m = next;
                next = i < K - 1 ? read(i + 1, false) : read(K - 1, true);
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[i][j] = fast_exp2(m.v.x * A[g][j]);
                    h[i][j] = __builtin_fmaf(a[i][j], i > 0 ? h[i > 0 ? i - 1 : 0][j] : h0[j], m.v.y * m.B[j]);
                    y = j == 0 ? m.C[j] * h[i][j] : __builtin_fmaf(m.C[j], h[i][j], y);
                }
                lds.y[wave][i][lane] = g > 0 ? y + m.share.x : y;
            }
            float dAt[4] = {}, f[K][4];
#pragma unroll
            for (int i = K - 1; i >= 0; --i) {
                const Token m = next;
                if (i > 0) next = read(i - 1, true);
                float uB = 0.f, qA = 0.f, forB[4], forC[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[g][j] = __builtin_fmaf(m.C[j], m.e, u[g][j]);
                    forC[j] = m.e * h[i][j];
                    forB[j] = u[g][j] * m.v.y;
                    uB = j == 0 ? u[g][j] * m.B[j] : __builtin_fmaf(u[g][j], m.B[j], uB);
                    u[g][j] *= a[i][j];
                    const float qq = u[g][j] * (i > 0 ? h[i > 0 ? i - 1 : 0][j] : h0[j]);
                    qA = j == 0 ? qq * A[g][j] : __builtin_fmaf(qq, A[g][j], qA);
                    dAt[j] = i == K - 1 ? qq * m.v.x : __builtin_fmaf(qq, m.v.x, dAt[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (lanes without a channel hold zeros: no share in the sums over channels)
                    f[i][j] = fold32(forC[j], forB[j]);
                    if (i < 4) f[i][j] = fold16(f[i][j], f[i + 4][j]);
                    if (i < 2) f[i][j] = fold_dpp<0x128>(f[i][j], f[i + 2][j], lane & 8);  // row_ror:8
                }
                if (g > 0) {
                    uB += m.share.x;
                    qA += m.share.y;
                }
                lds.uq[wave][i][lane] = make_float2(uB, qA);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dA[g][j] += dAt[j];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[0][j] = fold_dpp<0x141>(f[0][j], f[1][j], lane & 4);  // row_half_mirror
            f[0][0] = fold_dpp<0x4E>(f[0][0], f[0][2], lane & 2);  // quad_perm [2,3,0,1]
            f[0][1] = fold_dpp<0x4E>(f[0][1], f[0][3], lane & 2);
            f[0][0] = fold_dpp<0xB1>(f[0][0], f[0][1], lane & 1);  // quad_perm [1,0,3,2]
            if (bi < n) put_offset(bcp, bo + g * NW * 16, f[0][0]);
        }
        bcp -= (int64_t)K * 2 * p.N;
        __syncthreads();
        uint32_t ox[kItems], od[kItems], oz[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int r = min(r0 + k * kStep, K - 1);
            float2 y = make_float2(0.f, 0.f), uB, qA;
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                const float4 b = *reinterpret_cast<const float4 *>(&lds.uq[v][r][c]);
                uB = v == 0 ? make_float2(b.x, b.z) : make_float2(uB.x + b.x, uB.y + b.z);
                qA = v == 0 ? make_float2(b.y, b.w) : make_float2(qA.x + b.y, qA.y + b.w);
                if (gate) {
                    const float2 a = *reinterpret_cast<const float2 *>(&lds.y[v][r][c]);
                    y = make_float2(y.x + a.x, y.y + a.y);
                }
            }
            float dx[2], dt[2], dz[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float b = i ? uB.y : uB.x;
                dx[i] = __builtin_fmaf(step[k][i], b, skip[i] * e[k][i]);
                dt[i] = __builtin_fmaf(i ? qA.y : qA.x, kLn2, x[k][i] * b) * slope[k][i];
                dz[i] = wz[k][i] * __builtin_fmaf(skip[i], x[k][i], i ? y.y : y.x);
                if (r0 + k * kStep < n) {
                    dD[i] = __builtin_fmaf(e[k][i], x[k][i], dD[i]);
                    db[i] += dt[i];
                }
            }
            ox[k] = pack_bf16x2(dx[0], dx[1]);
            od[k] = pack_bf16x2(dt[0], dt[1]);
            oz[k] = pack_bf16x2(dz[0], dz[1]);
        }
        // the next tile's rows are waited for here, ahead of the stores
#pragma unroll
        for (int k = 0; k < kItems; ++k) asm volatile("" : "+v"(nx[k]), "+v"(nd[k]), "+v"(ny[k]), "+v"(nz[k]));
#pragma unroll
        for (int g = 0; g < G; ++g) asm volatile("" : "+v"(mark[g]));
        asm volatile("" : "+v"(nw));
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (r0 + k * kStep >= n || !in) continue;
            const uint32_t o = yo + k * kStep * ys;
            put_offset(dxp, o, ox[k]);
            put_offset(dtp, o, od[k]);
            if (gate) put_offset(dzp, o, oz[k]);
        }
        dxp = moved(dxp, -(int64_t)K * ys);
        dtp = moved(dtp, -(int64_t)K * ys);
        if (gate) dzp = moved(dzp, -(int64_t)K * ys);
    }
    const int64_t place = piece.number;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (!mine[g]) continue;
        const int n0 = (g * NW + wave) * 4;
        const f32x4 v = {u[g][0], u[g][1], u[g][2], u[g][3]};
        *reinterpret_cast<f32x4 *>(p.dA_part + place * p.D * p.N + at + n0) =
            f32x4{dA[g][0], dA[g][1], dA[g][2], dA[g][3]};
        if (s > 0) {
            if (s == nseg - 1) *reinterpret_cast<f32x4 *>(p.adj + (cut_place(p, q) + s) * p.D * p.N + at + n0) = v;
        } else if (p.d_init != nullptr) {
            if (p.state_bf16)
                store_state4<true>(p.d_init, state + n0, v);
            else
                store_state4<false>(p.d_init, state + n0, v);
        }
    }
    // sums over tokens of what belongs to channels
    __syncthreads();
    if (r0 < kTeams)
#pragma unroll
        for (int i = 0; i < 2; ++i) lds.sx[r0][c + i] = make_float2(dD[i], db[i]);
    __syncthreads();
    float *dD_to = p.dD_part + place * 2 * p.D + w.ch0;
    for (int i = threadIdx.x; i < w.nch; i += NT) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kTeams; ++k) {
            v.x += lds.sx[k][i].x;
            v.y += lds.sx[k][i].y;
        }
        dD_to[i] = v.x;
        dD_to[p.D + i] = v.y;
    }
}

// Whole sequences and last segments; what the segments between pass on.
template <int NW, int G>
__global__ __launch_bounds__(NW * 64, 2) void scan_grad_first(ScanParams p) {
    __shared__ Shared<NW, G> lds;
    const int place = blockIdx.x / p.blocks, block = blockIdx.x % p.blocks;
    Piece w;
    if (!piece_at<false>(p, place, w)) {  // an empty place adds nothing
        const Span c = span_of(p, block);
        const int lane = threadIdx.x & 63;
        for (int n0 = threadIdx.x / 64 * 4; lane < c.nch && n0 < p.N; n0 += NW * 4)
            *reinterpret_cast<f32x4 *>(p.dA_part + ((int64_t)place * p.D + c.ch0 + lane) * p.N + n0) =
                f32x4{0.f, 0.f, 0.f, 0.f};
        float *dD = p.dD_part + (int64_t)place * 2 * p.D + c.ch0;
        if (threadIdx.x < c.nch) dD[threadIdx.x] = dD[p.D + threadIdx.x] = 0.f;
        return;
    }
    if (w.s == w.nseg - 1)
        grad<NW, G>(p, lds, w, block);
    else if (w.s > 0)
        adjoint<NW, G>(p, lds, w.q, w.s, span_of(p, block));
}
template <int NW, int G>
__global__ __launch_bounds__(NW * 64, 2) void scan_grad_rest(ScanParams p) {
    __shared__ Shared<NW, G> lds;
    Piece w;
    if (piece_at<true>(p, blockIdx.x / p.blocks, w) && w.s < w.nseg - 1) grad<NW, G>(p, lds, w, blockIdx.x % p.blocks);
}

// The sums over blocks and places: dB and dC, the blocks of a group added in
// their order, by the first bc_blocks workgroups, and dA, dD, dbias.
__global__ __launch_bounds__(kSumThreads) void scan_sums(ScanParams p, int64_t bc_blocks, Sums sums) {
    if (blockIdx.x >= bc_blocks) return add_parts<64>(sums, blockIdx.x - bc_blocks);
    const int quads = p.N / 4;
    int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
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

// The wavefronts that hold N states, and the groups of 4 that each of them takes: one to 16 states, two above, which
// share a tile's preparation and let two wavefronts a SIMD keep their registers (8 x 1024 tokens of 4096 channels with
// one and two groups: 20 states 988 and 849 us, 32 states 1041 and 967; 64 states in 16 wavefronts, which had to spill,
// 3976, in 8 1866).  One of 4 wavefronts is left idle where 3 would do (12 states 610 -> 549 us: the rows of a tile
// come out even), not two of 4 (8 states 611 us in 2, 535 in 4, but with 16 sequences 669 and 941); one of 2 is, as a
// wavefront alone would spill (4 states 505 us in 1, 508 in 2, with 16 sequences 825 and 627, with 32 1023 and 1140).
template <typename F>
void by_groups(int N, F f) {
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    switch ((N + 3) / 4) {
    case 1:
    case 2: return f(std::integral_constant<int, 2>{}, one);
    case 3:
    case 4: return f(std::integral_constant<int, 4>{}, one);
    case 5:
    case 6:
    case 7:
    case 8: return f(std::integral_constant<int, 4>{}, two);
    default: return f(std::integral_constant<int, 8>{}, two);
    }
}

}  // namespace

int grad_waves_of(int N) {
    int waves = 0;
    by_groups(N, [&](auto n, auto) { waves = decltype(n)::value; });
    return waves;
}

hipError_t launch_scan_grad(const ScanParams &p, hipStream_t s) {
    hipError_t e = launch_scan_marks(p, s);
    if (e != hipSuccess) return e;
    by_groups(p.N, [&](auto n, auto groups) {
        constexpr int NW = decltype(n)::value, G = decltype(groups)::value;
        scan_grad_first<NW, G><<<dim3((unsigned)(p.places * p.blocks)), NW * 64, 0, s>>>(p);
        if (p.cut_places > 0)
            scan_grad_rest<NW, G><<<dim3((unsigned)(p.cut_places * p.blocks)), NW * 64, 0, s>>>(p);
    });
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t bc_blocks = ((int64_t)p.T * p.G * (p.N / 2) + kSumThreads - 1) / kSumThreads;
    const int64_t DN = (int64_t)p.D * p.N;
    const int n = (int)p.places;
    const Sums sums = {{{p.dA_part, n, DN, DN, p.dA}, {p.dD_part, n, 2 * p.D, p.D, p.dD},
                        {p.dD_part + p.D, n, 2 * p.D, p.D, p.dbias}}};
    scan_sums<<<dim3((unsigned)(bc_blocks + sum_blocks<64>(sums))), kSumThreads, 0, s>>>(p, bc_blocks, sums);
    return hipGetLastError();
}

}  // namespace layer
}  // namespace ssd
