// Gradients of the selective scan (selective_scan.cuh), from its inputs and the gradient of its
// outputs and final states; nothing of the forward pass is needed.
//
//   dy_t = dout_t silu(z_t)                     dz_t = dout_t (y_t + skip u_t) silu'(z_t)
//   g_t  = C_t dy_t + a_{t+1} g_{t+1}           (the gradient of h_t; a_t = exp(delta_t A))
//   dC_t = sum_d h_t dy_t                       dB_t = sum_d g_t delta_t u_t
//   e_t  = g_t a_t h_{t-1}                      (the gradient of delta_t A)
//   du_t = delta_t sum_m g_t B_t + skip dy_t    ddelta_t = u_t sum_m g_t B_t + sum_m e_t A
//   ddt  = ddelta sigmoid(dt + dt_bias)         dA_log = A sum_t e_t delta_t
//
// Both recurrences, h forwards and g backwards, are linear, so the time axis is cut into chunks of
// kTC tokens that run side by side:
//   1. scan_bwd_chunk_kernel  each chunk's end state from zero and its share of the gradient at its
//                             start, in one pass (the running product of decays takes no exponential)
//   2. scan_bwd_chain_kernel  the states at the chunk starts (forwards) and the gradients at the chunk
//                             ends (backwards), in place
//   3. scan_bwd_grad_kernel   every chunk's gradients: a pass forwards that keeps every eighth state,
//                             then eight tokens at a time recomputed into registers and run backwards
//   4. two sums of partial results over channel blocks (dB, dC) and over chunks (the weights)
// Three exponentials per (token, channel, state); sums are taken in a fixed order, so results do not
// vary between runs.
#pragma once

#include "selective_scan.cuh"

namespace kda {

struct ScanBwdParams {
    const void *u, *dt, *z, *B, *C, *dout;
    const float *A_log, *skip, *dt_bias;
    const int32_t *cu;
    const float *h0, *dhN;              // [num_seqs, D, n] or null
    void *du, *ddt, *dz, *dB, *dC;
    float *dA_log, *dskip, *ddt_bias, *dh0;
    // workspace; records as scan_segment with kTC tokens
    float *H;       // [records, D, n] chunk end states, then start states, then the chunk's sum of e delta
    float *R;       // [records, D, n] gradient at the chunk starts, then at the chunk ends
    float *sum_delta;   // [records, D]
    float *pskip, *pbias;   // [records, D] the chunk's share of dskip and ddt_bias
    float *pBC;     // [channel blocks, T, 2 n] the block's share of dB, dC
    int64_t total_tokens, records;
    int num_seqs, D, n, G, cbg;
    bool vec, vecn;
};

template <int L>
struct ScanBwdTile : ScanTile<L> {
    static constexpr int kTC = 2 * ScanTile<L>::kTT;   // tokens of a chunk (two staged tiles)
};

// Sum over LANES lanes (STRIDE apart, this one the idx-th) for V values at once: lane idx is left
// with the totals of v[idx V / LANES] .. in v[0] ..
template <int V, int LANES, int STRIDE>
__device__ __forceinline__ void transposed_sums(float (&v)[V], int idx) {
    static_assert(V % LANES == 0, "a whole number of values a lane");
    int half = V / 2;
#pragma unroll
    for (int w = LANES / 2; w > 0; w >>= 1) {
        const bool upper = idx & w;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if (i >= half) break;
            const float keep = upper ? v[i + half] : v[i];
            const float give = upper ? v[i] : v[i + half];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w * STRIDE);
        }
        half >>= 1;
    }
}

// What a chunk's block stages: delta, u and dy of its channels ([rows][kYS] each), B and C
// ([rows][4 L]).  Rows past t1 and channels past the group are zero: there a = 1 and every gradient
// is zero.  `row0`: rows of the first staged row in the arrays.
template <bool BF16, int L>
__device__ __forceinline__ void stage_bwd(const ScanBwdParams &p, int64_t t, int64_t t1, int g, int cbase, int row0,
                                          float *s_delta, float *s_u, float *s_dy, float *s_B, float *s_C) {
    using Tile = ScanTile<L>;
    constexpr int E = Tile::kE, YS = Tile::kYS;
    const int tid = threadIdx.x, DG = p.D / p.G;
    const int srow = tid / Tile::kTPR, scol = (tid % Tile::kTPR) * E;
    const int64_t sc = (int64_t)g * DG + cbase + scol;
    int left = DG - cbase - scol;
    left = left < 0 ? 0 : (left > E ? E : left);
    const int64_t tt = t + srow;
    const int v = tt < t1 ? left : 0;
    Piece<BF16, E> ru, rdt, rdo, rz;
    load_piece<BF16, E>(p.u, tt * p.D + sc, v, p.vec, ru);
    load_piece<BF16, E>(p.dt, tt * p.D + sc, v, p.vec, rdt);
    load_piece<BF16, E>(p.dout, tt * p.D + sc, v, p.vec, rdo);
    if (p.z) load_piece<BF16, E>(p.z, tt * p.D + sc, v, p.vec, rz);
    Piece<BF16, 4> rB[Tile::kQ], rC[Tile::kQ];
#pragma unroll
    for (int q = 0; q < Tile::kQ; ++q) {
        const int i = tid + q * kScanThreads;
        const int64_t tb = t + i / L;
        const int mm = 4 * (i % L);
        int v4 = p.n - mm;
        v4 = (i < Tile::kTT * L && tb < t1 && v4 > 0) ? (v4 > 4 ? 4 : v4) : 0;
        load_piece<BF16, 4>(p.B, (tb * p.G + g) * p.n + mm, v4, p.vecn, rB[q]);
        load_piece<BF16, 4>(p.C, (tb * p.G + g) * p.n + mm, v4, p.vecn, rC[q]);
    }
    float u[E], dt[E], dy[E];
    piece_to_f32<BF16, E>(ru, p.vec, u);
    piece_to_f32<BF16, E>(rdt, p.vec, dt);
    piece_to_f32<BF16, E>(rdo, p.vec, dy);
    if (p.z) {
        float z[E];
        piece_to_f32<BF16, E>(rz, p.vec, z);
#pragma unroll
        for (int i = 0; i < E; ++i) dy[i] *= silu(z[i]);
    }
    const int at = (row0 + srow) * YS + scol;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const bool in = i < v;
        s_delta[at + i] = in ? softplus(dt[i] + (p.dt_bias ? p.dt_bias[sc + i] : 0.f)) : 0.f;
        s_u[at + i] = u[i];
        s_dy[at + i] = in ? dy[i] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < Tile::kQ; ++q) {
        const int i = tid + q * kScanThreads;
        if (i < Tile::kTT * L) {
            float b[4], c[4];
            piece_to_f32<BF16, 4>(rB[q], p.vecn, b);
            piece_to_f32<BF16, 4>(rC[q], p.vecn, c);
            *reinterpret_cast<float4 *>(&s_B[row0 * 4 * L + 4 * i]) = make_float4(b[0], b[1], b[2], b[3]);
            *reinterpret_cast<float4 *>(&s_C[row0 * 4 * L + 4 * i]) = make_float4(c[0], c[1], c[2], c[3]);
        }
    }
}

template <bool BF16, int L>
__global__ void __launch_bounds__(kScanThreads) scan_bwd_chunk_kernel(const ScanBwdParams p) {
    using Tile = ScanBwdTile<L>;
    constexpr int TT = Tile::kTT, CH = Tile::kCH, YS = Tile::kYS;
    __shared__ float s_delta[TT * YS], s_u[TT * YS], s_dy[TT * YS];
    __shared__ __align__(16) float s_B[TT * 4 * L], s_C[TT * 4 * L];
    const int tid = threadIdx.x, ncb = p.G * p.cbg, cb = blockIdx.x % ncb;
    if (blockIdx.x == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    const int64_t rec = blockIdx.x / ncb;
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;
    int seq;
    int64_t j, t0, t1;
    bool last;
    if (!scan_segment(p.cu, p.num_seqs, p.total_tokens, Tile::kTC, rec, seq, j, t0, t1, last)) return;
    const int lane = tid % L, chl = tid / L, m0 = 4 * lane;
    const bool active = cbase + chl < DG;
    const int64_t c = (int64_t)g * DG + cbase + chl;
    float A2[4];
    load_decay(p.A_log, c, m0, p.n, active, A2);
    const f32x2 A01 = f2_pack(A2[0], A2[1]), A23 = f2_pack(A2[2], A2[3]);
    f32x2 h01 = 0ull, h23 = 0ull, r01 = 0ull, r23 = 0ull;
    f32x2 P01 = f2_splat(1.f), P23 = f2_splat(1.f);   // product of the decays so far
    float sum_delta = 0.f;
    for (int64_t t = t0; t < t1; t += TT) {
        if (t > t0) __syncthreads();
        stage_bwd<BF16, L>(p, t, t1, g, cbase, 0, s_delta, s_u, s_dy, s_B, s_C);
        __syncthreads();
        const int steps = static_cast<int>(min64(TT, t1 - t));
#pragma unroll 4
        for (int i = 0; i < steps; ++i) {
            const float d = s_delta[i * YS + chl], u = s_u[i * YS + chl], dy = s_dy[i * YS + chl];
            const float4 b = *reinterpret_cast<const float4 *>(&s_B[(i * L + lane) * 4]);
            const float4 cc = *reinterpret_cast<const float4 *>(&s_C[(i * L + lane) * 4]);
            const f32x2 dd = f2_splat(d), du = f2_splat(d * u), dyy = f2_splat(dy);
            float a0, a1, a2, a3;
            f2_unpack(f2_mul(A01, dd), a0, a1);
            f2_unpack(f2_mul(A23, dd), a2, a3);
            const f32x2 e01 = f2_pack(ex2_approx(a0), ex2_approx(a1)), e23 = f2_pack(ex2_approx(a2), ex2_approx(a3));
            h01 = f2_fma(e01, h01, f2_mul(du, f2_pack(b.x, b.y)));
            h23 = f2_fma(e23, h23, f2_mul(du, f2_pack(b.z, b.w)));
            P01 = f2_mul(P01, e01);
            P23 = f2_mul(P23, e23);
            r01 = f2_fma(P01, f2_mul(dyy, f2_pack(cc.x, cc.y)), r01);
            r23 = f2_fma(P23, f2_mul(dyy, f2_pack(cc.z, cc.w)), r23);
            sum_delta += d;
        }
    }
    if (!active) return;
    float h[4], r[4];
    f2_unpack(h01, h[0], h[1]);
    f2_unpack(h23, h[2], h[3]);
    f2_unpack(r01, r[0], r[1]);
    f2_unpack(r23, r[2], r[3]);
    const int64_t row = (rec * p.D + c) * p.n;
    store_quad(p.H + row, m0, p.n, p.vecn, h);
    store_quad(p.R + row, m0, p.n, p.vecn, r);
    if (lane == 0) p.sum_delta[rec * p.D + c] = sum_delta;
}

constexpr int kChainThreads = 128;
constexpr int kChainAhead = 8;   // records in flight

// grid: x = quads of [D, 4 L] in blocks of kChainThreads, y = sequence, z = direction (0: states forwards,
// 1: gradients backwards).  Every record's value is replaced by what comes into the chunk.
template <int L>
__global__ void __launch_bounds__(kChainThreads) scan_bwd_chain_kernel(const ScanBwdParams p) {
    constexpr int TC = ScanBwdTile<L>::kTC;
    const int64_t q = (int64_t)blockIdx.x * kChainThreads + threadIdx.x;
    const int64_t c = q / L;
    const int m0 = 4 * static_cast<int>(q % L);
    if (c >= p.D || m0 >= p.n) return;
    const bool back = blockIdx.z == 1;
    float A2[4];
    load_decay(p.A_log, c, m0, p.n, true, A2);
    for (int64_t seq = blockIdx.y; seq < p.num_seqs; seq += gridDim.y) {
        int64_t s0, s1;
        seq_span(p.cu, (int)seq, p.num_seqs, p.total_tokens, s0, s1);
        const int64_t base = s0 / TC + seq;
        int64_t count = (s1 - s0 + TC - 1) / TC;
        if (count < 1) count = 1;
        if (base + count > p.records) count = p.records - base;   // malformed cu_seqlens only
        float *X = back ? p.R : p.H;
        float cur[4] = {0.f, 0.f, 0.f, 0.f};
        const float *init = back ? p.dhN : p.h0;
        if (init) load_quad(init + (seq * p.D + c) * p.n, m0, p.n, p.vecn, cur);
        for (int64_t i0 = 0; i0 < count; i0 += kChainAhead) {
            float x[kChainAhead][4], sd[kChainAhead];
#pragma unroll
            for (int k = 0; k < kChainAhead; ++k) {
                const int64_t i = i0 + k;
                if (i >= count) break;
                const int64_t r = base + (back ? count - 1 - i : i);
                load_quad(X + (r * p.D + c) * p.n, m0, p.n, p.vecn, x[k]);
                sd[k] = p.sum_delta[r * p.D + c];
            }
#pragma unroll
            for (int k = 0; k < kChainAhead; ++k) {
                const int64_t i = i0 + k;
                if (i >= count) break;
                const int64_t r = base + (back ? count - 1 - i : i);
                store_quad(X + (r * p.D + c) * p.n, m0, p.n, p.vecn, cur);
#pragma unroll
                for (int w = 0; w < 4; ++w) cur[w] = fmaf(ex2_approx(A2[w] * sd[k]), cur[w], x[k][w]);
            }
        }
        if (back && p.dh0) store_quad(p.dh0 + (seq * p.D + c) * p.n, m0, p.n, p.vecn, cur);
    }
}

constexpr int kBack = 8;   // tokens recomputed into registers at once

template <int L>
struct ScanGradSmem {
    using Tile = ScanBwdTile<L>;
    static constexpr int kAct = Tile::kTC * Tile::kYS;                  // delta, u, dy
    static constexpr int kBC = Tile::kTC * 4 * L;                       // B, C
    static constexpr int kCkpt = Tile::kTC / kBack * 4 * kScanThreads;  // every eighth state
    static constexpr int kRed = 2 * (kScanThreads / 32) * kBack * 8 * L;   // two buffers of the warps' dB, dC rows
    static constexpr int kY = kAct > kRed ? kAct : kRed;                // the forward pass's outputs, then those rows
    static constexpr int kBytes = (3 * kAct + 2 * kBC + kCkpt + kY) * 4;
};

template <bool BF16, int L>
__global__ void __launch_bounds__(kScanThreads) scan_bwd_grad_kernel(const ScanBwdParams p) {
    using Tile = ScanBwdTile<L>;
    using SM = ScanGradSmem<L>;
    constexpr int TT = Tile::kTT, TC = Tile::kTC, CH = Tile::kCH, E = Tile::kE, YS = Tile::kYS;
    constexpr int KW = 32 / L;               // channels of a warp
    constexpr int TB = KW > 8 ? KW / 8 : 1;  // tokens whose dB, dC rows are summed over the warp at once
    constexpr int VPL = 8 * TB / KW;         // values of them a lane is left with
    constexpr int YB = L > kBack ? L : kBack;   // tokens whose outputs are summed over the states at once
    extern __shared__ __align__(16) float scan_smem[];
    float *s_delta = scan_smem, *s_u = s_delta + SM::kAct, *s_dy = s_u + SM::kAct;
    float *s_B = s_dy + SM::kAct, *s_C = s_B + SM::kBC;
    float4 *s_ckpt = reinterpret_cast<float4 *>(s_C + SM::kBC);
    float *s_y = s_C + SM::kBC + SM::kCkpt, *s_red = s_y;

    const int tid = threadIdx.x, ncb = p.G * p.cbg, cb = blockIdx.x % ncb;
    const int64_t rec = blockIdx.x / ncb;
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;
    const int lane = tid % L, chl = tid / L, m0 = 4 * lane, warp = tid / 32;
    const bool active = cbase + chl < DG;
    const int64_t c = (int64_t)g * DG + cbase + chl;
    const int64_t row = (rec * p.D + c) * p.n;
    int seq;
    int64_t j, t0, t1;
    bool last;
    if (!scan_segment(p.cu, p.num_seqs, p.total_tokens, TC, rec, seq, j, t0, t1, last)) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};   // a record without a chunk: nothing to the weights' sums
        if (active) {
            store_quad(p.H + row, m0, p.n, p.vecn, zero);
            if (lane == 0) p.pskip[rec * p.D + c] = p.pbias[rec * p.D + c] = 0.f;
        }
        return;
    }
    float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
    load_decay(p.A_log, c, m0, p.n, active, A2);
    if (active) {
        load_quad(p.H + row, m0, p.n, p.vecn, h);
        load_quad(p.R + row, m0, p.n, p.vecn, r);
    }
    const f32x2 A01 = f2_pack(A2[0], A2[1]), A23 = f2_pack(A2[2], A2[3]);
    f32x2 h01 = f2_pack(h[0], h[1]), h23 = f2_pack(h[2], h[3]);
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
        stage_bwd<BF16, L>(p, t0 + k * TT, t1, g, cbase, k * TT, s_delta, s_u, s_dy, s_B, s_C);
    __syncthreads();

    // forwards: every eighth state, and the outputs where the gate's gradient needs them
#pragma unroll 1
    for (int tb = 0; tb < TC; tb += YB) {
        float y[YB];
#pragma unroll
        for (int i = 0; i < YB; ++i) {
            if (i % kBack == 0) {
                float s[4];
                f2_unpack(h01, s[0], s[1]);
                f2_unpack(h23, s[2], s[3]);
                s_ckpt[(tb + i) / kBack * kScanThreads + tid] = make_float4(s[0], s[1], s[2], s[3]);
            }
            const float d = s_delta[(tb + i) * YS + chl], u = s_u[(tb + i) * YS + chl];
            const float4 b = *reinterpret_cast<const float4 *>(&s_B[((tb + i) * L + lane) * 4]);
            const float4 cc = *reinterpret_cast<const float4 *>(&s_C[((tb + i) * L + lane) * 4]);
            const f32x2 dd = f2_splat(d), du = f2_splat(d * u);
            float a0, a1, a2, a3;
            f2_unpack(f2_mul(A01, dd), a0, a1);
            f2_unpack(f2_mul(A23, dd), a2, a3);
            h01 = f2_fma(f2_pack(ex2_approx(a0), ex2_approx(a1)), h01, f2_mul(du, f2_pack(b.x, b.y)));
            h23 = f2_fma(f2_pack(ex2_approx(a2), ex2_approx(a3)), h23, f2_mul(du, f2_pack(b.z, b.w)));
            float lo, hi;
            f2_unpack(f2_fma(h23, f2_pack(cc.z, cc.w), f2_mul(h01, f2_pack(cc.x, cc.y))), lo, hi);
            y[i] = lo + hi;
        }
        if (p.z) {
            transposed_sums<YB, L, 1>(y, lane);
#pragma unroll
            for (int k = 0; k < YB / L; ++k) s_y[(tb + lane * (YB / L) + k) * YS + chl] = y[k];
        }
    }
    const int srow = tid / Tile::kTPR, scol = (tid % Tile::kTPR) * E;
    const int64_t sc = (int64_t)g * DG + cbase + scol;
    int left = DG - cbase - scol;
    left = left < 0 ? 0 : (left > E ? E : left);
    if (p.z) {
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int64_t tt = t0 + k * TT + srow;
            if (tt < t1 && left > 0) {
                Piece<BF16, E> rz, rdo;
                float z[E], o[E];
                load_piece<BF16, E>(p.z, tt * p.D + sc, left, p.vec, rz);
                load_piece<BF16, E>(p.dout, tt * p.D + sc, left, p.vec, rdo);
                piece_to_f32<BF16, E>(rz, p.vec, z);
                piece_to_f32<BF16, E>(rdo, p.vec, o);
                const int at = (k * TT + srow) * YS + scol;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float y = fmaf(i < left && p.skip ? p.skip[sc + i] : 0.f, s_u[at + i], s_y[at + i]);
                    const float s = sigmoid_fast(z[i]);
                    o[i] *= y * s * fmaf(z[i], 1.f - s, 1.f);
                }
                store_piece<BF16, E>(p.dz, tt * p.D + sc, left, p.vec, o);
            }
        }
        __syncthreads();   // s_red takes the place of s_y
    }

    // backwards
    const float skip = active && p.skip ? p.skip[c] : 0.f;
    f32x2 g01 = f2_pack(r[0], r[1]), g23 = f2_pack(r[2], r[3]);   // a_{t+1} g_{t+1}
    f32x2 dA01 = 0ull, dA23 = 0ull;
    float dskip = 0.f, dbias = 0.f;
#pragma unroll 1
    for (int sb = TC / kBack - 1; sb >= 0; --sb) {
        const int tb = sb * kBack;
        f32x2 a01[kBack], a23[kBack], p01[kBack], p23[kBack];   // a_t and a_t h_{t-1}
        {
            const float4 s = s_ckpt[sb * kScanThreads + tid];
            h01 = f2_pack(s.x, s.y);
            h23 = f2_pack(s.z, s.w);
        }
#pragma unroll
        for (int i = 0; i < kBack; ++i) {
            const float d = s_delta[(tb + i) * YS + chl], u = s_u[(tb + i) * YS + chl];
            const float4 b = *reinterpret_cast<const float4 *>(&s_B[((tb + i) * L + lane) * 4]);
            const f32x2 dd = f2_splat(d), du = f2_splat(d * u);
            float x0, x1, x2, x3;
            f2_unpack(f2_mul(A01, dd), x0, x1);
            f2_unpack(f2_mul(A23, dd), x2, x3);
            a01[i] = f2_pack(ex2_approx(x0), ex2_approx(x1));
            a23[i] = f2_pack(ex2_approx(x2), ex2_approx(x3));
            p01[i] = f2_mul(a01[i], h01);
            p23[i] = f2_mul(a23[i], h23);
            h01 = f2_fma(du, f2_pack(b.x, b.y), p01[i]);
            h23 = f2_fma(du, f2_pack(b.z, b.w), p23[i]);
        }
        float *red = s_red + (sb & 1) * ((kScanThreads / 32) * kBack * 8 * L) + warp * (kBack * 8 * L);
        float v[2 * kBack];
        float bc[8 * TB];
#pragma unroll
        for (int i = kBack - 1; i >= 0; --i) {
            const float d = s_delta[(tb + i) * YS + chl], u = s_u[(tb + i) * YS + chl], dy = s_dy[(tb + i) * YS + chl];
            const float4 b = *reinterpret_cast<const float4 *>(&s_B[((tb + i) * L + lane) * 4]);
            const float4 cc = *reinterpret_cast<const float4 *>(&s_C[((tb + i) * L + lane) * 4]);
            const f32x2 b01 = f2_pack(b.x, b.y), b23 = f2_pack(b.z, b.w);
            const f32x2 dd = f2_splat(d), du = f2_splat(d * u), dyy = f2_splat(dy);
            g01 = f2_fma(f2_pack(cc.x, cc.y), dyy, g01);
            g23 = f2_fma(f2_pack(cc.z, cc.w), dyy, g23);
            const f32x2 e01 = f2_mul(g01, p01[i]), e23 = f2_mul(g23, p23[i]);
            dA01 = f2_fma(e01, dd, dA01);
            dA23 = f2_fma(e23, dd, dA23);
            float lo, hi;
            f2_unpack(f2_fma(g23, b23, f2_mul(g01, b01)), lo, hi);
            v[2 * i] = lo + hi;
            f2_unpack(f2_fma(e23, A23, f2_mul(e01, A01)), lo, hi);
            v[2 * i + 1] = lo + hi;
            const int w = 8 * (i % TB);
            f2_unpack(f2_mul(g01, du), bc[w], bc[w + 1]);
            f2_unpack(f2_mul(g23, du), bc[w + 2], bc[w + 3]);
            f2_unpack(f2_mul(f2_fma(du, b01, p01[i]), dyy), bc[w + 4], bc[w + 5]);
            f2_unpack(f2_mul(f2_fma(du, b23, p23[i]), dyy), bc[w + 6], bc[w + 7]);
            g01 = f2_mul(a01[i], g01);
            g23 = f2_mul(a23[i], g23);
            if (i % TB == 0) {
                const int k = chl % KW;
                transposed_sums<8 * TB, KW, L>(bc, k);
                const int at = k * VPL;   // token at / 8 of the TB, value at % 8: dB (below 4) or dC of this lane's states
                float *dst = red + (i + at / 8) * (8 * L) + ((at % 8) / 4) * (4 * L) + m0 + at % 4;
#pragma unroll
                for (int x = 0; x < VPL; ++x) dst[x] = bc[x];
            }
        }
        // du and ddt in the place of u and delta: the lanes of a channel are in one warp and have read
        // both for these tokens
        transposed_sums<2 * kBack, L, 1>(v, lane);
        __syncwarp();
        auto finish = [&](int t, float dbu, float ddA) {
            const int at = t * YS + chl;
            const float d = s_delta[at], u = s_u[at], dy = s_dy[at];
            const float ddt = fmaf(u, dbu, 0.6931471805599453f * ddA) * -expm1f(-d);   // sigmoid(x) = 1 - exp(-softplus(x))
            s_u[at] = fmaf(d, dbu, skip * dy);
            s_delta[at] = ddt;
            dskip = fmaf(dy, u, dskip);
            dbias += ddt;
        };
        if constexpr (L <= kBack) {
#pragma unroll
            for (int k = 0; k < kBack / L; ++k) finish(tb + lane * (kBack / L) + k, v[2 * k], v[2 * k + 1]);
        } else {   // L = 16: one value a lane, a pair of lanes per token
            const float other = __shfl_xor_sync(0xffffffffu, v[0], 1);
            if ((lane & 1) == 0) finish(tb + lane / 2, v[0], other);
        }
        __syncthreads();
        // the block's dB and dC of these tokens (the other buffer takes the next ones meanwhile)
        const float *all = s_red + (sb & 1) * ((kScanThreads / 32) * kBack * 8 * L);
        for (int i = tid; i < kBack * 8 * L; i += kScanThreads) {
            const int t = tb + i / (8 * L), x = i % (8 * L), m = x % (4 * L);
            if (t0 + t < t1 && m < p.n) {
                float s = all[i];
#pragma unroll
                for (int w = 1; w < kScanThreads / 32; ++w) s += all[w * (kBack * 8 * L) + i];
                p.pBC[((int64_t)cb * p.total_tokens + t0 + t) * (2 * p.n) + (x / (4 * L)) * p.n + m] = s;
            }
        }
    }
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const int64_t tt = t0 + k * TT + srow;
        if (tt < t1 && left > 0) {
            float o[E];
            const int at = (k * TT + srow) * YS + scol;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = s_u[at + i];
            store_piece<BF16, E>(p.du, tt * p.D + sc, left, p.vec, o);
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = s_delta[at + i];
            store_piece<BF16, E>(p.ddt, tt * p.D + sc, left, p.vec, o);
        }
    }
#pragma unroll
    for (int w = L / 2; w > 0; w >>= 1) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, w);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, w);
    }
    if (active) {
        float e[4];
        f2_unpack(dA01, e[0], e[1]);
        f2_unpack(dA23, e[2], e[3]);
        store_quad(p.H + row, m0, p.n, p.vecn, e);   // read above by this thread
        if (lane == 0) {
            p.pskip[rec * p.D + c] = dskip;
            p.pbias[rec * p.D + c] = dbias;
        }
    }
}

// dB, dC: the sum over the channel blocks of a group
template <bool BF16>
__global__ void __launch_bounds__(256) scan_bwd_bc_kernel(const ScanBwdParams p) {
    const int64_t per_token = (int64_t)p.G * 2 * p.n;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.total_tokens * per_token) return;
    const int64_t t = i / per_token;
    const int x = static_cast<int>(i % per_token), g = x / (2 * p.n), w = x % (2 * p.n);
    const float *src = p.pBC + ((int64_t)g * p.cbg * p.total_tokens + t) * (2 * p.n) + w;
    const int64_t stride = p.total_tokens * 2 * p.n;
    float s = 0.f;
#pragma unroll 8
    for (int b = 0; b < p.cbg; ++b) s += __ldg(src + b * stride);
    store_out(w < p.n ? p.dB : p.dC, (t * p.G + g) * p.n + w % p.n, !BF16, s);
}

// dA_log, dskip and ddt_bias: column sums over the records.  32 columns a block, 8 rows at a time.
constexpr int kColRows = 8;
__global__ void __launch_bounds__(32 * kColRows) scan_bwd_weights_kernel(const ScanBwdParams p) {
    __shared__ float s_sum[kColRows][33];
    const int64_t nA = (int64_t)p.D * p.n;
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;   // [D n | D | D]
    float s = 0.f;
    if (col < nA + 2 * p.D) {
        const float *src;
        int64_t stride = p.D;
        if (col < nA) { src = p.H + col; stride = nA; }
        else if (col < nA + p.D) src = p.pskip + (col - nA);
        else src = p.pbias + (col - nA - p.D);
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < p.records; r += kColRows) s += src[r * stride];
    }
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || col >= nA + 2 * p.D) return;
#pragma unroll
    for (int k = 1; k < kColRows; ++k) s += s_sum[k][threadIdx.x];
    if (col < nA) p.dA_log[col] = -expf(p.A_log[col]) * s;
    else if (col < nA + p.D) { if (p.dskip) p.dskip[col - nA] = s; }
    else if (p.ddt_bias) p.ddt_bias[col - nA - p.D] = s;
}

}  // namespace kda
