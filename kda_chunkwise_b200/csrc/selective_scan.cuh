// Selective state space scan: prompts (packed sequences) and single tokens.
//
// Per channel d with n states, delta = softplus(dt + dt_bias), A = -exp(A_log):
//   h_t[m] = exp(delta_t A[m]) h_{t-1}[m] + delta_t u_t B_t[m]
//   out_t  = silu(z_t) (sum_m C_t[m] h_t[m] + skip u_t)
// B and C are shared by the D / G channels of a group.
//
// A prompt takes T D n exponentials and about seven times as many fp32 operations on 4 T D
// activations: the exponential unit (16 a clock and SM) bounds it, not memory.  So nothing is
// computed twice that takes an exponential, states stay in registers, and what is per (token,
// channel) (softplus, the gate) is done once by the thread that stages the value, not once per state.
//   - A channel's n states lie on L = 2^ceil(log2(n / 4)) lanes, four to a lane; a block of 128 threads
//     holds 128 / L channels of one group over one segment of one sequence, in tiles of kTT tokens.
//   - The next tile's activations are in flight in registers while a tile is scanned.
//   - The sum over m is taken for L tokens at once (transposed_sum): one value a lane.
// Sequences longer than seg_len tokens are cut into segments where the channels alone would leave
// the GPU empty: a first launch finds every segment's end state from zero and its sum of delta (the
// decay over a segment is exp(A sum delta)), the second joins those before its own and scans.
#pragma once

#include "activations.cuh"
#include "f32x2.cuh"

namespace kda {

constexpr int kScanThreads = 128;

template <int L>
struct ScanTile {
    static constexpr int kCH = kScanThreads / L;             // channels of a block
    static constexpr int kTT = L <= 4 ? 8 * L : 32;          // tokens of a tile
    static constexpr int kE = kTT * kCH / kScanThreads;      // elements of a tile per thread and tensor
    static constexpr int kTPR = kCH / kE;                    // threads that stage one row
    static constexpr int kQ = (kTT * L + kScanThreads - 1) / kScanThreads;   // quads of B (and C) a thread stages
    static constexpr int kYS = kCH + 32 / L;                 // row stride of the output tile: the lanes' rows fall on different banks
};

struct ScanParams {
    const void *u, *dt, *z, *B, *C;     // [T, D], [T, D], [T, D] or null, [T, G, n] x 2
    const float *A_log, *skip, *dt_bias;  // [D, n], [D] or null, [D] or null
    const int32_t *cu;                  // [num_seqs + 1]
    const float *h0;                    // [num_seqs, D, n] or null
    float *hN;                          // [num_seqs, D, n] or null
    void *out;                          // [T, D]
    float *seg_h;                       // [records, D, n] end state of a segment from a zero state (first segment: from h0)
    float *seg_delta;                   // [records, D] sum of delta over a segment
    float *seg_h0;                      // [num_seqs, D, n] copy of h0 for the second launch, so that hN may be h0
    int64_t total_tokens;
    int num_seqs, D, n, G;
    int cbg;                            // channel blocks of a group
    int64_t seg_len;
    bool vec;                           // rows of u, dt, z and out start on kE-element boundaries
    bool vecn;                          // n is a multiple of four
};

// The segment that record `rec` stands for: record base(s) + j, base(s) = cu[s] / seg_len + s, is the
// j-th segment of sequence s (an empty sequence has one, empty).  False if there is none.
__device__ __forceinline__ bool scan_segment(const int32_t *cu, int num_seqs, int64_t total, int64_t seg_len, int64_t rec,
                                             int &seq, int64_t &j, int64_t &t0, int64_t &t1, bool &last) {
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        int64_t c = cu[mid];
        c = c < 0 ? 0 : (c > total ? total : c);
        if (c / seg_len + mid <= rec) lo = mid;
        else hi = mid;
    }
    int64_t s0, s1;
    seq_span(cu, lo, num_seqs, total, s0, s1);
    seq = lo;
    j = rec - (s0 / seg_len + lo);
    if (j < 0) return false;
    t0 = s0 + j * seg_len;
    if (t0 >= s1 && j > 0) return false;
    t1 = min64(t0 + seg_len, s1);
    last = t1 == s1;
    return true;
}

// four states (or weights) of one channel from column m0 on; those past n are zero
__device__ __forceinline__ void load_quad(const float *row, int m0, int n, bool vecn, float (&v)[4]) {
    if (vecn) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m0 < n) x = *reinterpret_cast<const float4 *>(row + m0);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = m0 + i < n ? row[m0 + i] : 0.f;
    }
}

__device__ __forceinline__ void store_quad(float *row, int m0, int n, bool vecn, const float (&v)[4]) {
    if (vecn) {
        if (m0 < n) *reinterpret_cast<float4 *>(row + m0) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m0 + i < n) row[m0 + i] = v[i];
    }
}

// A log2(e) for four states; zero past n (a decay of one on states that stay zero)
__device__ __forceinline__ void load_decay(const float *A_log, int64_t c, int m0, int n, bool active, float (&A2)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = active && m0 + i < n ? -1.4426950408889634f * expf(A_log[c * n + m0 + i]) : 0.f;
}

__device__ __forceinline__ float silu(float x) { return x * sigmoid_fast(x); }

template <bool BF16, int L, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads) scan_fwd_kernel(const ScanParams p) {
    using Tile = ScanTile<L>;
    constexpr int CH = Tile::kCH, TT = Tile::kTT, E = Tile::kE, Q = Tile::kQ, YS = Tile::kYS;
    __shared__ float4 s_d[TT * CH];                       // delta, delta, delta u, delta u
    __shared__ __align__(16) float s_B[TT * 4 * L], s_C[SUMMARY ? 4 : TT * 4 * L];
    __shared__ float s_y[SUMMARY ? 1 : TT * YS];

    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && !SUMMARY) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    const int ncb = p.G * p.cbg;
    const int64_t rec = blockIdx.x / ncb;
    const int cb = blockIdx.x % ncb;
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;   // first channel of the block within its group
    int seq;
    int64_t j, t0, t1;
    bool last;
    if (!scan_segment(p.cu, p.num_seqs, p.total_tokens, p.seg_len, rec, seq, j, t0, t1, last)) return;
    if (SUMMARY && last) return;

    // scan role: channel and states of this thread
    const int lane = tid % L, chl = tid / L, m0 = 4 * lane;
    const bool active = cbase + chl < DG;
    const int64_t c = (int64_t)g * DG + cbase + chl;
    const int64_t row_s = ((int64_t)seq * p.D + c) * p.n;
    float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f};
    load_decay(p.A_log, c, m0, p.n, active, A2);
    if (active) {
        if (j == 0) {
            // with several segments, hN of the last one may be written over h0 while this block runs
            const float *src = (SUMMARY || last) ? p.h0 : p.seg_h0;
            if (p.h0) load_quad(src + row_s, m0, p.n, p.vecn, h);
            if (SUMMARY && p.h0) store_quad(p.seg_h0 + row_s, m0, p.n, p.vecn, h);
        } else if (!SUMMARY) {   // join the segments before this one
            for (int64_t i = 0; i < j; ++i) {
                const int64_t r = rec - j + i;
                float e[4];
                load_quad(p.seg_h + (r * p.D + c) * p.n, m0, p.n, p.vecn, e);
                const float sum = p.seg_delta[r * p.D + c];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = fmaf(i > 0 ? ex2_approx(A2[k] * sum) : 0.f, h[k], e[k]);
            }
        }
    }
    f32x2 A01 = f2_pack(A2[0], A2[1]), A23 = f2_pack(A2[2], A2[3]);
    f32x2 h01 = f2_pack(h[0], h[1]), h23 = f2_pack(h[2], h[3]);
    float sum_delta = 0.f;

    // staging role: E consecutive channels of one row of a tile
    const int srow = tid / Tile::kTPR, scol = (tid % Tile::kTPR) * E;
    const int64_t sc = (int64_t)g * DG + cbase + scol;
    int left = DG - cbase - scol;
    left = left < 0 ? 0 : (left > E ? E : left);
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = i < left && p.dt_bias ? p.dt_bias[sc + i] : 0.f;
        skip[i] = !SUMMARY && i < left && p.skip ? p.skip[sc + i] : 0.f;
    }
    Piece<BF16, E> ru, rdt, rz;
    Piece<BF16, 4> rB[Q], rC[SUMMARY ? 1 : Q];
    auto fetch = [&](int64_t t) {
        const int64_t tt = t + srow;
        const int v = tt < t1 ? left : 0;
        load_piece<BF16, E>(p.u, tt * p.D + sc, v, p.vec, ru);
        load_piece<BF16, E>(p.dt, tt * p.D + sc, v, p.vec, rdt);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int i = tid + q * kScanThreads;   // row i / L, states 4 (i % L) ..
            const int64_t tb = t + i / L;
            const int mm = 4 * (i % L);
            int v4 = p.n - mm;
            v4 = (i < TT * L && tb < t1 && v4 > 0) ? (v4 > 4 ? 4 : v4) : 0;
            load_piece<BF16, 4>(p.B, (tb * p.G + g) * p.n + mm, v4, p.vecn, rB[q]);
            if constexpr (!SUMMARY) load_piece<BF16, 4>(p.C, (tb * p.G + g) * p.n + mm, v4, p.vecn, rC[q]);
        }
    };

    fetch(t0);
    for (int64_t t = t0; t < t1; t += TT) {
        // stage the tile
        float u[E];
        {
            float dt[E];
            piece_to_f32<BF16, E>(ru, p.vec, u);
            piece_to_f32<BF16, E>(rdt, p.vec, dt);
            const bool row_in = t + srow < t1;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float d = row_in && i < left ? softplus(dt[i] + bias[i]) : 0.f;   // zero: the state passes unchanged
                s_d[srow * CH + scol + i] = make_float4(d, d, d * u[i], d * u[i]);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = tid + q * kScanThreads;
                if (i < TT * L) {
                    float v[4];
                    piece_to_f32<BF16, 4>(rB[q], p.vecn, v);
                    *reinterpret_cast<float4 *>(&s_B[4 * i]) = make_float4(v[0], v[1], v[2], v[3]);
                    if constexpr (!SUMMARY) {
                        piece_to_f32<BF16, 4>(rC[q], p.vecn, v);
                        *reinterpret_cast<float4 *>(&s_C[4 * i]) = make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
        }
        __syncthreads();
        if constexpr (!SUMMARY)
            if (p.z) load_piece<BF16, E>(p.z, (t + srow) * p.D + sc, t + srow < t1 ? left : 0, p.vec, rz);
        if (t + TT < t1) fetch(t + TT);

        const int steps = static_cast<int>(min64(TT, t1 - t));
        for (int tb = 0; tb < steps; tb += L) {
            float y[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const float4 d = s_d[(tb + i) * CH + chl];
                const float4 b = *reinterpret_cast<const float4 *>(&s_B[((tb + i) * L + lane) * 4]);
                const f32x2 dd = f2_pack(d.x, d.y), du = f2_pack(d.z, d.w);
                float a0, a1, a2, a3;
                f2_unpack(f2_mul(A01, dd), a0, a1);
                f2_unpack(f2_mul(A23, dd), a2, a3);
                const f32x2 e01 = f2_pack(ex2_approx(a0), ex2_approx(a1)), e23 = f2_pack(ex2_approx(a2), ex2_approx(a3));
                h01 = f2_fma(e01, h01, f2_mul(du, f2_pack(b.x, b.y)));
                h23 = f2_fma(e23, h23, f2_mul(du, f2_pack(b.z, b.w)));
                if constexpr (SUMMARY) {
                    sum_delta += d.x;
                } else {
                    const float4 cc = *reinterpret_cast<const float4 *>(&s_C[((tb + i) * L + lane) * 4]);
                    float lo, hi;
                    f2_unpack(f2_fma(h23, f2_pack(cc.z, cc.w), f2_mul(h01, f2_pack(cc.x, cc.y))), lo, hi);
                    y[i] = lo + hi;
                }
            }
            if constexpr (!SUMMARY) s_y[(tb + lane) * YS + chl] = transposed_sum<L>(y, lane);
        }
        __syncthreads();
        if constexpr (!SUMMARY) {
            if (t + srow < t1 && left > 0) {
                float o[E], z[E];
                if (p.z) piece_to_f32<BF16, E>(rz, p.vec, z);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    o[i] = fmaf(skip[i], u[i], s_y[srow * YS + scol + i]);
                    if (p.z) o[i] *= silu(z[i]);
                }
                store_piece<BF16, E>(p.out, (t + srow) * p.D + sc, left, p.vec, o);
            }
        }
    }

    f2_unpack(h01, h[0], h[1]);
    f2_unpack(h23, h[2], h[3]);
    if (!active) return;
    if constexpr (SUMMARY) {
        store_quad(p.seg_h + (rec * p.D + c) * p.n, m0, p.n, p.vecn, h);
        if (lane == 0) p.seg_delta[rec * p.D + c] = sum_delta;
    } else {
        if (last && p.hN) store_quad(p.hN + row_s, m0, p.n, p.vecn, h);
    }
}

// ---- single tokens ------------------------------------------------------------------------------

struct ScanStepParams {
    const void *u, *dt, *z, *B, *C;       // [N, D], [N, D], [N, D] or null, [N, G, n] x 2
    const float *A_log, *skip, *dt_bias;
    float *state;                         // [N, D, n], in place
    void *out;                            // [N, D]
    int N, D, n, G;
    bool vecn;
};

constexpr int kScanStepThreads = 256;

// One token of N states: the state is read once and written once (0.9 flop a byte), so the kernel
// streams it.  A thread owns four states of one channel (16 bytes), in U rows of the batch at once so
// that enough loads are in flight; the decay's weights are read once for the U rows.
template <bool BF16, int L, int U>
__global__ void __launch_bounds__(kScanStepThreads) scan_step_kernel(const ScanStepParams p) {
    const int64_t q = (int64_t)blockIdx.x * kScanStepThreads + threadIdx.x;   // quad of a row of the batch
    const int lane = static_cast<int>(q % L), m0 = 4 * lane;
    const int64_t c = q / L;
    const bool active = c < p.D;   // the L lanes of a channel agree
    const int g = active ? static_cast<int>(c / (p.D / p.G)) : 0;
    float A2[4];
    load_decay(p.A_log, c, m0, p.n, active, A2);
    const float bias = active && p.dt_bias ? p.dt_bias[c] : 0.f, skip = active && p.skip ? p.skip[c] : 0.f;
    int v4 = p.n - m0;
    v4 = active && v4 > 0 ? (v4 > 4 ? 4 : v4) : 0;
    for (int64_t r0 = (int64_t)blockIdx.y * U; r0 < p.N; r0 += (int64_t)gridDim.y * U) {
        float h[U][4], u[U], dt[U], z[U];
        Piece<BF16, 4> B[U], C[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t r = r0 + k;
            const bool on = active && r < p.N;
            h[k][0] = h[k][1] = h[k][2] = h[k][3] = 0.f;
            if (on) {
                if (p.vecn) {
                    if (m0 < p.n) {
                        const float4 x = __ldcs(reinterpret_cast<const float4 *>(p.state + (r * p.D + c) * p.n + m0));
                        h[k][0] = x.x; h[k][1] = x.y; h[k][2] = x.z; h[k][3] = x.w;
                    }
                } else {
                    load_quad(p.state + (r * p.D + c) * p.n, m0, p.n, false, h[k]);
                }
            }
            u[k] = on ? load_elem<BF16>(p.u, r * p.D + c) : 0.f;
            dt[k] = on ? load_elem<BF16>(p.dt, r * p.D + c) : 0.f;
            z[k] = on && p.z ? load_elem<BF16>(p.z, r * p.D + c) : 0.f;
            load_piece<BF16, 4>(p.B, (r * p.G + g) * p.n + m0, on ? v4 : 0, p.vecn, B[k]);
            load_piece<BF16, 4>(p.C, (r * p.G + g) * p.n + m0, on ? v4 : 0, p.vecn, C[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t r = r0 + k;
            const bool on = active && r < p.N;
            const float d = softplus(dt[k] + bias), du = d * u[k];
            float b[4], cc[4], y = 0.f;
            piece_to_f32<BF16, 4>(B[k], p.vecn, b);
            piece_to_f32<BF16, 4>(C[k], p.vecn, cc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[k][i] = fmaf(ex2_approx(A2[i] * d), h[k][i], du * b[i]);
                y = fmaf(h[k][i], cc[i], y);
            }
#pragma unroll
            for (int w = L / 2; w > 0; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
            if (!on) continue;
            if (p.vecn) {
                if (m0 < p.n)
                    __stcs(reinterpret_cast<float4 *>(p.state + (r * p.D + c) * p.n + m0),
                           make_float4(h[k][0], h[k][1], h[k][2], h[k][3]));
            } else {
                store_quad(p.state + (r * p.D + c) * p.n, m0, p.n, false, h[k]);
            }
            if (lane == 0) {
                y = fmaf(skip, u[k], y);
                if (p.z) y *= silu(z[k]);
                store_out(p.out, r * p.D + c, !BF16, y);
            }
        }
    }
}

}  // namespace kda
