// Layer norm over the last dimension and its gradients.
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy w, xh = (x - mean) rstd:  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: a row is read once into registers (RT threads, EK elements each), its statistics
// are taken there in two passes (the mean first, so that no difference of large sums is formed), and
// it is written from there.  Backwards each group of RT threads walks over rows with its columns'
// shares of dw and db in registers and leaves one row of partial sums; a second launch adds those in
// a fixed order.
#pragma once

#include "activations.cuh"
#include "conv_state.cuh"   // column_sum

namespace kda {

struct NormParams {
    const void *x, *dy;
    const float *w, *b;
    float *mean, *rstd;         // [rows]; written forwards, read backwards
    void *y;                    // y forwards, dx backwards
    float *part;                // [groups, 2, d] shares of dw and db
    int64_t rows;
    int d;
    float eps;
};

// elements of a thread: piece k is E consecutive columns (VEC), else E columns RT apart
template <int RT, int E, bool VEC>
__device__ __forceinline__ int norm_col(int k, int i, int lane) {
    return VEC ? (k * RT + lane) * E + i : (k * E + i) * RT + lane;
}

template <bool BF16, int RT, int E, int K, bool VEC>
__device__ __forceinline__ void norm_load(const void *p, int64_t row, int d, int lane, bool on, Piece<BF16, E> (&r)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = norm_col<RT, E, VEC>(k, 0, lane);
        load_piece<BF16, E, VEC>(p, row * d + c, !on || c >= d ? 0 : (VEC ? E : (d - c + RT - 1) / RT), r[k], VEC ? 1 : RT);
    }
}

template <bool BF16, int RT, int E, bool VEC>
__device__ __forceinline__ void norm_store(void *p, int64_t row, int d, int k, int lane, const float (&v)[E]) {
    const int c = norm_col<RT, E, VEC>(k, 0, lane);
    store_piece<BF16, E, VEC>(p, row * d + c, c >= d ? 0 : (VEC ? E : (d - c + RT - 1) / RT), v, VEC ? 1 : RT);
}

// Sum of N values over the RT threads of a group.  A group of more than one warp is a whole block;
// `buf` alternates between calls, so that one barrier a call is enough.
template <int RT, int N>
__device__ __forceinline__ void norm_sum(float (&v)[N], float *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (RT > 32) {
        constexpr int NW = RT / 32;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i * NW + threadIdx.x / 32] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v[i] += buf[i * NW + w];
        }
    }
}

template <int RT>
struct NormBlock {
    static constexpr int kThreads = RT < 128 ? 128 : RT;
    static constexpr int kGroups = kThreads / RT;   // rows a block works on at once
};

template <bool BF16, int RT, int EK, bool VEC>
__global__ void __launch_bounds__(NormBlock<RT>::kThreads) layer_norm_fwd_kernel(const NormParams p) {
    constexpr int E = BF16 ? 8 : 4, K = EK / E;
    __shared__ float s_sum[2][RT > 32 ? RT / 32 : 1];
    const int lane = threadIdx.x % RT;
    const int64_t row = (int64_t)blockIdx.x * NormBlock<RT>::kGroups + threadIdx.x / RT;
    const bool on = row < p.rows;
    Piece<BF16, E> r[K];
    norm_load<BF16, RT, E, K, VEC>(p.x, row, p.d, lane, on, r);
    float x[K][E], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        piece_to_f32<BF16, E, VEC>(r[k], x[k]);
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += x[k][i];
    }
    norm_sum<RT, 1>(s, s_sum[0]);
    const float mean = s[0] / p.d;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float c = x[k][i] - mean;
            if (norm_col<RT, E, VEC>(k, i, lane) < p.d) s[0] = fmaf(c, c, s[0]);
        }
    norm_sum<RT, 1>(s, s_sum[1]);
    const float rstd = 1.f / sqrtf(s[0] / p.d + p.eps);
    if (!on) return;
    if (lane == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = norm_col<RT, E, VEC>(k, i, lane);
            y[i] = c < p.d ? fmaf((x[k][i] - mean) * rstd, __ldg(p.w + c), p.b ? __ldg(p.b + c) : 0.f) : 0.f;
        }
        norm_store<BF16, RT, E, VEC>(p.y, row, p.d, k, lane, y);
    }
}

template <bool BF16, int RT, int EK, bool VEC>
__global__ void __launch_bounds__(NormBlock<RT>::kThreads) layer_norm_bwd_kernel(const NormParams p) {
    constexpr int E = BF16 ? 8 : 4, K = EK / E;
    __shared__ float s_sum[2][RT > 32 ? 2 * (RT / 32) : 1];
    const int lane = threadIdx.x % RT;
    const int64_t group = (int64_t)blockIdx.x * NormBlock<RT>::kGroups + threadIdx.x / RT;
    const int64_t groups = (int64_t)gridDim.x * NormBlock<RT>::kGroups;
    float w[K][E], dw[K][E], db[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = norm_col<RT, E, VEC>(k, i, lane);
            w[k][i] = c < p.d ? p.w[c] : 0.f;   // zero past d: nothing to the row's sums
            dw[k][i] = db[k][i] = 0.f;
        }
    Piece<BF16, E> rx[K], rd[K];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t row) {
        const bool on = row < p.rows;
        norm_load<BF16, RT, E, K, VEC>(p.x, row, p.d, lane, on, rx);
        norm_load<BF16, RT, E, K, VEC>(p.dy, row, p.d, lane, on, rd);
        mean = on ? p.mean[row] : 0.f;
        rstd = on ? p.rstd[row] : 0.f;
    };
    fetch(group);
    int flip = 0;
    // every group of a block takes the same number of turns (the sums hold barriers)
    const int64_t first = (int64_t)blockIdx.x * NormBlock<RT>::kGroups;
    for (int64_t row = group, lead = first; lead < p.rows; row += groups, lead += groups, flip ^= 1) {
        float xh[K][E], dy[K][E], s[2] = {0.f, 0.f};
        const float m = mean, rs = rstd;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            piece_to_f32<BF16, E, VEC>(rx[k], xh[k]);
            piece_to_f32<BF16, E, VEC>(rd[k], dy[k]);
        }
        if (lead + groups < p.rows) fetch(row + groups);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                xh[k][i] = (xh[k][i] - m) * rs;
                dw[k][i] = fmaf(dy[k][i], xh[k][i], dw[k][i]);
                db[k][i] += dy[k][i];
                dy[k][i] *= w[k][i];
                s[0] += dy[k][i];
                s[1] = fmaf(dy[k][i], xh[k][i], s[1]);
            }
        norm_sum<RT, 2>(s, s_sum[flip]);
        if (row < p.rows) {
            const float c0 = s[0] / p.d, c1 = s[1] / p.d;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dx[E];
#pragma unroll
                for (int i = 0; i < E; ++i) dx[i] = rs * (dy[k][i] - c0 - xh[k][i] * c1);
                norm_store<BF16, RT, E, VEC>(p.y, row, p.d, k, lane, dx);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = norm_col<RT, E, VEC>(k, i, lane);
            if (c < p.d) {
                p.part[group * 2 * p.d + c] = dw[k][i];
                p.part[group * 2 * p.d + p.d + c] = db[k][i];
            }
        }
}

__global__ void __launch_bounds__(32 * kSumRows) norm_weight_sum_kernel(const float *part, int64_t groups, int d, float *dw,
                                                                        float *db) {
    column_sum(part, groups, (int64_t)2 * d, [&](int64_t col, float s) {
        if (col < d) dw[col] = s;
        else if (db) db[col - d] = s;
    });
}

}  // namespace kda
