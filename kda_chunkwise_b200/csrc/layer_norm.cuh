// Layer norm over the last dimension and its gradients.
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy w, xh = (x - mean) rstd:  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory.  A group of RT threads (a block; a warp for short rows) walks over rows, EK elements
// of each in a thread's registers, so that a row is read once and its statistics are taken in two passes
// (the mean first: no difference of large sums).  The next rows are on their way into a ring in shared
// memory meanwhile, 16 bytes a copy, every thread reading back its own; the weights stay in registers.
// 8192 x 4096 in bf16: forward 25 us (134 MB, 5.4 TB/s, 0.82 of a copy), backward 43 to 45 us + 9 for the weights'
// sums, cold (201 MB, 4.5 to 4.7 TB/s, 0.68 to 0.71; two blocks an SM, one barrier a row).  Its registers do not hold everything of wide
// rows: 200 to 304 bytes a thread are spilled above 8192 columns, up to 24 in fp32 at 1025 to 4096 and in bf16 at 4097 to 8192.
// Backwards each group keeps its columns' shares of dw and db in registers and leaves one row of
// partial sums; a second launch adds those in a fixed order.
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

// The ring: stages of NT tensors' rows, as many as four while they fit; none (rows are then loaded when they
// are needed) for rows that are not whole vectors or do not fit three times.
template <bool BF16, int RT, int EK, bool VEC, int NT>
struct NormRing {
    static constexpr int kE = BF16 ? 8 : 4, kK = EK / kE;
    static constexpr int kStage = NT * kK * NormBlock<RT>::kThreads * 16;
    static constexpr int kStages = !VEC ? 0 : (4 * kStage <= 131072 ? 4 : (3 * kStage <= 196608 ? 3 : 0));
    static constexpr int kBytes = kStages * kStage;

    // tensor `which` of row `row` into the stage of turn `it` (zeros where there is no such row; past the row's end zeros,
    // or with FILL its first columns again)
    template <bool FILL = false>
    __device__ __forceinline__ static void copy(unsigned char *ring, int it, int which, const void *p, int64_t row, int d, int lane,
                                                bool on) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            int c = (k * RT + lane) * kE;
            const bool in = FILL ? on : on && c < d;
            if (FILL && c >= d) c = 0;
            cp_async_16(smem_u32(ring) + (((it % kStages) * NT + which) * kK + k) * (NormBlock<RT>::kThreads * 16) + threadIdx.x * 16,
                        static_cast<const char *>(p) + (in ? (row * d + c) * (BF16 ? 2 : 4) : 0), in ? 16 : 0);
        }
    }
    __device__ __forceinline__ static void read(const unsigned char *ring, int it, int which, float (&v)[kK][kE]) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const uint4 w = *reinterpret_cast<const uint4 *>(ring + (((it % kStages) * NT + which) * kK + k) * (NormBlock<RT>::kThreads * 16) +
                                                             threadIdx.x * 16);
            Piece<BF16, kE> r;
            r.w[0] = w.x; r.w[1] = w.y; r.w[2] = w.z; r.w[3] = w.w;
            piece_to_f32<BF16, kE, true>(r, v[k]);
        }
    }
};

// per-column weights of a thread's piece k: fp32 [d], zero past d
template <int RT, int E, bool VEC>
__device__ __forceinline__ void norm_weights(const float *w, int k, int lane, int d, float (&v)[E]) {
    const int c = norm_col<RT, E, VEC>(k, 0, lane);
    Piece<false, E> r;
    load_piece<false, E, VEC>(w, c, c >= d ? 0 : (VEC ? E : (d - c + RT - 1) / RT), r, VEC ? 1 : RT);
    piece_to_f32<false, E, VEC>(r, v);
}

template <bool BF16, int RT, int EK, bool VEC>
__global__ void __launch_bounds__(NormBlock<RT>::kThreads) layer_norm_fwd_kernel(const NormParams p) {
    using Ring = NormRing<BF16, RT, EK, VEC, 1>;
    constexpr int E = Ring::kE, K = Ring::kK, S = Ring::kStages;
    constexpr bool KEEP = EK <= 16;   // the weights stay in registers
    extern __shared__ __align__(16) unsigned char norm_ring[];
    __shared__ float s_sum[4][RT > 32 ? RT / 32 : 1];
    const int lane = threadIdx.x % RT;
    const int64_t first = (int64_t)blockIdx.x * NormBlock<RT>::kGroups, step = (int64_t)gridDim.x * NormBlock<RT>::kGroups;
    const int64_t row0 = first + threadIdx.x / RT;
    if constexpr (S > 0) {
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) {
            Ring::copy(norm_ring, i, 0, p.x, row0 + i * step, p.d, lane, row0 + i * step < p.rows);
            cp_async_commit();
        }
    }
    float w[KEEP ? K : 1][E], b[KEEP ? K : 1][E];
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            norm_weights<RT, E, VEC>(p.w, k, lane, p.d, w[k]);
            norm_weights<RT, E, VEC>(p.b, k, lane, p.b ? p.d : 0, b[k]);
        }
    }
    const float inv_d = 1.f / p.d;
    int it = 0;
    for (int64_t lead = first, row = row0; lead < p.rows; lead += step, row += step, ++it) {   // (every group of a block takes the same turns)
        const bool on = row < p.rows;
        float x[K][E], s[1] = {0.f};
        if constexpr (S > 0) {
            cp_async_wait_group<S - 2>();
            Ring::read(norm_ring, it, 0, x);
            const int64_t next = row + (S - 1) * step;
            Ring::copy(norm_ring, it + S - 1, 0, p.x, next, p.d, lane, next < p.rows);
            cp_async_commit();
        } else {
            Piece<BF16, E> r[K];
            norm_load<BF16, RT, E, K, VEC>(p.x, row, p.d, lane, on, r);
#pragma unroll
            for (int k = 0; k < K; ++k) piece_to_f32<BF16, E, VEC>(r[k], x[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) s[0] += x[k][i];
        norm_sum<RT, 1>(s, s_sum[2 * (it & 1)]);
        const float mean = s[0] * inv_d;
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                x[k][i] -= mean;
                if (VEC || norm_col<RT, E, VEC>(k, i, lane) < p.d) q = fmaf(x[k][i], x[k][i], q);
            }
            if (!VEC || norm_col<RT, E, VEC>(k, 0, lane) < p.d) s[0] += q;
        }
        norm_sum<RT, 1>(s, s_sum[2 * (it & 1) + 1]);
        const float rstd = 1.f / sqrtf(fmaf(s[0], inv_d, p.eps));
        if (!on) continue;
        if (lane == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float y[E], wv[E], bv[E];
            if constexpr (!KEEP) {
                norm_weights<RT, E, VEC>(p.w, k, lane, p.d, wv);
                norm_weights<RT, E, VEC>(p.b, k, lane, p.b ? p.d : 0, bv);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) y[i] = fmaf(x[k][i] * rstd, KEEP ? w[KEEP ? k : 0][i] : wv[i], KEEP ? b[KEEP ? k : 0][i] : bv[i]);
            norm_store<BF16, RT, E, VEC>(p.y, row, p.d, k, lane, y);
        }
    }
    if constexpr (S > 0) cp_async_wait_all();
}

template <bool BF16, int RT, int EK, bool VEC>
__global__ void __launch_bounds__(NormBlock<RT>::kThreads, RT == 256 ? 2 : 1) layer_norm_bwd_kernel(const NormParams p) {
    using Ring = NormRing<BF16, RT, EK, VEC, 2>;
    constexpr int E = Ring::kE, K = Ring::kK, S = Ring::kStages;
    extern __shared__ __align__(16) unsigned char norm_ring[];
    __shared__ float s_sum[2][RT > 32 ? 2 * (RT / 32) : 1];
    const int lane = threadIdx.x % RT;
    const int64_t first = (int64_t)blockIdx.x * NormBlock<RT>::kGroups, step = (int64_t)gridDim.x * NormBlock<RT>::kGroups;
    const int64_t group = first + threadIdx.x / RT;
    auto fetch = [&](int it) {
        if constexpr (S > 0) {
            const int64_t row = group + it * step;
            // (past the row's end the weight is zero, and xhat one of the row's own: no zero times an infinite mean rstd)
            Ring::template copy<true>(norm_ring, it, 0, p.x, row, p.d, lane, row < p.rows);
            Ring::template copy<true>(norm_ring, it, 1, p.dy, row, p.d, lane, row < p.rows);
            cp_async_commit();
        }
    };
    if constexpr (S > 0)
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) fetch(i);
    float dw[K][E], db[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int i = 0; i < E; ++i) dw[k][i] = db[k][i] = 0.f;
    }
    float mean = group < p.rows ? p.mean[group] : 0.f, rstd = group < p.rows ? p.rstd[group] : 0.f;
    const float inv_d = 1.f / p.d;
    int it = 0;
    for (int64_t row = group, lead = first; lead < p.rows; row += step, lead += step, ++it) {
        const bool on = row < p.rows;
        float xh[K][E], dy[K][E], s[2] = {0.f, 0.f};
        const float m = on ? mean : 0.f, rs = on ? rstd : 0.f;
        if constexpr (S > 0) {
            cp_async_wait_group<S - 2>();
            Ring::read(norm_ring, it, 0, xh);
            Ring::read(norm_ring, it, 1, dy);
            fetch(it + S - 1);
        } else {
            Piece<BF16, E> rx[K], rd[K];
            norm_load<BF16, RT, E, K, VEC>(p.x, row, p.d, lane, on, rx);
            norm_load<BF16, RT, E, K, VEC>(p.dy, row, p.d, lane, on, rd);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                piece_to_f32<BF16, E, VEC>(rx[k], xh[k]);
                piece_to_f32<BF16, E, VEC>(rd[k], dy[k]);
            }
        }
        if (row + step < p.rows) {
            mean = p.mean[row + step];
            rstd = p.rstd[row + step];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float wv[E];   // (read again each row: the registers do more for occupancy)
            norm_weights<RT, E, VEC>(p.w, k, lane, p.d, wv);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                xh[k][i] = (xh[k][i] - m) * (S > 0 || norm_col<RT, E, VEC>(k, i, lane) < p.d ? rs : 0.f);
                dw[k][i] = fmaf(dy[k][i], xh[k][i], dw[k][i]);
                db[k][i] += dy[k][i];
                dy[k][i] *= wv[i];   // zero past d: nothing to the row's sums
                s[0] += dy[k][i];
                s[1] = fmaf(dy[k][i], xh[k][i], s[1]);
            }
        }
        norm_sum<RT, 2>(s, s_sum[it & 1]);
        if (on) {
            const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dx[E];
#pragma unroll
                for (int i = 0; i < E; ++i) dx[i] = rs * (dy[k][i] - c0 - xh[k][i] * c1);
                norm_store<BF16, RT, E, VEC>(p.y, row, p.d, k, lane, dx);
            }
        }
    }
    if constexpr (S > 0) cp_async_wait_all();
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
