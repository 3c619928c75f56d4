// The short causal convolution with its carried window: prompts that continue, single tokens and
// gradients (preprocess.cuh holds the stateless form).
//
//   p_t[c] = bias[c] + sum_{j < W} w[c][j] x_{t-(W-1)+j}[c]      (x before a sequence: its carried state)
//   s = silu(p) or p;   y = s, or s / sqrt(|s|^2 + 1e-12) over the head's channels
// The carried state is the last W - 1 inputs, [num_seqs, W - 1, C] in the inputs' type, oldest first.
//
// All three are bound by memory (about 10 flops a byte at most): each input is read once, its
// neighbours in time come from registers, and a thread keeps several rows in flight, in a ring in shared
// memory that it alone reads.  A thread owns E channels: consecutive ones, moved as one vector, where the
// rows allow it, else channels a block apart, so that single elements are still read side by side (and
// then a batch of rows in registers).
#pragma once

#include "activations.cuh"
#include "preprocess.cuh"

namespace kda {

constexpr int kConvThreads = 128;

struct ConvStateParams {
    const void *x, *dy;                 // [T, C]
    const float *w, *bias;              // [C, W], [C] or null
    const int32_t *cu;
    const void *h0, *dhN;               // [num_seqs, W - 1, C] or null
    void *y, *hN;                       // y: the output (forward) or dx (backward)
    void *dh0;
    float *part;                        // [runs, W + 1, C] the run's share of dw and dbias (backward)
    int64_t total_tokens, run_len, runs, first_block;
    int num_seqs, C, d;
    bool silu, l2norm;
};

// The channels of a thread: c0 + i step (VEC: consecutive, moved as vectors).
template <bool BF16, int E, bool VEC>
struct ChannelGroup {
    int64_t c0;
    static constexpr int step = VEC ? 1 : kConvThreads;
    int count;   // how many of the E are channels

    __device__ __forceinline__ ChannelGroup(int64_t block, int C) {
        c0 = block * kConvThreads * E + (VEC ? (int64_t)threadIdx.x * E : threadIdx.x);
        const int64_t n = c0 < C ? (C - c0 + step - 1) / step : 0;
        count = static_cast<int>(n > E ? E : n);
    }
    template <bool RO = true>
    __device__ __forceinline__ void load(const void *p, int64_t row, bool on, Piece<BF16, E> &r) const {
        load_piece<BF16, E, VEC, RO>(p, row + c0, on ? count : 0, r, step);
    }
    // one row's vector into this thread's place of a ring slot, and back (VEC only)
    static constexpr int kVec = E * (BF16 ? 2 : 4);   // bytes: 8 or 16
    __device__ __forceinline__ void copy(unsigned char *slot, const void *p, int64_t row, bool on) const {
        const bool in = on && count > 0;
        const char *src = static_cast<const char *>(p) + (in ? (row + c0) * (BF16 ? 2 : 4) : 0);
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(smem_u32(slot) + threadIdx.x * kVec), "l"(src),
                     "n"(kVec), "r"(in ? kVec : 0) : "memory");
    }
    __device__ __forceinline__ void read(const unsigned char *slot, float (&v)[E]) const {
        Piece<BF16, E> r;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(slot + threadIdx.x * kVec);
        if constexpr (kVec == 16) {
            const uint4 x = *reinterpret_cast<const uint4 *>(w);
            r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(w);
            r.w[0] = x.x; r.w[1] = x.y;
        }
        get(r, v);
    }
    __device__ __forceinline__ void get(const Piece<BF16, E> &r, float (&v)[E]) const { piece_to_f32<BF16, E, VEC>(r, v); }
    template <bool RO = true>
    __device__ __forceinline__ void load_f32(const void *p, int64_t row, bool on, float (&v)[E]) const {
        Piece<BF16, E> r;
        load<RO>(p, row, on, r);
        get(r, v);
    }
    __device__ __forceinline__ void store(void *p, int64_t row, const float (&v)[E]) const {
        store_piece<BF16, E, VEC>(p, row + c0, count, v, step);
    }
};

// The taps of a thread's channels: W floats of a channel lie together, so that four taps are one load.
template <int W, int E, class Group>
__device__ __forceinline__ void load_taps(const ConvStateParams &p, const Group &cg, float (&w)[W][E], float (&bias)[E]) {
    const bool whole = (reinterpret_cast<uintptr_t>(p.w) & (W * 4 - 1)) == 0;   // (a power of two where it matters)
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int64_t c = cg.c0 + i * cg.step;
        const bool on = i < cg.count;
        bias[i] = on && p.bias ? __ldg(p.bias + c) : 0.f;
        uint32_t r[W];
#pragma unroll
        for (int j = 0; j < W; ++j) r[j] = 0u;
        if constexpr (W == 2 || W == 4) {
            if (whole) {
                load_if<W * 4, true>(p.w + c * W, on, r);
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][i] = __uint_as_float(r[j]);
                continue;
            }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = on ? __ldg(p.w + c * W + j) : 0.f;
    }
}

// sum over the lanes of one head (d / E lanes of a warp)
__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One row's output from its window (xw[0] oldest) and input.
template <int W, int E>
__device__ __forceinline__ void conv_row(const ConvStateParams &p, const float (&w)[W][E], const float (&bias)[E],
                                         const float (&xw)[W > 1 ? W - 1 : 1][E], const float (&x)[E], float (&y)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float a = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][i], xw[j][i], a);
        a = fmaf(w[W - 1][i], x[i], a);
        y[i] = p.silu ? a * sigmoid_fast(a) : a;
    }
    if (p.l2norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(y[i], y[i], ss);
        const float inv = rsqrtf(head_sum(ss, p.d / E) + 1e-12f);
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] *= inv;
    }
}

template <int W, int E>
__device__ __forceinline__ void slide(float (&xw)[W > 1 ? W - 1 : 1][E], const float (&x)[E]) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) xw[j][i] = xw[j + 1][i];
    if (W > 1)
#pragma unroll
        for (int i = 0; i < E; ++i) xw[W > 1 ? W - 2 : 0][i] = x[i];
}

// The window before token t of a sequence starting at s0: inputs, or rows of its carried state.
template <int W, int E, class Group>
__device__ __forceinline__ void load_window(const ConvStateParams &p, const Group &cg, int64_t t, int64_t s0,
                                            int64_t seq, float (&xw)[W > 1 ? W - 1 : 1][E]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t tt = t - (W - 1) + j;
        if (tt >= s0) cg.load_f32(p.x, tt * p.C, true, xw[j]);
        else {   // a row below zero only where cu_seqlens is malformed
            const int64_t r = tt - s0 + W - 1;
            cg.template load_f32<false>(p.h0, (seq * (W - 1) + r) * p.C, p.h0 != nullptr && r >= 0, xw[j]);
        }
    }
}

constexpr int kConvRows = 8;   // rows in flight per thread

// grid: x = runs of run_len tokens, then one block per sequence for the final states; y = blocks of
// channels.  With hN = h0 the two are separate launches (first_block skips the runs).
template <bool BF16, int W, int E, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_state_fwd_kernel(const ConvStateParams p) {
    const ChannelGroup<BF16, E, VEC> cg(blockIdx.y, p.C);
    constexpr int SLOT = kConvThreads * ChannelGroup<BF16, E, VEC>::kVec;
    __shared__ __align__(16) unsigned char ring[VEC ? kConvRows * SLOT : 16];
    const int64_t bx = p.first_block + blockIdx.x;
    if (bx == 0 && blockIdx.y == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    float xw[W > 1 ? W - 1 : 1][E];
    if (bx >= p.runs) {   // the state after a sequence: its last W - 1 inputs, all read before any is written
        const int64_t seq = bx - p.runs;
        int64_t s0, s1;
        seq_span(p.cu, (int)seq, p.num_seqs, p.total_tokens, s0, s1);
        load_window<W, E>(p, cg, s1, s0, seq, xw);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) cg.store(p.hN, (seq * (W - 1) + j) * p.C, xw[j]);
        return;
    }
    const int64_t r0 = bx * p.run_len, r1 = min64(r0 + p.run_len, p.total_tokens);
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < kConvRows; ++k) {
            cg.copy(ring + k * SLOT, p.x, (r0 + k) * p.C, r0 + k < r1);
            cp_async_commit();
        }
    }
    float w[W][E], bias[E];
    load_taps<W, E>(p, cg, w, bias);
    int64_t seq = seq_of(p.cu, p.num_seqs, r0), s0, s1;
    seq_span(p.cu, (int)seq, p.num_seqs, p.total_tokens, s0, s1);
    load_window<W, E>(p, cg, r0, s0, seq, xw);
    for (int64_t t0 = r0; t0 < r1; t0 += kConvRows) {
        Piece<BF16, E> rx[VEC ? 1 : kConvRows];
        if constexpr (!VEC) {
#pragma unroll
            for (int k = 0; k < kConvRows; ++k) cg.load(p.x, (t0 + k) * p.C, t0 + k < r1, rx[k]);
        }
#pragma unroll
        for (int k = 0; k < kConvRows; ++k) {
            const int64_t t = t0 + k;
            if (t >= r1) break;
            float x[E], y[E];
            if constexpr (VEC) {
                cp_async_wait_group<kConvRows - 1>();
                cg.read(ring + k * SLOT, x);
                cg.copy(ring + k * SLOT, p.x, (t + kConvRows) * p.C, t + kConvRows < r1);
                cp_async_commit();
            } else {
                cg.get(rx[k], x);
            }
            if (t >= s1 && seq + 1 < p.num_seqs) {   // the next sequence that has tokens starts here
                do seq_span(p.cu, (int)++seq, p.num_seqs, p.total_tokens, s0, s1);
                while (t >= s1 && seq + 1 < p.num_seqs);
                load_window<W, E>(p, cg, t, t, seq, xw);
            }
            conv_row<W, E>(p, w, bias, xw, x, y);
            cg.store(p.y, t * p.C, y);
            slide<W, E>(xw, x);
        }
    }
    cp_async_wait_all();
}

// One token of num_seqs sequences; the state (hN) in place.
template <bool BF16, int W, int E, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvStateParams p) {
    const ChannelGroup<BF16, E, VEC> cg(blockIdx.y, p.C);
    float w[W][E], bias[E];
    load_taps<W, E>(p, cg, w, bias);
    for (int64_t r = blockIdx.x; r < p.num_seqs; r += gridDim.x) {
        float xw[W > 1 ? W - 1 : 1][E], x[E], y[E];
        cg.load_f32(p.x, r * p.C, true, x);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) cg.template load_f32<false>(p.h0, (r * (W - 1) + j) * p.C, true, xw[j]);
        conv_row<W, E>(p, w, bias, xw, x, y);
        slide<W, E>(xw, x);
        cg.store(p.y, r * p.C, y);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) cg.store(p.hN, (r * (W - 1) + j) * p.C, xw[j]);
    }
}

// Gradients over runs of run_len tokens, one pass forwards in time: the gradient q of p is known at token t
// from the window of inputs, and the input W - 1 tokens back is then complete,
//   dx_u = sum_{i < W} w[W-1-i] q_{u+i}    (tokens of the same sequence only).
// A run reads W - 1 tokens past its end to complete its last inputs.  Positions before a sequence's
// first token are the rows of its carried state.
template <bool BF16, int W, int E, bool VEC>
__global__ void __launch_bounds__(kConvThreads) conv_state_bwd_kernel(const ConvStateParams p) {
    const ChannelGroup<BF16, E, VEC> cg(blockIdx.y, p.C);
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    constexpr int ROWS = kConvRows, SLOT = kConvThreads * ChannelGroup<BF16, E, VEC>::kVec;
    __shared__ __align__(16) unsigned char ring[VEC ? 2 * ROWS * SLOT : 16];   // rows of x, of dy
    float w[W][E], bias[E], dw[W][E], db[E];
    load_taps<W, E>(p, cg, w, bias);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    const int64_t r0 = blockIdx.x * p.run_len, r1 = min64(r0 + p.run_len, p.total_tokens);
    const bool last_run = r1 == p.total_tokens;
    // the first sequence that ends past r0 or is empty and starts there
    int64_t lo = 0, hi = p.num_seqs;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] > r0 || (p.cu[mid + 1] == r0 && p.cu[mid] == r0)) hi = mid;
        else lo = mid + 1;
    }
    for (int64_t seq = lo; seq < p.num_seqs; ++seq) {
        int64_t s0, s1;
        seq_span(p.cu, (int)seq, p.num_seqs, p.total_tokens, s0, s1);
        if (s0 >= r1 && !(last_run && s0 == r1)) break;
        if (s0 == s1 && s0 < r0) continue;
        const int64_t p0 = s0 > r0 ? s0 : r0, p1 = min64(s1, r1);   // this run's tokens of the sequence
        if (p0 > p1 || (p0 == p1 && s0 != s1)) continue;
        float xw[W > 1 ? W - 1 : 1][E], qw[W > 1 ? W - 1 : 1][E];   // inputs and gradients of the last W - 1 tokens
        load_window<W, E>(p, cg, p0, s0, seq, xw);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) qw[j][i] = 0.f;
        const int64_t end = p1 + W - 1, stop = min64(end, s1);   // past `stop` there are no tokens
        auto copy = [&](int slot, int64_t t) {
            if constexpr (VEC) {
                cg.copy(ring + slot * SLOT, p.x, t * p.C, t < stop);
                cg.copy(ring + (ROWS + slot) * SLOT, p.dy, t * p.C, t < stop);
                cp_async_commit();
            }
        };
#pragma unroll
        for (int k = 0; k < ROWS; ++k) copy(k, p0 + k);
        constexpr int BATCH = VEC ? ROWS : 4;
        for (int64_t t0 = p0; t0 < end; t0 += BATCH) {
            Piece<BF16, E> rx[VEC ? 1 : BATCH], rd[VEC ? 1 : BATCH];
            if constexpr (!VEC) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    cg.load(p.x, (t0 + k) * p.C, t0 + k < stop, rx[k]);
                    cg.load(p.dy, (t0 + k) * p.C, t0 + k < stop, rd[k]);
                }
            }
#pragma unroll VEC ? 2 : BATCH
            for (int k = 0; k < BATCH; ++k) {
                const int64_t t = t0 + k;
                if (t >= end) break;
                float x[E], q[E];   // q: dy, then the gradient of p
                if constexpr (VEC) {
                    cp_async_wait_group<ROWS - 1>();
                    cg.read(ring + k * SLOT, x);
                    cg.read(ring + (ROWS + k) * SLOT, q);
                    copy(k, t + ROWS);
                } else {
                    cg.get(rx[k], x);
                    cg.get(rd[k], q);
                }
                if (t < stop) {
                    float a[E], sg[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        float v = bias[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) v = fmaf(w[j][i], xw[j][i], v);
                        a[i] = fmaf(w[W - 1][i], x[i], v);
                        sg[i] = p.silu ? sigmoid_fast(a[i]) : 1.f;
                    }
                    if (p.l2norm) {   // y = s inv:  ds = inv (dy - y (y . dy))
                        float ss = 0.f, sd = 0.f;
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float s = p.silu ? a[i] * sg[i] : a[i];
                            ss = fmaf(s, s, ss);
                            sd = fmaf(s, q[i], sd);
                        }
                        const int lanes = p.d / E;
                        for (int o = lanes / 2; o > 0; o >>= 1) {
                            ss += __shfl_xor_sync(0xffffffffu, ss, o);
                            sd += __shfl_xor_sync(0xffffffffu, sd, o);
                        }
                        const float inv = rsqrtf(ss + 1e-12f), k2 = inv * inv * sd;
#pragma unroll
                        for (int i = 0; i < E; ++i) q[i] = inv * fmaf(-k2, p.silu ? a[i] * sg[i] : a[i], q[i]);
                    }
                    if (p.silu)
#pragma unroll
                        for (int i = 0; i < E; ++i) q[i] *= sg[i] * fmaf(a[i], 1.f - sg[i], 1.f);
                    if (t < p1)
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            db[i] += q[i];
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(q[i], xw[j][i], dw[j][i]);
                            dw[W - 1][i] = fmaf(q[i], x[i], dw[W - 1][i]);
                        }
                }
                const int64_t pos = t - (W - 1);   // complete now
                if (pos >= p0 || (p0 == s0 && p.dh0)) {
                    float dx[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        float v = w[0][i] * q[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) v = fmaf(w[W - 1 - j][i], qw[j][i], v);
                        dx[i] = v;
                    }
                    const int64_t f = pos - s1 + W - 1;   // row of the final state that holds this input
                    if (f >= 0 && p.dhN) {
                        float e[E];
                        cg.load_f32(p.dhN, (seq * (W - 1) + f) * p.C, true, e);
#pragma unroll
                        for (int i = 0; i < E; ++i) dx[i] += e[i];
                    }
                    if (pos >= p0) cg.store(p.y, pos * p.C, dx);
                    else cg.store(p.dh0, (seq * (W - 1) + (pos - s0 + W - 1)) * p.C, dx);
                }
                slide<W, E>(xw, x);
                slide<W, E>(qw, q);
            }
        }
        if constexpr (VEC) cp_async_wait_all();   // (the next sequence's rows go into the same slots)
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (i >= cg.count) break;
        float *dst = p.part + (int64_t)blockIdx.x * (W + 1) * p.C + cg.c0 + i * cg.step;
#pragma unroll
        for (int j = 0; j < W; ++j) dst[(int64_t)j * p.C] = dw[j][i];
        dst[(int64_t)W * p.C] = db[i];
    }
}

// Column sums of [rows, cols]: 32 columns a block, kSumRows rows at a time, in a fixed order.  put(col, sum)
// takes the result.
constexpr int kSumRows = 16;
template <class Put>
__device__ __forceinline__ void column_sum(const float *in, int64_t rows, int64_t cols, Put put) {
    __shared__ float s_sum[kSumRows][33];
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (col < cols)
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < rows; r += kSumRows) s += in[r * cols + col];
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || col >= cols) return;
#pragma unroll
    for (int k = 1; k < kSumRows; ++k) s += s_sum[k][threadIdx.x];
    put(col, s);
}

__global__ void __launch_bounds__(32 * kSumRows) conv_weight_sum_kernel(const float *part, int64_t runs, int C, int W,
                                                                        float *dw, float *dbias) {
    column_sum(part, runs, (int64_t)(W + 1) * C, [&](int64_t col, float s) {
        const int64_t j = col / C, c = col % C;
        if (j < W) dw[c * W + j] = s;
        else if (dbias) dbias[c] = s;
    });
}

}  // namespace kda
