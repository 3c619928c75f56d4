// The short causal convolution with its carried window: prompts that continue, single tokens and
// gradients (preprocess.cuh holds the stateless form).
//
//   p_t[c] = bias[c] + sum_{j < W} w[c][j] x_{t-(W-1)+j}[c]      (x before a sequence: its carried state)
//   s = silu(p) or p;   y = s, or s / sqrt(|s|^2 + 1e-12) over the head's channels
// The carried state is the last W - 1 inputs, [num_seqs, W - 1, C] in the inputs' type, oldest first.
//
// About 10 flops a byte at most, so each input is read once, its neighbours in time come from registers, and a
// thread keeps several rows in flight, in a ring in shared memory that it alone reads.  A thread owns E channels, laid
// out as ConvCols says; where they are not moved as vectors, a batch of rows is in registers instead.  8192 x 4096 channels, W = 4, SiLU and unit rows, bf16: forward
// 38 us (134 MB, 3.6 TB/s), backward 75 us + 6 for the weights' sums (201 MB, 2.7 TB/s).  Neither reaches memory's
// rate: the instructions and their latency hold them, 44 % and 53 % of the issue slots busy at four blocks an SM.
#pragma once

#include <type_traits>

#include "activations.cuh"
#include "f32x2.cuh"
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

// How a thread's E channels lie.
enum class ConvCols {
    kVector,     // consecutive, moved as one vector: where the rows allow it
    kApart,      // a block's threads apart, moved one by one: single elements are still read side by side
    kTogether,   // consecutive, moved one by one: with l2norm, since a head's sum is taken over a thread's channels and
                 // its neighbours'
};

// The channels of a thread: c0 + i step.
template <bool BF16, int E, ConvCols COLS>
struct ChannelGroup {
    static constexpr bool VEC = COLS == ConvCols::kVector;
    static constexpr int step = COLS == ConvCols::kApart ? kConvThreads : 1;
    int64_t c0;
    int count;   // how many of the E are channels

    __device__ __forceinline__ ChannelGroup(int64_t block, int C) {
        c0 = block * kConvThreads * E + (step == 1 ? (int64_t)threadIdx.x * E : threadIdx.x);
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
    __device__ __forceinline__ void read(const unsigned char *slot, f32x2 (&v)[E / 2]) const {
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
    // the channels in pairs, for the paired fp32 instructions
    __device__ __forceinline__ void get(const Piece<BF16, E> &r, f32x2 (&v)[E / 2]) const {
        float f[E];
        piece_to_f32<BF16, E, VEC>(r, f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[i] = f2_pack(f[2 * i], f[2 * i + 1]);
    }
    template <bool RO = true>
    __device__ __forceinline__ void load_f32(const void *p, int64_t row, bool on, f32x2 (&v)[E / 2]) const {
        Piece<BF16, E> r;
        load<RO>(p, row, on, r);
        get(r, v);
    }
    __device__ __forceinline__ void store(void *p, int64_t row, const f32x2 (&v)[E / 2]) const {
        float f[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) f2_unpack(v[i], f[2 * i], f[2 * i + 1]);
        store_piece<BF16, E, VEC>(p, row + c0, count, f, step);
    }
};

// The taps of a thread's channels: W floats of a channel lie together, so that four taps are one load.
template <int W, int E, class Group>
__device__ __forceinline__ void load_taps(const ConvStateParams &p, const Group &cg, f32x2 (&w)[W][E / 2], f32x2 (&bias)[E / 2]) {
    const bool whole = (reinterpret_cast<uintptr_t>(p.w) & (W * 4 - 1)) == 0;   // (a power of two where it matters)
    float wf[W][E], bf[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int64_t c = cg.c0 + i * cg.step;
        const bool on = i < cg.count;
        bf[i] = on && p.bias ? __ldg(p.bias + c) : 0.f;
        uint32_t r[W];
#pragma unroll
        for (int j = 0; j < W; ++j) r[j] = 0u;
        if ((W == 2 || W == 4) && whole) {
            if constexpr (W == 2 || W == 4) load_if<W * 4, true>(p.w + c * W, on, r);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) load_if<4, true>(p.w + c * W + j, on, &r[j]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) wf[j][i] = __uint_as_float(r[j]);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        bias[i] = f2_pack(bf[2 * i], bf[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = f2_pack(wf[j][2 * i], wf[j][2 * i + 1]);
    }
}

// sums over the lanes of one head (a power of two up to a warp)
template <int N>
__device__ __forceinline__ void head_sums(float (&v)[N], int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// the sigmoids of a pair
__device__ __forceinline__ f32x2 sigmoids(f32x2 a) {
    float x, y;
    f2_unpack(a, x, y);
    return f2_pack(sigmoid_fast(x), sigmoid_fast(y));
}

template <int N>
__device__ __forceinline__ float pair_dot(const f32x2 (&a)[N], const f32x2 (&b)[N]) {
    f32x2 s = f2_mul(a[0], b[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) s = f2_fma(a[i], b[i], s);
    float x, y;
    f2_unpack(s, x, y);
    return x + y;
}

// One row's p from its window (xw[0] oldest) and input.
template <int W, int N>
__device__ __forceinline__ void conv_taps(const f32x2 (&w)[W][N], const f32x2 (&bias)[N], const f32x2 (&xw)[W > 1 ? W - 1 : 1][N],
                                          const f32x2 (&x)[N], f32x2 (&a)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a[i] = f2_fma(w[j][i], xw[j][i], a[i]);
        a[i] = f2_fma(w[W - 1][i], x[i], a[i]);
    }
}

// One row's output.
template <int W, int N>
__device__ __forceinline__ void conv_row(const ConvStateParams &p, const f32x2 (&w)[W][N], const f32x2 (&bias)[N],
                                         const f32x2 (&xw)[W > 1 ? W - 1 : 1][N], const f32x2 (&x)[N], f32x2 (&y)[N], int lanes) {
    conv_taps<W, N>(w, bias, xw, x, y);
    if (p.silu)
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = f2_mul(y[i], sigmoids(y[i]));
    if (p.l2norm) {
        float ss[1] = {pair_dot(y, y)};
        head_sums(ss, lanes);
        const f32x2 inv = f2_splat(rsqrtf(ss[0] + 1e-12f));
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = f2_mul(y[i], inv);
    }
}

template <int W, int N>
__device__ __forceinline__ void slide(f32x2 (&xw)[W > 1 ? W - 1 : 1][N], const f32x2 (&x)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) xw[j][i] = xw[j + 1][i];
    if (W > 1)
#pragma unroll
        for (int i = 0; i < N; ++i) xw[W > 1 ? W - 2 : 0][i] = x[i];
}

// The window before token t of a sequence starting at s0: inputs, or rows of its carried state.
template <int W, int E, class Group>
__device__ __forceinline__ void load_window(const ConvStateParams &p, const Group &cg, int64_t t, int64_t s0,
                                            int64_t seq, f32x2 (&xw)[W > 1 ? W - 1 : 1][E / 2]) {
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

constexpr int kConvRows = 8;     // rows in flight per thread
constexpr int kConvUnroll = 6;   // rows of one turn of a loop: a multiple of every window, so that sliding is renaming

// Rows on their way: a ring whose slot i % kConvRows holds row i of a run, or (not VEC) the rows of one turn in
// registers.
template <bool BF16, int E, ConvCols COLS>
struct ConvRows {
    using Group = ChannelGroup<BF16, E, COLS>;
    static constexpr bool VEC = Group::VEC;
    static constexpr int kSlot = kConvThreads * Group::kVec;
    static constexpr int kBytes = VEC ? kConvRows * kSlot : 16;
    unsigned char *ring;
    const void *p;
    Piece<BF16, E> rows[VEC ? 1 : kConvUnroll];
    __device__ __forceinline__ void copy(const Group &cg, int i, int64_t row, bool on) {
        if constexpr (VEC) cg.copy(ring + i % kConvRows * kSlot, p, row, on);
    }
    __device__ __forceinline__ void fetch(const Group &cg, int k, int64_t row, bool on) {
        if constexpr (!VEC) cg.load(p, row, on, rows[k]);
    }
    __device__ __forceinline__ void read(const Group &cg, int i, int k, f32x2 (&v)[E / 2]) const {
        if constexpr (VEC) cg.read(ring + i % kConvRows * kSlot, v);
        else cg.get(rows[k], v);
    }
};

// grid: x = runs of run_len tokens, then one block per sequence for the final states; y = blocks of
// channels.  With hN = h0 the two are separate launches (first_block skips the runs).
template <bool BF16, int W, int E, ConvCols COLS>
__global__ void __launch_bounds__(kConvThreads) conv_state_fwd_kernel(const ConvStateParams p) {
    constexpr int N = E / 2;
    using Rows = ConvRows<BF16, E, COLS>;
    __shared__ __align__(16) unsigned char slots[Rows::kBytes];
    const ChannelGroup<BF16, E, COLS> cg(blockIdx.y, p.C);
    Rows xs;
    xs.ring = slots;
    xs.p = p.x;
    const int64_t bx = p.first_block + blockIdx.x;
    if (bx == 0 && blockIdx.y == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    f32x2 xw[W > 1 ? W - 1 : 1][N];
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
    const int rows = static_cast<int>(r1 - r0);
#pragma unroll
    for (int k = 0; k < kConvRows; ++k) {
        xs.copy(cg, k, (r0 + k) * p.C, k < rows);
        cp_async_commit();
    }
    const int lanes = p.d / E;
    f32x2 w[W][N], bias[N];
    load_taps<W, E>(p, cg, w, bias);
    int64_t seq = seq_of(p.cu, p.num_seqs, r0), s0, s1;
    seq_span(p.cu, (int)seq, p.num_seqs, p.total_tokens, s0, s1);
    load_window<W, E>(p, cg, r0, s0, seq, xw);
    int64_t at = r0 * p.C;   // of row i
    auto row = [&](int i, int k) {   // the k-th of a turn
        f32x2 x[N], y[N];
        cp_async_wait_group<kConvRows - 1>();
        xs.read(cg, i, k, x);
        xs.copy(cg, i, at + (int64_t)kConvRows * p.C, i + kConvRows < rows);
        cp_async_commit();
        conv_row<W, N>(p, w, bias, xw, x, y, lanes);
        cg.store(p.y, at, y);
        slide<W, N>(xw, x);
        at += p.C;
    };
    int i = 0;
    while (true) {
        // rows of this sequence
        const int end = seq + 1 < p.num_seqs ? static_cast<int>(min64(s1 > r0 ? s1 - r0 : 0, rows)) : rows;
        for (; i + kConvUnroll <= end; i += kConvUnroll) {
#pragma unroll
            for (int k = 0; k < kConvUnroll; ++k) xs.fetch(cg, k, at + (int64_t)k * p.C, true);
#pragma unroll
            for (int k = 0; k < kConvUnroll; ++k) row(i + k, k);
        }
#pragma unroll 1
        for (; i < end; ++i) {
            xs.fetch(cg, 0, at, true);
            row(i, 0);
        }
        if (i >= rows) break;
        do seq_span(p.cu, (int)++seq, p.num_seqs, p.total_tokens, s0, s1);   // the next sequence that has tokens starts here
        while (r0 + i >= s1 && seq + 1 < p.num_seqs);
        load_window<W, E>(p, cg, r0 + i, r0 + i, seq, xw);
    }
    cp_async_wait_all();
}

// One token of num_seqs sequences; the state (hN) in place.  A block walks over rows of the batch.
template <bool BF16, int W, int E, ConvCols COLS>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvStateParams p) {
    constexpr int N = E / 2;
    const ChannelGroup<BF16, E, COLS> cg(blockIdx.y, p.C);
    const int lanes = p.d / E;
    f32x2 w[W][N], bias[N];
    load_taps<W, E>(p, cg, w, bias);
    for (int64_t r = blockIdx.x; r < p.num_seqs; r += gridDim.x) {
        f32x2 xw[W > 1 ? W - 1 : 1][N], x[N], y[N];
        cg.load_f32(p.x, r * p.C, true, x);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) cg.template load_f32<false>(p.h0, (r * (W - 1) + j) * p.C, true, xw[j]);
        conv_row<W, N>(p, w, bias, xw, x, y, lanes);
        slide<W, N>(xw, x);
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
template <bool BF16, int W, int E, ConvCols COLS>
__global__ void __launch_bounds__(kConvThreads) conv_state_bwd_kernel(const ConvStateParams p) {
    constexpr int N = E / 2;
    using Rows = ConvRows<BF16, E, COLS>;
    __shared__ __align__(16) unsigned char slots[2 * Rows::kBytes];
    const ChannelGroup<BF16, E, COLS> cg(blockIdx.y, p.C);
    Rows xs, ds;   // of x, of dy
    xs.ring = slots;
    ds.ring = slots + Rows::kBytes;
    xs.p = p.x;
    ds.p = p.dy;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    const int lanes = p.d / E;
    f32x2 w[W][N], bias[N], dw[W][N], db[N];
    load_taps<W, E>(p, cg, w, bias);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        db[i] = 0ull;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0ull;
    }
    const f32x2 one = f2_splat(1.f), minus = f2_splat(-1.f);
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
        if (s0 == s1) {   // no tokens: the final state was the initial one
            if (p.dh0)
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    f32x2 e[N];
                    cg.load_f32(p.dhN, (seq * (W - 1) + j) * p.C, p.dhN != nullptr, e);
                    cg.store(p.dh0, (seq * (W - 1) + j) * p.C, e);
                }
            continue;
        }
        // rows i = 0 .. from p0 on: own of them are this run's, with_data have tokens, end complete the inputs
        const int own = static_cast<int>(p1 - p0), end = own + W - 1, with_data = static_cast<int>(min64(end, s1 - p0));
        f32x2 xw[W > 1 ? W - 1 : 1][N], qw[W > 1 ? W - 1 : 1][N];   // inputs and gradients of the last W - 1 tokens
        load_window<W, E>(p, cg, p0, s0, seq, xw);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) qw[j][i] = 0ull;
        int64_t at = p0 * p.C;   // of row i
        auto copy = [&](int i, int64_t off) {
            xs.copy(cg, i, off, i < with_data);
            ds.copy(cg, i, off, i < with_data);
            cp_async_commit();
        };
        auto fetch = [&](int i, int k, int64_t off) {
            xs.fetch(cg, k, off, i < with_data);
            ds.fetch(cg, k, off, i < with_data);
        };
#pragma unroll
        for (int k = 0; k < kConvRows; ++k) copy(k, at + (int64_t)k * p.C);
        // INNER: an own row whose complete input is an own one too, and no row of the final state
        auto row = [&](int i, int turn, auto inner) {   // the turn-th row of a turn
            constexpr bool INNER = decltype(inner)::value;
            f32x2 x[N], q[N];   // q: dy, then the gradient of p
            cp_async_wait_group<kConvRows - 1>();
            xs.read(cg, i, turn, x);
            ds.read(cg, i, turn, q);
            copy(i + kConvRows, at + (int64_t)kConvRows * p.C);
            if (INNER || i < with_data) {
                f32x2 a[N], sg[N];
                conv_taps<W, N>(w, bias, xw, x, a);
#pragma unroll
                for (int k = 0; k < N; ++k) sg[k] = p.silu ? sigmoids(a[k]) : one;
                if (p.l2norm) {   // y = s inv:  ds = inv (dy - y (y . dy)) = inv dy - s inv^3 (s . dy)
                    f32x2 s[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) s[k] = f2_mul(a[k], sg[k]);
                    float sum[2] = {pair_dot(s, s), pair_dot(s, q)};
                    head_sums(sum, lanes);
                    const float inv = rsqrtf(sum[0] + 1e-12f);
                    const f32x2 iv = f2_splat(inv), k2 = f2_splat(-inv * inv * sum[1]);
#pragma unroll
                    for (int k = 0; k < N; ++k) q[k] = f2_mul(iv, f2_fma(k2, s[k], q[k]));
                }
                if (p.silu)   // silu' = sg (1 + a (1 - sg))
#pragma unroll
                    for (int k = 0; k < N; ++k) q[k] = f2_mul(q[k], f2_mul(sg[k], f2_fma(a[k], f2_fma(sg[k], minus, one), one)));
                if (INNER || i < own)
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        db[k] = f2_add(db[k], q[k]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][k] = f2_fma(q[k], xw[j][k], dw[j][k]);
                        dw[W - 1][k] = f2_fma(q[k], x[k], dw[W - 1][k]);
                    }
            }
            const bool carried = i < W - 1;   // the input completed now is a row of the carried state, if any
            if (INNER || !carried || (p0 == s0 && p.dh0)) {
                f32x2 dx[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    dx[k] = f2_mul(w[0][k], q[k]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dx[k] = f2_fma(w[W - 1 - j][k], qw[j][k], dx[k]);
                }
                if (!INNER && p.dhN && p0 + i >= s1) {   // it is also row p0 + i - s1 of the final state
                    f32x2 e[N];
                    cg.load_f32(p.dhN, (seq * (W - 1) + (p0 + i - s1)) * p.C, true, e);
#pragma unroll
                    for (int k = 0; k < N; ++k) dx[k] = f2_add(dx[k], e[k]);
                }
                if (INNER || !carried) cg.store(p.y, at - (int64_t)(W - 1) * p.C, dx);
                else cg.store(p.dh0, (seq * (W - 1) + i) * p.C, dx);
            }
            slide<W, N>(xw, x);
            slide<W, N>(qw, q);
            at += p.C;
        };
        int i = 0;
        auto edge = [&](int last) {
#pragma unroll 1
            for (; i < last; ++i) {
                fetch(i, 0, at);
                row(i, 0, std::false_type());
            }
        };
        edge(W - 1 < end ? W - 1 : end);
        for (; i + kConvUnroll <= own; i += kConvUnroll) {
#pragma unroll
            for (int k = 0; k < kConvUnroll; ++k) fetch(i + k, k, at + (int64_t)k * p.C);
#pragma unroll
            for (int k = 0; k < kConvUnroll; ++k) row(i + k, k, std::true_type());
        }
        edge(end);
        cp_async_wait_all();   // (the next sequence's rows go into the same slots)
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (i >= cg.count) break;
        float *dst = p.part + (int64_t)blockIdx.x * (W + 1) * p.C + cg.c0 + i * cg.step;
        float v[2];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            f2_unpack(dw[j][i / 2], v[0], v[1]);
            dst[(int64_t)j * p.C] = v[i & 1];
        }
        f2_unpack(db[i / 2], v[0], v[1]);
        dst[(int64_t)W * p.C] = v[i & 1];
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
