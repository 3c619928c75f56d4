// Activations of either storage type (bf16 or fp32), read as vectors where every row starts on a
// vector boundary and element by element elsewhere.  A piece of N elements is held as raw words between
// the load and its use, so that a prefetched piece costs no conversion (and no wait) at the load.
#pragma once

#include "common.cuh"
#include "mma_frag.cuh"   // pack_bf16, cp_async

namespace kda {

template <int BYTES> struct VecOf;
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<16> { using type = uint4; };

template <bool BF16, int N>
struct Piece {
    uint32_t w[N];   // vector loads of bf16 fill the lower half; element loads take a word each
};

// Loads of 2, 4, 8 or 16 bytes where `on`, else the words stay as they are.  Written as predicated
// instructions: a branch around a load would make the compiler wait for it at the join, and a prefetch
// would be none.  RO: through the read-only path (not for what the kernel also writes).
template <int BYTES, bool RO>
__device__ __forceinline__ void load_if(const void *p, bool on, uint32_t *w) {
    const int o = on;
    if constexpr (BYTES == 2 && RO)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; @q ld.global.nc.u16 %0, [%1];}" : "+r"(w[0]) : "l"(p), "r"(o));
    else if constexpr (BYTES == 2)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; @q ld.global.u16 %0, [%1];}" : "+r"(w[0]) : "l"(p), "r"(o) : "memory");
    else if constexpr (BYTES == 4 && RO)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; @q ld.global.nc.b32 %0, [%1];}" : "+r"(w[0]) : "l"(p), "r"(o));
    else if constexpr (BYTES == 4)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; @q ld.global.b32 %0, [%1];}" : "+r"(w[0]) : "l"(p), "r"(o) : "memory");
    else if constexpr (BYTES == 8 && RO)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %3, 0; @q ld.global.nc.v2.b32 {%0, %1}, [%2];}"
                     : "+r"(w[0]), "+r"(w[1]) : "l"(p), "r"(o));
    else if constexpr (BYTES == 8)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %3, 0; @q ld.global.v2.b32 {%0, %1}, [%2];}"
                     : "+r"(w[0]), "+r"(w[1]) : "l"(p), "r"(o) : "memory");
    else if constexpr (RO)
        asm volatile("{.reg .pred q; setp.ne.s32 q, %5, 0; @q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];}"
                     : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]) : "l"(p), "r"(o));
    else
        asm volatile("{.reg .pred q; setp.ne.s32 q, %5, 0; @q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];}"
                     : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]) : "l"(p), "r"(o) : "memory");
}

// N elements from element `off` on, `step` apart; only the first `valid` are read, the others are zero.
// VEC: as vectors (step is 1, off is a multiple of N, valid is 0 or N).
template <bool BF16, int N, bool VEC, bool RO = true>
__device__ __forceinline__ void load_piece(const void *p, int64_t off, int valid, Piece<BF16, N> &r, int step = 1) {
    constexpr int kElem = BF16 ? 2 : 4, kBytes = N * kElem;
    const char *src = static_cast<const char *>(p) + off * kElem;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = 0u;
    if constexpr (VEC) {
        constexpr int kOne = kBytes > 16 ? 16 : kBytes;
#pragma unroll
        for (int i = 0; i < kBytes / kOne; ++i) load_if<kOne, RO>(src + i * kOne, valid > 0, r.w + i * (kOne / 4));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) load_if<kElem, RO>(src + (int64_t)i * step * kElem, i < valid, r.w + i);
    }
}

template <bool BF16, int N, bool VEC>
__device__ __forceinline__ void piece_to_f32(const Piece<BF16, N> &r, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (!BF16) v[i] = __uint_as_float(r.w[i]);
        else if constexpr (VEC) v[i] = __uint_as_float((i & 1) ? (r.w[i / 2] & 0xFFFF0000u) : (r.w[i / 2] << 16));
        else v[i] = __uint_as_float(r.w[i] << 16);
    }
}

// Rounds once to the storage type and stores the first `valid` of N elements (as load_piece).
template <bool BF16, int N, bool VEC>
__device__ __forceinline__ void store_piece(void *p, int64_t off, int valid, const float (&v)[N], int step = 1) {
    if constexpr (VEC) {
        if (valid <= 0) return;
        constexpr int kBytes = N * (BF16 ? 2 : 4), kOne = kBytes > 16 ? 16 : kBytes;
        using V = typename VecOf<kOne>::type;
        char *dst = static_cast<char *>(p) + off * (BF16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < kBytes / kOne; ++i) {
            union { V v; uint32_t w[kOne / 4]; } x;
#pragma unroll
            for (int k = 0; k < kOne / 4; ++k) {
                const int e = i * (kOne / 4) + k;
                if constexpr (BF16) x.w[k] = pack_bf16(v[2 * e], v[2 * e + 1]);
                else x.w[k] = __float_as_uint(v[e]);
            }
            reinterpret_cast<V *>(dst)[i] = x.v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < valid) store_out(p, off + (int64_t)i * step, !BF16, v[i]);
    }
}

// Flags cu_seqlens that is not 0 = cu[0] <= cu[1] <= ... = total.  Called by one block of a launch;
// the kernels clamp what they read, so malformed values are reported and never followed.
__device__ __forceinline__ void check_seqlens(const int32_t *cu, int num_seqs, int64_t total) {
    bool ok = true;
    for (int s = threadIdx.x; s < num_seqs; s += blockDim.x) {
        int64_t a, b;
        ok = ok && seq_span(cu, s, num_seqs, total, a, b);
    }
    if (!ok) atomicOr(&g_kda_error_word, kErrBadSeqlens);
}

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|), with log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, and
// atanh(s) / s by the polynomial of degree four in s^2 of least relative error on [0, 1/9] (Remez exchange: 4e-9).
// From zero on a few units in the last place; below zero the relative error is that of e, whose exponent is rounded:
// 1.23 |x| 2^-24 and a few units (8 x 2^-24 at -10, 16 at -20).  Zero below -87.3, where e is flushed.
__device__ __forceinline__ float softplus(float x) {
    const float e = ex2_approx(-1.4426950408889634f * fabsf(x));
    const float s = e * rcp_approx(2.f + e), q = s * s;
    float r = fmaf(q, 0.1408916711807251f, 0.13980300724506378f);
    r = fmaf(r, q, 0.20012454688549042f);
    r = fmaf(r, q, 0.3333315849304199f);
    r = fmaf(r, q, 1.f);
    return fmaf(2.f * s, r, fmaxf(x, 0.f));   // (a NaN passes through s)
}

// 1 - exp(-x) for x >= 0, to a few units in the last place: the series below 1/4 (the first term left out is
// below 5e-8 of the sum), the difference above.
__device__ __forceinline__ float one_minus_exp_neg(float x) {
    float r = fmaf(x, -1.f / 720.f, 1.f / 120.f);
    r = fmaf(r, x, -1.f / 24.f);
    r = fmaf(r, x, 1.f / 6.f);
    r = fmaf(r, x, -0.5f);
    r = fmaf(r, x, 1.f);
    return x < 0.25f ? x * r : 1.f - ex2_approx(-1.4426950408889634f * x);
}

// Sum over LANES lanes (STRIDE apart, this one the idx-th) for V values at once: lane idx is left
// with the totals of v[idx V / LANES] .. in v[0] ..  Each step sends half of what is left to the
// partner lane, so V values take under V shuffles instead of V log2(LANES).
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

}  // namespace kda
