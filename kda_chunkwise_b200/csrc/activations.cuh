// Activations of either storage type (bf16 or fp32), read as vectors where every row starts on a
// vector boundary and element by element elsewhere.  A piece of N consecutive elements is held as
// raw words between the load and its use, so that a prefetched piece costs no conversion (and no
// wait) at the load.
#pragma once

#include "common.cuh"

namespace kda {

template <int BYTES> struct VecOf;
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<16> { using type = uint4; };

template <bool BF16, int N>
struct Piece {
    uint32_t w[N];   // vector loads of bf16 fill the lower half; element loads take a word each
};

// A load through the read-only path, or (RO false) one that may be followed by a store to the same place.
template <bool RO, class V>
__device__ __forceinline__ V load_value(const V *p) {
    if constexpr (RO) return __ldg(p);
    else return *p;
}

// N elements from element `off` on; only the first `valid` are read, the others are zero.  `vec`:
// off is a multiple of N, N elements are 4 bytes or more, and valid is 0 or N.
template <bool BF16, int N, bool RO = true>
__device__ __forceinline__ void load_piece(const void *p, int64_t off, int valid, bool vec, Piece<BF16, N> &r) {
    constexpr int kBytes = N * (BF16 ? 2 : 4);
    if constexpr (kBytes >= 4) {
        if (vec) {
            constexpr int kOne = kBytes > 16 ? 16 : kBytes;
            using V = typename VecOf<kOne>::type;
            const char *src = static_cast<const char *>(p) + off * (BF16 ? 2 : 4);
#pragma unroll
            for (int i = 0; i < kBytes / kOne; ++i) {
                union { V v; uint32_t w[kOne / 4]; } x;
                if (valid > 0) x.v = load_value<RO>(reinterpret_cast<const V *>(src) + i);
                else
#pragma unroll
                    for (int k = 0; k < kOne / 4; ++k) x.w[k] = 0u;
#pragma unroll
                for (int k = 0; k < kOne / 4; ++k) r.w[i * (kOne / 4) + k] = x.w[k];
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (BF16) r.w[i] = i < valid ? (uint32_t)load_value<RO>(static_cast<const uint16_t *>(p) + off + i) : 0u;
        else r.w[i] = i < valid ? load_value<RO>(static_cast<const uint32_t *>(p) + off + i) : 0u;
    }
}

template <bool BF16, int N>
__device__ __forceinline__ void piece_to_f32(const Piece<BF16, N> &r, bool vec, float (&v)[N]) {
    if constexpr (!BF16) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
        if constexpr (N >= 2) {
            if (vec) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] = __uint_as_float((i & 1) ? (r.w[i / 2] & 0xFFFF0000u) : (r.w[i / 2] << 16));
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r.w[i] << 16);
    }
}

// Rounds once to the storage type and stores the first `valid` of N elements.
template <bool BF16, int N>
__device__ __forceinline__ void store_piece(void *p, int64_t off, int valid, bool vec, const float (&v)[N]) {
    constexpr int kBytes = N * (BF16 ? 2 : 4);
    if constexpr (kBytes >= 4) {
        if (vec) {
            if (valid <= 0) return;
            constexpr int kOne = kBytes > 16 ? 16 : kBytes;
            using V = typename VecOf<kOne>::type;
            char *dst = static_cast<char *>(p) + off * (BF16 ? 2 : 4);
#pragma unroll
            for (int i = 0; i < kBytes / kOne; ++i) {
                union { V v; uint32_t w[kOne / 4]; } x;
#pragma unroll
                for (int k = 0; k < kOne / 4; ++k) {
                    const int e = i * (kOne / 4) + k;
                    if constexpr (BF16)
                        x.w[k] = (uint32_t)f32_to_bf16(v[2 * e]) | ((uint32_t)f32_to_bf16(v[2 * e + 1]) << 16);
                    else
                        x.w[k] = __float_as_uint(v[e]);
                }
                reinterpret_cast<V *>(dst)[i] = x.v;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < valid) store_out(p, off + i, !BF16, v[i]);
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void *p, int64_t off) {
    if constexpr (BF16) return bf16_to_f32(__ldg(static_cast<const uint16_t *>(p) + off));
    else return __ldg(static_cast<const float *>(p) + off);
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

// log(1 + exp(x)), to fp32 precision at both ends
__device__ __forceinline__ float softplus(float x) {
    const float e = log1pf(expf(-fabsf(x)));
    return x > 0.f ? x + e : e;
}

// Sum over the L lanes that hold one channel, for L values at once: lane l (of L) is left with the
// total of v[l].  Each step sends half of what is left to the partner lane, so L values take L - 1
// shuffles instead of L log2(L).
template <int L>
__device__ __forceinline__ float transposed_sum(float (&v)[L], int lane) {
#pragma unroll
    for (int w = L / 2; w > 0; w >>= 1) {
        const bool upper = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = upper ? v[i + w] : v[i];
            const float give = upper ? v[i] : v[i + w];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    return v[0];
}

}  // namespace kda
