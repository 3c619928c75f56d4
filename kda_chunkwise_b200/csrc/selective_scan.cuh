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
// channel) (softplus, the gate) is done once, not once per state.
//   - A channel's n states lie on L = 2^ceil(log2(n / 4)) lanes, four to a lane; 128 threads scan
//     128 / L channels of one group over one segment of one sequence.
//   - 256 more threads (or 128: launch_scan_fwd says where) stage the next tile of tokens and write the
//     outputs of the last one meanwhile, so that the scanning warps only scan: with one sequence there is
//     about one of them per scheduler.
//   - What a scanning thread reads from shared memory per token is the next bound: B and C lie next to
//     each other, in bf16 where they came in bf16, so that four states of both are one load.
//   - The sum over the states is taken for L tokens at once (transposed_sums): one value a lane.
// 8192 tokens x 4096 channels x 16 states in bf16 take 297 us; the states' exponentials alone would take 119.
// At 2048 tokens the exponential unit is 56 %, the issue slots 51 % and the shared-memory data path 46 % busy, with
// four scanning and eight staging warps an SM.  Two states a lane, so twice the scanning warps, took
// 300 us against 306 without the call around it: 2 %, not taken.
// Sequences longer than seg_len tokens are cut into segments where the channels of all sequences together would leave
// the GPU half empty (scan_segment_len; one long sequence among short ones is therefore not cut): a first launch finds every segment's end state from zero and its sum of delta (the
// decay over a segment is exp(A sum delta)), the second joins those before its own and scans.
#pragma once

#include "activations.cuh"
#include "f32x2.cuh"

namespace kda {

constexpr int kScanThreads = 128;   // that scan

// ST: threads that stage for them
template <int L, int ST>
struct ScanTile {
    static constexpr int kCH = kScanThreads / L;             // channels of a block
    static constexpr int kTT = L >= 4 ? 64 : 16 * L;         // tokens of a tile
    static constexpr int kFR = kCH / 4;                      // fours of channels of a row
    static constexpr int kR = (kTT * kFR + ST - 1) / ST;           // of them a staging thread holds
    static constexpr int kQ = (kTT * L + ST - 1) / ST;             // fours of states of B (and C) it holds
    static constexpr int kYS = kCH + (L == 16 ? 4 : 32 / L); // row stride of outputs: the lanes' rows fall on different banks
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
    int unit, unit_n;                   // channels (states of B and C) that may be moved at once: 4, 2 or 1
    bool vecn;                          // states are moved in fours
    bool by_length;                     // blocks of long sequences first
};

// The segment that record `rec` stands for: record base(s) + j, base(s) = cu[s] / seg_len + s, is the
// j-th segment of sequence s (an empty sequence has one, empty).  False if there is none.
__device__ __forceinline__ bool scan_segment(const int32_t *cu, int num_seqs, int64_t total, int64_t seg_len, int64_t rec,
                                             int &seq, int64_t &j, int64_t &t0, int64_t &t1, bool &last) {
    int lo = 0, hi = num_seqs;
    if (seg_len > total) lo = static_cast<int>(rec);   // uncut: a record is a sequence
    else while (hi - lo > 1) {
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

// The sequence with `rank` longer ones before it, in uncut batches of up to kRankSeqs sequences: blocks of long
// sequences start first, so that the last ones to end are short.  All threads of the block call it.
constexpr int kRankSeqs = 64;
__device__ __forceinline__ int sequence_of_rank(const int32_t *cu, int num_seqs, int rank) {
    __shared__ int s_seq;
    if (threadIdx.x == 0) s_seq = rank;
    __syncthreads();
    const int i = threadIdx.x;
    if (i < num_seqs) {
        const int64_t len = (int64_t)cu[i + 1] - cu[i];
        int before = 0;
        for (int k = 0; k < num_seqs; ++k) {
            const int64_t other = (int64_t)cu[k + 1] - cu[k];
            before += other > len || (other == len && k < i);
        }
        if (before == rank) s_seq = i;
    }
    __syncthreads();
    return s_seq;
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

// A log2(e) of N states; zero past n (a decay of one on states that stay zero).  Finite, so that the tokens past a
// sequence's end (delta = 0) leave the state as it is whatever A is; a NaN stays one.
template <int N>
__device__ __forceinline__ void load_decay(const float *A_log, int64_t c, int m0, int n, bool active, float (&A2)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = active && m0 + i < n ? -1.4426950408889634f * expf(A_log[c * n + m0 + i]) : 0.f;
        A2[i] = a < -3e38f ? -3e38f : a;
    }
}

__device__ __forceinline__ float silu(float x) { return x * sigmoid_fast(x); }

// Four neighbouring states' values of B or C, raw; `on`: how many exist.  (Each way of loading has its own
// registers: two loads into one would wait for each other.)
template <bool BF16> struct Quad;
template <> struct Quad<true> {
    uint32_t v[2], e[4];
    __device__ __forceinline__ void load(const void *p, int64_t off, int on, bool vec) {
        const uint16_t *src = static_cast<const uint16_t *>(p) + off;
        v[0] = v[1] = e[0] = e[1] = e[2] = e[3] = 0u;
        load_if<8, true>(src, vec && on > 0, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_if<2, true>(src + i, !vec && on > i, &e[i]);
    }
    __device__ __forceinline__ uint2 get(bool vec) const {
        return vec ? make_uint2(v[0], v[1]) : make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
    }
};
template <> struct Quad<false> {
    uint32_t e[4];
    __device__ __forceinline__ void load(const void *p, int64_t off, int on, bool) {
        const float *src = static_cast<const float *>(p) + off;
        e[0] = e[1] = e[2] = e[3] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_if<4, true>(src + i, on > i, &e[i]);
    }
    __device__ __forceinline__ float4 get(bool) const {
        return make_float4(__uint_as_float(e[0]), __uint_as_float(e[1]), __uint_as_float(e[2]), __uint_as_float(e[3]));
    }
};

// Four states' B and C of one token, as they lie in shared memory: bf16 as it came, else fp32.
template <bool BF16> struct QuadBC;
template <> struct QuadBC<true> {
    uint2 b, c;
    __device__ __forceinline__ static f32x2 two(uint32_t w) { return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
    __device__ __forceinline__ static void get(const uint2 &v, f32x2 &lo, f32x2 &hi) { lo = two(v.x); hi = two(v.y); }
};
template <> struct QuadBC<false> {
    float4 b, c;
    __device__ __forceinline__ static void get(const float4 &v, f32x2 &lo, f32x2 &hi) { lo = f2_pack(v.x, v.y); hi = f2_pack(v.z, v.w); }
};

// both at once: one 16-byte load for bf16
__device__ __forceinline__ QuadBC<true> load_bc(const QuadBC<true> *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    QuadBC<true> q;
    q.b = make_uint2(v.x, v.y);
    q.c = make_uint2(v.z, v.w);
    return q;
}
__device__ __forceinline__ QuadBC<false> load_bc(const QuadBC<false> *p) { return *p; }

// the decays exp(A delta) of four states (single products: a pair would need delta twice in registers)
__device__ __forceinline__ void decays(const float (&A2)[4], float delta, f32x2 &a01, f32x2 &a23) {
    a01 = f2_pack(ex2_approx(A2[0] * delta), ex2_approx(A2[1] * delta));
    a23 = f2_pack(ex2_approx(A2[2] * delta), ex2_approx(A2[3] * delta));
}

constexpr int kSmSharedBytes = 228 * 1024, kBlockReserve = 1024;   // an SM's shared memory, and what every block takes of it besides its own

template <bool BF16, int L, int ST>
struct ScanSmem {
    using Tile = ScanTile<L, ST>;
    static constexpr int kD = Tile::kTT * Tile::kCH;       // float2 (delta, delta u)
    static constexpr int kBC = Tile::kTT * L;              // QuadBC
    static constexpr int kY = Tile::kTT * Tile::kYS;       // float
    static constexpr int kBuf = kD * 8 + kBC * (int)sizeof(QuadBC<BF16>) + kY * 4;   // of one tile being scanned
    static constexpr int kFour = BF16 ? 8 : 16;            // bytes of four raw elements
    static constexpr int kRaw = ST * (3 * Tile::kR * kFour + Tile::kQ * (int)sizeof(QuadBC<BF16>));   // of one tile on its way
    static constexpr int kStages = 3;
    static constexpr int kBytes = 2 * kBuf + kStages * kRaw;
    static constexpr bool kPair = 2 * (kBytes + kBlockReserve) <= kSmSharedBytes;   // two blocks fit an SM
    static constexpr bool kAllStage = Tile::kTT * Tile::kFR >= ST;                  // a tile's rows hold fours of channels for all
};

// Asynchronous copy of four elements to shared memory, or zeros past `on` of them; `unit`: how many elements (4, 2
// or 1) the addresses allow to be moved at once.  Single bf16 elements cannot be copied asynchronously: they are
// read with read_four and stored with store_raw instead.
template <bool BF16>
__device__ __forceinline__ void copy_four(void *dst, const void *tensor, const char *at, int on, int unit) {
    constexpr int kElem = BF16 ? 2 : 4;
    const char *src = on > 0 ? at : static_cast<const char *>(tensor);   // (an address that may be named)
    const uint32_t to = smem_u32(dst);
    if (unit == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(to), "l"(src), "n"(4 * kElem), "r"(on > 0 ? 4 * kElem : 0) : "memory");
    } else if (BF16 || unit == 2) {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(to + kElem * i), "l"(src + (on > i ? kElem * i : 0)),
                         "n"(2 * kElem), "r"(on > i + 1 ? 2 * kElem : 0) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(to + 4 * i), "l"(src + (on > i ? 4 * i : 0)), "r"(on > i ? 4 : 0) : "memory");
    }
}

__device__ __forceinline__ void read_four(const char *at, int on, uint32_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = 0u;
        load_if<2, true>(at + 2 * i, on > i, &v[i]);
    }
}

__device__ __forceinline__ void store_raw(void *dst, const uint32_t (&v)[4]) {
    *static_cast<uint2 *>(dst) = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
}

template <bool BF16>
__device__ __forceinline__ void raw_four(const void *p, float (&v)[4]) {
    if constexpr (BF16) {
        const uint2 w = *static_cast<const uint2 *>(p);
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const float4 w = *static_cast<const float4 *>(p);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
}

// Threads 0 .. 127 scan, ST more stage; one barrier a tile.  While tile i is scanned, the outputs of tile i - 1
// are written, tile i + 1 is converted and the tiles after it are on their way into a ring (every
// staging thread reads back what it copied itself).
template <bool BF16, int L, int ST, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads + ST, ST == 128 && ScanSmem<BF16, L, ST>::kPair ? 2 : 1) scan_fwd_kernel(const ScanParams p) {
    using Tile = ScanTile<L, ST>;
    using SM = ScanSmem<BF16, L, ST>;
    static_assert(ST == 256 || SM::kPair || !ScanSmem<BF16, L, 256>::kAllStage, "fewer staging threads for nothing");
    constexpr int CH = Tile::kCH, TT = Tile::kTT, R = Tile::kR, Q = Tile::kQ, YS = Tile::kYS, FR = Tile::kFR, NS = SM::kStages;
    extern __shared__ __align__(16) unsigned char scan_tiles[];
    auto buf_bc = [&](int b) { return reinterpret_cast<QuadBC<BF16> *>(scan_tiles + b * SM::kBuf); };
    auto buf_d = [&](int b) { return reinterpret_cast<float2 *>(buf_bc(b) + SM::kBC); };
    auto buf_y = [&](int b) { return reinterpret_cast<float *>(buf_d(b) + SM::kD); };

    if (blockIdx.x == 0 && !SUMMARY) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    const int ncb = p.G * p.cbg;
    int64_t rec = blockIdx.x / ncb;
    const int cb = blockIdx.x % ncb;
    if (p.by_length) rec = sequence_of_rank(p.cu, p.num_seqs, static_cast<int>(rec));   // (uncut: a record is a sequence)
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;   // first channel of the block within its group
    int seq;
    int64_t j, t0, t1;
    bool last;
    if (!scan_segment(p.cu, p.num_seqs, p.total_tokens, p.seg_len, rec, seq, j, t0, t1, last)) return;
    if (SUMMARY && last) return;
    const int64_t c0 = (int64_t)g * DG + cbase;
    const int tiles = static_cast<int>((t1 - t0 + TT - 1) / TT);

    if (threadIdx.x >= kScanThreads) {
        // ---- staging ----
        const int tid = threadIdx.x - kScanThreads;
        // four i of this thread: row row0 + i kRowStep of a tile (past it where there are more threads than
        // fours), and the channels within the block, the same for every i
        constexpr int kElem = BF16 ? 2 : 4, kRowStep = ST / FR;
        const int row0 = tid / FR, col = 4 * (tid % FR), left = DG - cbase - col, four_on = left > 0 ? (left > 4 ? 4 : left) : 0;
        const int len = static_cast<int>(t1 - t0);
        // how many channels of four i exist in the tile whose first token is t0 + t
        auto on_of = [&](int i, int t) { return row0 + i * kRowStep < TT && t + row0 + i * kRowStep < len ? four_on : 0; };
        float bias[4], skip[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bias[k] = p.dt_bias && four_on > k ? p.dt_bias[c0 + col + k] : 0.f;
            skip[k] = p.skip && four_on > k ? p.skip[c0 + col + k] : 0.f;
        }
        // This thread's part of a ring slot: fours of u, dt and z, and of B and C.  Offsets (in bytes of global memory,
        // in slots of the ring) move along with the tiles.
        unsigned char *const ring = scan_tiles + 2 * SM::kBuf + tid * SM::kFour;
        auto raw = [&](int slot, int which) { return ring + slot * SM::kRaw + which * (ST * SM::kFour); };
        unsigned char *const ring_bc = scan_tiles + 2 * SM::kBuf + 3 * R * ST * SM::kFour + tid * sizeof(QuadBC<BF16>);
        auto raw_bc = [&](int slot, int q) {
            return reinterpret_cast<QuadBC<BF16> *>(ring_bc + slot * SM::kRaw + q * (ST * sizeof(QuadBC<BF16>)));
        };
        auto next = [&](int slot) { return slot + 1 == NS ? 0 : slot + 1; };
        const int64_t row_bytes = (int64_t)p.D * kElem, bc_bytes = (int64_t)p.G * p.n * kElem;
        const int64_t at0 = ((t0 + row0) * p.D + c0 + col) * kElem;
        int64_t fetch_at = at0, out_at = at0, bc_at = (t0 * p.G + g) * p.n * kElem;
        int fetch_slot = 0, convert_slot = 0, out_slot = 0, fetch_t = 0, convert_t = 0, out_t = 0;
        auto fetch = [&]() {
            if (fetch_t < len) {
                if (BF16 && p.unit == 1) {   // all on their way before the first is waited for
                    uint32_t r[3 * R][4];
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const int64_t off = fetch_at + i * kRowStep * row_bytes;
                        const int on = on_of(i, fetch_t);
                        read_four(static_cast<const char *>(p.u) + off, on, r[3 * i]);
                        read_four(static_cast<const char *>(p.dt) + off, on, r[3 * i + 1]);
                        read_four(static_cast<const char *>(p.z) + off, !SUMMARY && p.z ? on : 0, r[3 * i + 2]);
                    }
#pragma unroll
                    for (int i = 0; i < 3 * R; ++i) store_raw(raw(fetch_slot, i), r[i]);
                } else
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int64_t off = fetch_at + i * kRowStep * row_bytes;
                    const int on = on_of(i, fetch_t);
                    copy_four<BF16>(raw(fetch_slot, 3 * i), p.u, static_cast<const char *>(p.u) + off, on, p.unit);
                    copy_four<BF16>(raw(fetch_slot, 3 * i + 1), p.dt, static_cast<const char *>(p.dt) + off, on, p.unit);
                    if (!SUMMARY && p.z) copy_four<BF16>(raw(fetch_slot, 3 * i + 2), p.z, static_cast<const char *>(p.z) + off, on, p.unit);
                }
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const int i = tid + q * ST, mm = 4 * (i % L);   // row i / L, states 4 (i % L) ..
                    int v4 = p.n - mm;
                    v4 = (i < TT * L && fetch_t + i / L < len && v4 > 0) ? (v4 > 4 ? 4 : v4) : 0;
                    const int64_t off = bc_at + (i / L) * bc_bytes + mm * kElem;
                    const char *b = static_cast<const char *>(p.B) + off, *c = static_cast<const char *>(p.C) + off;
                    if (BF16 && p.unit_n == 1) {
                        uint32_t r[2][4];
                        read_four(b, v4, r[0]);
                        read_four(c, SUMMARY ? 0 : v4, r[1]);
                        store_raw(&raw_bc(fetch_slot, q)->b, r[0]);
                        store_raw(&raw_bc(fetch_slot, q)->c, r[1]);
                    } else {
                        copy_four<BF16>(&raw_bc(fetch_slot, q)->b, p.B, b, v4, p.unit_n);
                        if (!SUMMARY) copy_four<BF16>(&raw_bc(fetch_slot, q)->c, p.C, c, v4, p.unit_n);
                    }
                }
            }
            cp_async_commit();
            fetch_at += TT * row_bytes;
            bc_at += TT * bc_bytes;
            fetch_t += TT;
            fetch_slot = next(fetch_slot);
        };
        auto convert = [&](int buf) {
            float2 *d = buf_d(buf);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (row0 + i * kRowStep >= TT) break;
                const int on = on_of(i, convert_t);
                float u[4], dt[4];
                raw_four<BF16>(raw(convert_slot, 3 * i), u);
                raw_four<BF16>(raw(convert_slot, 3 * i + 1), dt);
#pragma unroll
                for (int k = 0; k < 4; ++k) dt[k] = on > k ? softplus(dt[k] + bias[k]) : 0.f;   // zero: the state passes unchanged
                float4 *dst = reinterpret_cast<float4 *>(&d[(row0 + i * kRowStep) * CH + col]);
                dst[0] = make_float4(dt[0], dt[0] * u[0], dt[1], dt[1] * u[1]);
                dst[1] = make_float4(dt[2], dt[2] * u[2], dt[3], dt[3] * u[3]);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = tid + q * ST;
                if (i < TT * L) {
                    if constexpr (SUMMARY) buf_bc(buf)[i].b = raw_bc(convert_slot, q)->b;
                    else buf_bc(buf)[i] = *raw_bc(convert_slot, q);
                }
            }
            convert_t += TT;
            convert_slot = next(convert_slot);
        };
        auto write_out = [&](int buf) {
            if constexpr (!SUMMARY) {
                const float *y = buf_y(buf);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int on = on_of(i, out_t);
                    if (on == 0) continue;
                    const float4 yv = *reinterpret_cast<const float4 *>(&y[(row0 + i * kRowStep) * YS + col]);
                    float o[4] = {yv.x, yv.y, yv.z, yv.w}, r[4];
                    if (p.skip) {
                        raw_four<BF16>(raw(out_slot, 3 * i), r);
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[k] = fmaf(skip[k], r[k], o[k]);
                    }
                    if (p.z) {
                        raw_four<BF16>(raw(out_slot, 3 * i + 2), r);
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[k] *= silu(r[k]);
                    }
                    char *dst = static_cast<char *>(p.out) + out_at + i * kRowStep * row_bytes;
                    if (p.unit == 4) {
                        store_piece<BF16, 4, true>(dst, 0, on, o);
                    } else if (p.unit == 2) {
                        const float lo[2] = {o[0], o[1]}, hi[2] = {o[2], o[3]};
                        store_piece<BF16, 2, true>(dst, 0, on, lo);
                        store_piece<BF16, 2, true>(dst, 2, on - 2, hi);
                    } else {
                        store_piece<BF16, 4, false>(dst, 0, on, o);
                    }
                }
                out_at += TT * row_bytes;
                out_t += TT;
                out_slot = next(out_slot);
            }
        };
        for (int i = 0; i + 1 < NS; ++i) fetch();
        cp_async_wait_group<NS - 2>();
        if (tiles > 0) convert(0);
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {              // tile i is being scanned
            if (i > 0) write_out((i - 1) & 1);         // the last use of that tile's slot
            fetch();                                   // tile i - 1 + NS
            cp_async_wait_group<NS - 2>();             // tile i + 1 has landed
            if (i + 1 < tiles) convert((i + 1) & 1);
            __syncthreads();
        }
        cp_async_wait_all();
        if (tiles > 0) write_out((tiles - 1) & 1);
        return;
    }

    // ---- scanning: four states of one channel ----
    const int tid = threadIdx.x, lane = tid % L, chl = tid / L, m0 = 4 * lane;
    const bool active = cbase + chl < DG;
    const int64_t c = c0 + chl, row_s = ((int64_t)seq * p.D + c) * p.n;
    float A2[4], hv[4] = {0.f, 0.f, 0.f, 0.f}, sum_delta = 0.f;
    load_decay(p.A_log, c, m0, p.n, active, A2);
    if (active) {
        if (j == 0) {
            // with several segments, hN of the last one may be written over h0 while this block runs
            const float *src = (SUMMARY || last) ? p.h0 : p.seg_h0;
            if (p.h0) load_quad(src + row_s, m0, p.n, p.vecn, hv);
            if (SUMMARY && p.h0) store_quad(p.seg_h0 + row_s, m0, p.n, p.vecn, hv);
        } else if (!SUMMARY) {   // join the segments before this one
            for (int64_t i = 0; i < j; ++i) {
                const int64_t r = rec - j + i;
                float e[4];
                load_quad(p.seg_h + (r * p.D + c) * p.n, m0, p.n, p.vecn, e);
                const float sum = p.seg_delta[r * p.D + c];
#pragma unroll
                for (int w = 0; w < 4; ++w) hv[w] = fmaf(i > 0 ? ex2_approx(A2[w] * sum) : 0.f, hv[w], e[w]);
            }
        }
    }
    f32x2 h01 = f2_pack(hv[0], hv[1]), h23 = f2_pack(hv[2], hv[3]);
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const float2 *d = buf_d(i & 1) + chl;
        const QuadBC<BF16> *bc = buf_bc(i & 1) + lane;
        float *sy = buf_y(i & 1) + chl;
        // groups of U tokens, whose outputs are summed over the states together; tokens past the end have
        // delta = 0 and leave the state as it is
        constexpr int U = L < 4 ? 4 : L, N = (TT < 32 ? TT : 32) / U;
        const int groups = static_cast<int>((min64(TT, t1 - t0 - (int64_t)i * TT) + U - 1) / U);
        auto group = [&](int grp, float (&y)[U]) {
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int t = grp * U + x;
                const float2 v = d[t * CH];
                f32x2 a01, a23, b01, b23, c01, c23;
                if constexpr (SUMMARY) {
                    QuadBC<BF16>::get(bc[t * L].b, b01, b23);
                } else {
                    const QuadBC<BF16> q = load_bc(&bc[t * L]);
                    QuadBC<BF16>::get(q.b, b01, b23);
                    QuadBC<BF16>::get(q.c, c01, c23);
                }
                decays(A2, v.x, a01, a23);
                const f32x2 du = f2_splat(v.y);
                h01 = f2_fma(a01, h01, f2_mul(du, b01));
                h23 = f2_fma(a23, h23, f2_mul(du, b23));
                if constexpr (SUMMARY) {
                    sum_delta += v.x;
                } else {
                    float lo, hi;
                    f2_unpack(f2_fma(h23, c23, f2_mul(h01, c01)), lo, hi);
                    y[x] = lo + hi;
                }
            }
            if constexpr (!SUMMARY) transposed_sums<U, L, 1>(y, lane);
        };
        auto put = [&](int grp, const float (&y)[U]) {
            if constexpr (!SUMMARY) {
#pragma unroll
                for (int x = 0; x < U / L; ++x) sy[(grp * U + lane * (U / L) + x) * YS] = y[x];
            }
        };
        int grp = 0;
#pragma unroll 1
        for (; grp + N <= groups; grp += N) {   // unrolled, the outputs stored at the end: no store keeps a later load back
            float y[N][U];
#pragma unroll
            for (int x = 0; x < N; ++x) group(grp + x, y[x]);
#pragma unroll
            for (int x = 0; x < N; ++x) put(grp + x, y[x]);
        }
#pragma unroll 1
        for (; grp < groups; ++grp) {
            float y[U];
            group(grp, y);
            put(grp, y);
        }
        __syncthreads();
    }
    if (!active) return;
    f2_unpack(h01, hv[0], hv[1]);
    f2_unpack(h23, hv[2], hv[3]);
    if constexpr (SUMMARY) {
        store_quad(p.seg_h + (rec * p.D + c) * p.n, m0, p.n, p.vecn, hv);
        if (lane == 0) p.seg_delta[rec * p.D + c] = sum_delta;
    } else {
        if (last && p.hN) store_quad(p.hN + row_s, m0, p.n, p.vecn, hv);
    }
}

// ---- single tokens ------------------------------------------------------------------------------

struct ScanStepParams {
    const void *u, *dt, *z, *B, *C;       // [N, D], [N, D], [N, D] or null, [N, G, n] x 2
    const float *A_log, *skip, *dt_bias;
    float *state;                         // [N, D, n], in place
    void *out;                            // [N, D]
    int N, D, n, G;
};

constexpr int kScanStepThreads = 256;

// One token of N states: the state is read once and written once (0.9 flop a byte), so the kernel
// streams it.  A thread owns four states of one channel (16 bytes) and walks over rows of the batch, the
// decay's weights read once for all its rows.  256 rows of 4096 channels and 16 states (143 MB) take 36 us a call,
// 4.0 TB/s.  Few registers, so that many warps hide the loads, do better than a row in advance or several rows at once
// (29 us against 33 and 37 with the kernel alone repeated, part of the state then in the L2).
template <bool BF16, int L, bool VEC>
__global__ void __launch_bounds__(kScanStepThreads) scan_step_kernel(const ScanStepParams p) {
    const int64_t q = (int64_t)blockIdx.x * kScanStepThreads + threadIdx.x;   // quad of a row of the batch
    const int lane = static_cast<int>(q % L), m0 = 4 * lane;
    const int64_t c = q / L;
    const bool active = c < p.D;   // the L lanes of a channel agree
    const int g = active ? static_cast<int>(c / (p.D / p.G)) : 0;
    int v4 = p.n - m0;
    v4 = active && v4 > 0 ? (v4 > 4 ? 4 : v4) : 0;
    float A2[4];
    load_decay(p.A_log, c, m0, p.n, active, A2);
    const float bias = active && p.dt_bias ? p.dt_bias[c] : 0.f, skip = active && p.skip ? p.skip[c] : 0.f;
    for (int64_t r = blockIdx.y; r < p.N; r += gridDim.y) {
        const int64_t x = r * p.D + c;
        Piece<false, 4> rh;
        Piece<BF16, 4> rB, rC;
        Piece<BF16, 1> ru, rdt, rz;
        load_piece<false, 4, VEC, false>(p.state, x * p.n + m0, v4, rh);
        load_piece<BF16, 1, false>(p.u, x, active, ru);
        load_piece<BF16, 1, false>(p.dt, x, active, rdt);
        load_piece<BF16, 1, false>(p.z, x, active && p.z, rz);
        load_piece<BF16, 4, VEC>(p.B, (r * p.G + g) * p.n + m0, v4, rB);
        load_piece<BF16, 4, VEC>(p.C, (r * p.G + g) * p.n + m0, v4, rC);
        float h[4], b[4], cc[4], u[1], dt[1], z[1], y = 0.f;
        piece_to_f32<false, 4, VEC>(rh, h);
        piece_to_f32<BF16, 4, VEC>(rB, b);
        piece_to_f32<BF16, 4, VEC>(rC, cc);
        piece_to_f32<BF16, 1, false>(ru, u);
        piece_to_f32<BF16, 1, false>(rdt, dt);
        piece_to_f32<BF16, 1, false>(rz, z);
        const float d = softplus(dt[0] + bias), du = d * u[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = fmaf(ex2_approx(A2[i] * d), h[i], du * b[i]);
            y = fmaf(h[i], cc[i], y);
        }
#pragma unroll
        for (int w = L / 2; w > 0; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
        if constexpr (VEC) {
            if (v4 > 0) __stcs(reinterpret_cast<float4 *>(p.state + x * p.n + m0), make_float4(h[0], h[1], h[2], h[3]));
        } else {
            store_piece<false, 4, false>(p.state, x * p.n + m0, v4, h);
        }
        if (lane == 0 && active) {
            if (p.skip) y = fmaf(skip, u[0], y);   // (no skip is no term: zero times an infinite u would be one)
            if (p.z) y *= silu(z[0]);
            store_out(p.out, x, !BF16, y);
        }
    }
}

}  // namespace kda
