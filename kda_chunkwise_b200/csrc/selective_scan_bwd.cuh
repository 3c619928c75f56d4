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
//   3. scan_bwd_grad_kernel   every chunk's gradients: a pass forwards that keeps every kBack-th state,
//                             then kBack tokens at a time recomputed into registers and run backwards;
//                             du, ddt and the output take the places of u, delta and dy
//   4. two sums of partial results over channel blocks (dB, dC) and over chunks (the weights)
// Under three exponentials per (token, channel, state); sums are taken in a fixed order, so results do not
// vary between runs.  8192 tokens x 4096 channels x 16 states in bf16: 249 + 51 + 794 + 15 + 20 us, cold.
// At 2048 tokens the chunk kernel has the exponential unit 62 % and the issue slots 68 % busy, the gradient kernel
// the slots 59 % and the shared-memory data path 44 % (three blocks an SM: 168 registers, 66 KB); the chain moves
// 268 MB.  Taken out one at a time, the sums of dB and dC over a warp's channels save 121 us of the gradient
// kernel, the pass forwards 76, the sums over states 60, the last stage 49.  64-token chunks with eight tokens
// recomputed at once halve the chain (35 us) but leave two blocks an SM: chunk and gradient kernel 259 + 881 us
// against 243 + 772 in the same run.
#pragma once

#include <cfloat>
#include <type_traits>

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
    bool vecn;
};

constexpr int kBackKC = 2;   // channels of a thread: B and C are read, and dB and dC summed over a warp, once for both

template <int L>
struct ScanBwdTile {
    static constexpr int kStep = kScanThreads / L;
    static constexpr int kCH = kBackKC * kStep;             // channels of a block
    static constexpr int kTC = L > 4 ? 64 : (L == 4 ? 32 : 16 * L);   // tokens of a chunk
    static constexpr int kBack = L > 4 ? 8 : 4;             // tokens recomputed into registers at once
    static constexpr int kFR = kCH / 4;                     // fours of channels of a row
    static constexpr int kR = kTC * kFR / kScanThreads;     // fours of a chunk per thread
    static constexpr int kYS = kCH + (L == 16 ? 4 : 32 / L);   // row stride: the lanes' rows fall on different banks
};

// Where a block's channels lie and which of a chunk's rows and fours of channels a thread moves.
template <int L>
struct ScanBwdPlace {
    using Tile = ScanBwdTile<L>;
    int64_t t0, t1, c0;
    int left;   // channels of the group from c0 on
    __device__ __forceinline__ int row(int i) const { return threadIdx.x / Tile::kFR + i * (kScanThreads / Tile::kFR); }
    __device__ __forceinline__ int col() const { return 4 * (threadIdx.x % Tile::kFR); }
    __device__ __forceinline__ int on(int i) const {   // how many channels of four i exist
        const int n = left - col();
        return t0 + row(i) < t1 && n > 0 ? (n > 4 ? 4 : n) : 0;
    }
    __device__ __forceinline__ int64_t off(int i, int D) const { return (t0 + row(i)) * D + c0 + col(); }
};

// Stages delta, u and dy of the block's channels ([kTC][kYS] each), B and C.  Rows past the end and channels
// past the group are zero: there a = 1 and every gradient is zero.
template <bool BF16, int L, bool VEC>
__device__ __forceinline__ void stage_bwd(const ScanBwdParams &p, const ScanBwdPlace<L> &at, int g, float *s_delta, float *s_u,
                                          float *s_dy, QuadBC<BF16> *s_bc) {
    using Tile = ScanBwdTile<L>;
    constexpr int YS = Tile::kYS, R = Tile::kR, AHEAD = R < 4 ? R : 4;
    // rows up to the end of the last kBack tokens that hold any
    const int rows = (static_cast<int>(at.t1 - at.t0) + Tile::kBack - 1) / Tile::kBack * Tile::kBack;
    for (int i = threadIdx.x; i < rows * L; i += kScanThreads) {   // row i / L, states 4 (i % L) ..
        const int64_t tb = at.t0 + i / L;
        const int mm = 4 * (i % L);
        int v4 = p.n - mm;
        v4 = tb < at.t1 && v4 > 0 ? (v4 > 4 ? 4 : v4) : 0;
        Quad<BF16> rB, rC;
        rB.load(p.B, (tb * p.G + g) * p.n + mm, v4, p.vecn);
        rC.load(p.C, (tb * p.G + g) * p.n + mm, v4, p.vecn);
        s_bc[i].b = rB.get(p.vecn);
        s_bc[i].c = rC.get(p.vecn);
    }
    float bias[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) bias[k] = p.dt_bias && at.left > at.col() + k ? p.dt_bias[at.c0 + at.col() + k] : 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 * (kScanThreads / Tile::kFR) < rows; i0 += AHEAD) {
        Piece<BF16, 4> ru[AHEAD], rdt[AHEAD], rdo[AHEAD], rz[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int on = at.on(i0 + k);
            const int64_t off = at.off(i0 + k, p.D);
            load_piece<BF16, 4, VEC>(p.u, off, on, ru[k]);
            load_piece<BF16, 4, VEC>(p.dt, off, on, rdt[k]);
            load_piece<BF16, 4, VEC>(p.dout, off, on, rdo[k]);
            load_piece<BF16, 4, VEC>(p.z, off, p.z ? on : 0, rz[k]);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int on = at.on(i0 + k), x = at.row(i0 + k) * YS + at.col();
            float u[4], d[4], dy[4];
            piece_to_f32<BF16, 4, VEC>(ru[k], u);
            piece_to_f32<BF16, 4, VEC>(rdt[k], d);
            piece_to_f32<BF16, 4, VEC>(rdo[k], dy);
            if (p.z) {
                float z[4];
                piece_to_f32<BF16, 4, VEC>(rz[k], z);
#pragma unroll
                for (int w = 0; w < 4; ++w) dy[w] *= silu(z[w]);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) d[w] = on > w ? softplus(d[w] + bias[w]) : 0.f;
            *reinterpret_cast<float4 *>(&s_delta[x]) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4 *>(&s_u[x]) = make_float4(u[0], u[1], u[2], u[3]);
            *reinterpret_cast<float4 *>(&s_dy[x]) = make_float4(dy[0], dy[1], dy[2], dy[3]);
        }
    }
}

template <bool BF16, int L>
struct ScanBwdSmem {
    using Tile = ScanBwdTile<L>;
    static constexpr int kAct = Tile::kTC * Tile::kYS * 4;                               // delta, u, dy
    static constexpr int kBC = Tile::kTC * L * (int)sizeof(QuadBC<BF16>);
    static constexpr int kChunk = 3 * kAct + kBC;                                        // of the chunk kernel
    static constexpr int kCkpt = Tile::kTC / Tile::kBack * kBackKC * 16 * kScanThreads;  // every kBack-th state
    static constexpr int kRed = 2 * (kScanThreads / 32) * Tile::kBack * 8 * L * 4;             // two buffers of the warps' dB, dC rows
    static constexpr int kGrad = kChunk + kCkpt + kRed;
    // Blocks an SM that the kernels' registers are bounded for: no more than its shared memory holds.
    static constexpr int at_most(int blocks, int bytes) { return blocks * (bytes + kBlockReserve) <= kSmSharedBytes ? blocks : at_most(blocks - 1, bytes); }
    static constexpr int kChunkBlocks = at_most(L > 4 ? 3 : 5, kChunk), kGradBlocks = at_most(L > 4 ? 2 : 3, kGrad);
};

template <bool BF16, int L, bool VEC>
__global__ void __launch_bounds__(kScanThreads, (ScanBwdSmem<BF16, L>::kChunkBlocks)) scan_bwd_chunk_kernel(const ScanBwdParams p) {
    using Tile = ScanBwdTile<L>;
    using SM = ScanBwdSmem<BF16, L>;
    constexpr int CH = Tile::kCH, YS = Tile::kYS, KC = kBackKC;
    extern __shared__ __align__(16) unsigned char scan_smem[];
    QuadBC<BF16> *s_bc = reinterpret_cast<QuadBC<BF16> *>(scan_smem);
    float *s_delta = reinterpret_cast<float *>(scan_smem + SM::kBC), *s_u = s_delta + SM::kAct / 4, *s_dy = s_u + SM::kAct / 4;
    const int tid = threadIdx.x, ncb = p.G * p.cbg, cb = blockIdx.x % ncb;
    if (blockIdx.x == 0) check_seqlens(p.cu, p.num_seqs, p.total_tokens);
    const int64_t rec = blockIdx.x / ncb;
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;
    int seq;
    int64_t j;
    bool last;
    ScanBwdPlace<L> at;
    at.c0 = (int64_t)g * DG + cbase;
    at.left = DG - cbase;
    if (!scan_segment(p.cu, p.num_seqs, p.total_tokens, Tile::kTC, rec, seq, j, at.t0, at.t1, last)) return;
    const int lane = tid % L, chl = tid / L, m0 = 4 * lane;
    f32x2 h01[KC], h23[KC], r01[KC], r23[KC], P01[KC], P23[KC];   // P: product of the decays so far
    float A2[KC][4], sum_delta[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        load_decay(p.A_log, at.c0 + chl + k * Tile::kStep, m0, p.n, chl + k * Tile::kStep < at.left, A2[k]);
        h01[k] = h23[k] = r01[k] = r23[k] = 0ull;
        P01[k] = P23[k] = f2_splat(1.f);
        sum_delta[k] = 0.f;
    }
    stage_bwd<BF16, L, VEC>(p, at, g, s_delta, s_u, s_dy, s_bc);
    __syncthreads();
    const int steps = static_cast<int>(at.t1 - at.t0);
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
        const QuadBC<BF16> q = load_bc(&s_bc[i * L + lane]);
        f32x2 b01, b23, c01, c23;
        QuadBC<BF16>::get(q.b, b01, b23);
        QuadBC<BF16>::get(q.c, c01, c23);
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int x = i * YS + chl + k * Tile::kStep;
            const float d = s_delta[x];
            const f32x2 du = f2_splat(d * s_u[x]), dy = f2_splat(s_dy[x]);
            f32x2 a01, a23;
            decays(A2[k], d, a01, a23);
            h01[k] = f2_fma(a01, h01[k], f2_mul(du, b01));
            h23[k] = f2_fma(a23, h23[k], f2_mul(du, b23));
            P01[k] = f2_mul(P01[k], a01);
            P23[k] = f2_mul(P23[k], a23);
            r01[k] = f2_fma(P01[k], f2_mul(dy, c01), r01[k]);
            r23[k] = f2_fma(P23[k], f2_mul(dy, c23), r23[k]);
            sum_delta[k] += d;
        }
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        if (chl + k * Tile::kStep >= at.left) continue;
        const int64_t c = at.c0 + chl + k * Tile::kStep, row = (rec * p.D + c) * p.n;
        float h[4], r[4];
        f2_unpack(h01[k], h[0], h[1]);
        f2_unpack(h23[k], h[2], h[3]);
        f2_unpack(r01[k], r[0], r[1]);
        f2_unpack(r23[k], r[2], r[3]);
        store_quad(p.H + row, m0, p.n, p.vecn, h);
        store_quad(p.R + row, m0, p.n, p.vecn, r);
        if (lane == 0) p.sum_delta[rec * p.D + c] = sum_delta[k];
    }
}

constexpr int kChainThreads = 128;
constexpr int kChainAhead = 16;   // records in flight

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
        auto record = [&](int64_t i) { return base + (back ? count - 1 - i : i); };
        auto pass = [&](int64_t r, const float (&x)[4], float sd) {   // what comes in replaces the record; what goes out
            store_quad(X + (r * p.D + c) * p.n, m0, p.n, p.vecn, cur);
#pragma unroll
            for (int w = 0; w < 4; ++w) cur[w] = fmaf(ex2_approx(A2[w] * sd), cur[w], x[w]);
        };
        int64_t i = 0;
        for (; i + kChainAhead <= count; i += kChainAhead) {
            float x[kChainAhead][4], sd[kChainAhead];
#pragma unroll
            for (int k = 0; k < kChainAhead; ++k) {
                const int64_t r = record(i + k);
                load_quad(X + (r * p.D + c) * p.n, m0, p.n, p.vecn, x[k]);
                sd[k] = p.sum_delta[r * p.D + c];
            }
#pragma unroll
            for (int k = 0; k < kChainAhead; ++k) pass(record(i + k), x[k], sd[k]);
        }
        for (; i < count; ++i) {
            const int64_t r = record(i);
            float x[4];
            load_quad(X + (r * p.D + c) * p.n, m0, p.n, p.vecn, x);
            pass(r, x, p.sum_delta[r * p.D + c]);
        }
        if (back && p.dh0) store_quad(p.dh0 + (seq * p.D + c) * p.n, m0, p.n, p.vecn, cur);
    }
}

template <bool BF16, int L, bool VEC>
__global__ void __launch_bounds__(kScanThreads, (ScanBwdSmem<BF16, L>::kGradBlocks)) scan_bwd_grad_kernel(const ScanBwdParams p) {
    using Tile = ScanBwdTile<L>;
    using SM = ScanBwdSmem<BF16, L>;
    constexpr int TC = Tile::kTC, CH = Tile::kCH, YS = Tile::kYS, KC = kBackKC, kBack = Tile::kBack;
    constexpr int KW = 32 / L;               // channels side by side in a warp
    constexpr int TB = KW > 8 ? KW / 8 : 1;  // tokens whose dB, dC rows are summed over the warp at once
    constexpr int VPL = 8 * TB / KW;         // values of them a lane is left with
    constexpr int RED = kBack * 8 * L;       // dB, dC rows of kBack tokens
    extern __shared__ __align__(16) unsigned char scan_smem[];
    QuadBC<BF16> *s_bc = reinterpret_cast<QuadBC<BF16> *>(scan_smem);
    float *s_delta = reinterpret_cast<float *>(scan_smem + SM::kBC), *s_u = s_delta + SM::kAct / 4, *s_dy = s_u + SM::kAct / 4;
    float4 *s_ckpt = reinterpret_cast<float4 *>(scan_smem + SM::kChunk);
    float *s_red = reinterpret_cast<float *>(scan_smem + SM::kChunk + SM::kCkpt);

    const int tid = threadIdx.x, ncb = p.G * p.cbg, cb = blockIdx.x % ncb;
    const int64_t rec = blockIdx.x / ncb;
    const int DG = p.D / p.G, g = cb / p.cbg, cbase = (cb % p.cbg) * CH;
    const int lane = tid % L, chl = tid / L, m0 = 4 * lane, warp = tid / 32;
    int seq;
    int64_t j;
    bool last;
    ScanBwdPlace<L> at;
    at.c0 = (int64_t)g * DG + cbase;
    at.left = DG - cbase;
    const bool chunk = scan_segment(p.cu, p.num_seqs, p.total_tokens, TC, rec, seq, j, at.t0, at.t1, last) && at.t0 < at.t1;
    f32x2 h01[KC], h23[KC], g01[KC], g23[KC];   // g: a_{t+1} g_{t+1}
    float A2[KC][4];
    f32x2 dA01[KC], dA23[KC];
    float skip[KC], dskip[KC], dbias[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const bool active = chl + k * Tile::kStep < at.left;
        const int64_t c = at.c0 + chl + k * Tile::kStep, row = (rec * p.D + c) * p.n;
        float h[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
        if (!chunk) {   // a record without tokens: nothing to the weights' sums
            if (active) {
                store_quad(p.H + row, m0, p.n, p.vecn, h);
                if (lane == 0) p.pskip[rec * p.D + c] = p.pbias[rec * p.D + c] = 0.f;
            }
            continue;
        }
        load_decay(p.A_log, c, m0, p.n, active, A2[k]);
        if (active) {
            load_quad(p.H + row, m0, p.n, p.vecn, h);
            load_quad(p.R + row, m0, p.n, p.vecn, r);
        }
        h01[k] = f2_pack(h[0], h[1]);
        h23[k] = f2_pack(h[2], h[3]);
        g01[k] = f2_pack(r[0], r[1]);
        g23[k] = f2_pack(r[2], r[3]);
        dA01[k] = dA23[k] = 0ull;
        skip[k] = active && p.skip ? p.skip[c] : 0.f;
        dskip[k] = dbias[k] = 0.f;
    }
    if (!chunk) return;
    stage_bwd<BF16, L, VEC>(p, at, g, s_delta, s_u, s_dy, s_bc);
    __syncthreads();

    // forwards: the state before every kBack tokens (read back by the thread that wrote it)
    const int blocks = static_cast<int>((at.t1 - at.t0 + kBack - 1) / kBack);
#pragma unroll 1
    for (int sb = 0; sb < blocks; ++sb) {
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            float s[4];
            f2_unpack(h01[k], s[0], s[1]);
            f2_unpack(h23[k], s[2], s[3]);
            s_ckpt[(sb * KC + k) * kScanThreads + tid] = make_float4(s[0], s[1], s[2], s[3]);
        }
        if (sb + 1 == blocks) break;
#pragma unroll
        for (int i = 0; i < kBack; ++i) {
            f32x2 b01, b23;
            QuadBC<BF16>::get(s_bc[(sb * kBack + i) * L + lane].b, b01, b23);
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int x = (sb * kBack + i) * YS + chl + k * Tile::kStep;
                const float d = s_delta[x];
                const f32x2 du = f2_splat(d * s_u[x]);
                f32x2 a01, a23;
                decays(A2[k], d, a01, a23);
                h01[k] = f2_fma(a01, h01[k], f2_mul(du, b01));
                h23[k] = f2_fma(a23, h23[k], f2_mul(du, b23));
            }
        }
    }

    // backwards
    const int tokens = static_cast<int>(at.t1 - at.t0);
    float *bc_out = p.pBC + ((int64_t)cb * p.total_tokens + at.t0) * (2 * p.n);
    // kBack tokens; PAD: rows that stand for no token among them
    auto block = [&](int sb, auto pad) {
        constexpr bool PAD = decltype(pad)::value;
        const int tb = sb * kBack;
        f32x2 a01[kBack][KC], a23[kBack][KC], p01[kBack][KC], p23[kBack][KC];   // a_t and a_t h_{t-1}
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const float4 s = s_ckpt[(sb * KC + k) * kScanThreads + tid];
            h01[k] = f2_pack(s.x, s.y);
            h23[k] = f2_pack(s.z, s.w);
        }
#pragma unroll
        for (int i = 0; i < kBack; ++i) {
            f32x2 b01, b23;
            QuadBC<BF16>::get(s_bc[(tb + i) * L + lane].b, b01, b23);
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int x = (tb + i) * YS + chl + k * Tile::kStep;
                const float d = s_delta[x];
                const f32x2 du = f2_splat(d * s_u[x]);
                decays(A2[k], d, a01[i][k], a23[i][k]);
                p01[i][k] = f2_mul(a01[i][k], h01[k]);
                p23[i][k] = f2_mul(a23[i][k], h23[k]);
                h01[k] = f2_fma(du, b01, p01[i][k]);
                h23[k] = f2_fma(du, b23, p23[i][k]);
            }
        }
        float *red = s_red + (sb & 1) * (kScanThreads / 32 * RED) + warp * RED;
        // sums over a channel's states: of g B (the gradient of delta u), of e A (of delta), and the output
        constexpr int NV = L > kBack ? 4 : 3;   // (more lanes than tokens: four a token, so that two lanes hold one)
        float v[KC][NV * kBack];
        float bc[8 * TB];
#pragma unroll
        for (int i = kBack - 1; i >= 0; --i) {
            const QuadBC<BF16> q = load_bc(&s_bc[(tb + i) * L + lane]);
            f32x2 b01, b23, c01, c23, dB01 = 0ull, dB23 = 0ull, dC01 = 0ull, dC23 = 0ull;
            QuadBC<BF16>::get(q.b, b01, b23);
            QuadBC<BF16>::get(q.c, c01, c23);
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int x = (tb + i) * YS + chl + k * Tile::kStep;
                const float d = s_delta[x];
                const f32x2 dd = f2_splat(d), du = f2_splat(d * s_u[x]), dy = f2_splat(s_dy[x]);
                const f32x2 hh01 = f2_fma(du, b01, p01[i][k]), hh23 = f2_fma(du, b23, p23[i][k]);
                g01[k] = f2_fma(c01, dy, g01[k]);
                g23[k] = f2_fma(c23, dy, g23[k]);
                f32x2 e01 = f2_mul(g01[k], p01[i][k]), e23 = f2_mul(g23[k], p23[i][k]);
                // (no token: a = 1 and g comes from after the chunk, so that e would be large, or infinite, and no term)
                if (PAD && tb + i >= tokens) e01 = e23 = 0ull;
                dA01[k] = f2_fma(e01, dd, dA01[k]);
                dA23[k] = f2_fma(e23, dd, dA23[k]);
                float lo, hi;
                f2_unpack(f2_fma(g23[k], b23, f2_mul(g01[k], b01)), lo, hi);
                v[k][NV * i] = lo + hi;
                f2_unpack(f2_fma(e23, f2_pack(A2[k][2], A2[k][3]), f2_mul(e01, f2_pack(A2[k][0], A2[k][1]))), lo, hi);
                v[k][NV * i + 1] = lo + hi;
                f2_unpack(f2_fma(hh23, c23, f2_mul(hh01, c01)), lo, hi);
                v[k][NV * i + 2] = lo + hi;
                if constexpr (NV == 4) v[k][NV * i + 3] = 0.f;
                dB01 = f2_fma(g01[k], du, dB01);
                dB23 = f2_fma(g23[k], du, dB23);
                dC01 = f2_fma(hh01, dy, dC01);
                dC23 = f2_fma(hh23, dy, dC23);
                g01[k] = f2_mul(a01[i][k], g01[k]);
                g23[k] = f2_mul(a23[i][k], g23[k]);
            }
            const int w = 8 * (i % TB);
            f2_unpack(dB01, bc[w], bc[w + 1]);
            f2_unpack(dB23, bc[w + 2], bc[w + 3]);
            f2_unpack(dC01, bc[w + 4], bc[w + 5]);
            f2_unpack(dC23, bc[w + 6], bc[w + 7]);
            if (i % TB == 0) {
                const int k = chl % KW;
                transposed_sums<8 * TB, KW, L>(bc, k);
                const int o = k * VPL;   // token o / 8 of the TB, value o % 8: dB (below 4) or dC of this lane's states
                float *dst = red + (i + o / 8) * (8 * L) + ((o % 8) / 4) * (4 * L) + m0 + o % 4;
#pragma unroll
                for (int x = 0; x < VPL; ++x) dst[x] = bc[x];
            }
        }
        // du, ddt and the output in the place of u, delta and dy: the lanes of a channel are in one warp and
        // have read all three for these tokens
#pragma unroll
        for (int k = 0; k < KC; ++k) transposed_sums<NV * kBack, L, 1>(v[k], lane);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            auto finish = [&](int t, float dbu, float ddA, float y) {
                const int x = t * YS + chl + k * Tile::kStep;
                const float d = s_delta[x], u = s_u[x], dy = s_dy[x];
                const float ddt = fmaf(u, dbu, 0.6931471805599453f * ddA) * one_minus_exp_neg(d);   // sigmoid(x) = 1 - exp(-softplus(x))
                // (no skip is no term: zero times an infinite u or dy would be one)
                s_u[x] = fmaf(d, dbu, p.skip ? skip[k] * dy : 0.f);
                s_delta[x] = ddt;
                s_dy[x] = p.skip ? fmaf(skip[k], u, y) : y;
                dskip[k] = fmaf(dy, u, dskip[k]);
                dbias[k] += ddt;
            };
            if constexpr (L <= kBack) {
#pragma unroll
                for (int i = 0; i < kBack / L; ++i) finish(tb + lane * (kBack / L) + i, v[k][3 * i], v[k][3 * i + 1], v[k][3 * i + 2]);
            } else {   // 16 lanes: two values a lane, a pair of lanes a token
                const float y = __shfl_xor_sync(0xffffffffu, v[k][0], 1);
                if ((lane & 1) == 0) finish(tb + lane / 2, v[k][0], v[k][1], y);
            }
        }
        __syncthreads();
        // the block's dB and dC of these tokens (the other buffer takes the next ones meanwhile)
        const float *all = s_red + (sb & 1) * (kScanThreads / 32 * RED);
#pragma unroll
        for (int i0 = 0; i0 < RED; i0 += kScanThreads) {
            const int i = i0 + tid, t = tb + i / (8 * L), x = i % (8 * L), m = x % (4 * L);
            if (i < RED && t < tokens && m < p.n) {
                float s = all[i];
#pragma unroll
                for (int w = 1; w < kScanThreads / 32; ++w) s += all[w * RED + i];
                bc_out[t * (2 * p.n) + (x / (4 * L)) * p.n + m] = s;
            }
        }
    };
    int sb = blocks - 1;
    if (tokens % kBack != 0) block(sb--, std::true_type());   // (code of its own: tested in the loop it costs 1 % and more)
#pragma unroll 1
    for (; sb >= 0; --sb) block(sb, std::false_type());
#pragma unroll 2
    for (int i = 0; i < Tile::kR && i * (kScanThreads / Tile::kFR) < tokens; ++i) {
        const int on = at.on(i), x = at.row(i) * YS + at.col();
        const int64_t off = at.off(i, p.D);
        Piece<BF16, 4> rz, rdo;
        load_piece<BF16, 4, VEC>(p.z, off, p.z ? on : 0, rz);
        load_piece<BF16, 4, VEC>(p.dout, off, p.z ? on : 0, rdo);
        const float4 du = *reinterpret_cast<const float4 *>(&s_u[x]), ddt = *reinterpret_cast<const float4 *>(&s_delta[x]);
        const float du4[4] = {du.x, du.y, du.z, du.w}, ddt4[4] = {ddt.x, ddt.y, ddt.z, ddt.w};
        store_piece<BF16, 4, VEC>(p.du, off, on, du4);
        store_piece<BF16, 4, VEC>(p.ddt, off, on, ddt4);
        if (p.z) {
            const float4 yv = *reinterpret_cast<const float4 *>(&s_dy[x]);
            const float y[4] = {yv.x, yv.y, yv.z, yv.w};
            float z[4], o[4];
            piece_to_f32<BF16, 4, VEC>(rz, z);
            piece_to_f32<BF16, 4, VEC>(rdo, o);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float sg = sigmoid_fast(z[k]);
                o[k] *= y[k] * sg * fmaf(z[k], 1.f - sg, 1.f);
            }
            store_piece<BF16, 4, VEC>(p.dz, off, on, o);
        }
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) {
#pragma unroll
        for (int w = L / 2; w > 0; w >>= 1) {
            dskip[k] += __shfl_xor_sync(0xffffffffu, dskip[k], w);
            dbias[k] += __shfl_xor_sync(0xffffffffu, dbias[k], w);
        }
        if (chl + k * Tile::kStep < at.left) {
            const int64_t c = at.c0 + chl + k * Tile::kStep;
            float e[4];
            f2_unpack(dA01[k], e[0], e[1]);
            f2_unpack(dA23[k], e[2], e[3]);
            store_quad(p.H + (rec * p.D + c) * p.n, m0, p.n, p.vecn, e);   // read above by this thread
            if (lane == 0) {
                p.pskip[rec * p.D + c] = dskip[k];
                p.pbias[rec * p.D + c] = dbias[k];
            }
        }
    }
}

// dB, dC: the sum over the channel blocks of a group; W = 4 values a thread where a token's 2 n are whole fours.
// Eight warps of a block take every eighth channel block each.
constexpr int kBcSlices = 8;
template <bool BF16, int W>
__global__ void __launch_bounds__(32 * kBcSlices) scan_bwd_bc_kernel(const ScanBwdParams p) {
    __shared__ float s_sum[kBcSlices][32][W + 1];
    const int64_t per_token = (int64_t)p.G * 2 * p.n;
    const int64_t i = ((int64_t)blockIdx.x * 32 + threadIdx.x) * W;
    const bool in = i < p.total_tokens * per_token;
    const int64_t t = in ? i / per_token : 0;
    const int x = in ? static_cast<int>(i % per_token) : 0, g = x / (2 * p.n), w = x % (2 * p.n);
    const float *src = p.pBC + ((int64_t)g * p.cbg * p.total_tokens + t) * (2 * p.n) + w;
    const int64_t stride = p.total_tokens * 2 * p.n;
    float s[W] = {};
    if (in) {
#pragma unroll 8
        for (int b = threadIdx.y; b < p.cbg; b += kBcSlices) {
            if constexpr (W == 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(src + b * stride));
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            } else {
                s[0] += __ldg(src + b * stride);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < W; ++k) s_sum[threadIdx.y][threadIdx.x][k] = s[k];
    __syncthreads();
    if (threadIdx.y >= W || !in) return;
    const int k = threadIdx.y;   // a warp a value
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < kBcSlices; ++b) sum += s_sum[b][threadIdx.x][k];
    store_out(w + k < p.n ? p.dB : p.dC, (t * p.G + g) * p.n + (w + k) % p.n, !BF16, sum);
}

// dA_log, dskip and ddt_bias: column sums over the records.  32 columns a block, kColRows rows at a time.
constexpr int kColRows = 16;
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
#pragma unroll 8
        for (int64_t r = threadIdx.y; r < p.records; r += kColRows) s += src[r * stride];
    }
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || col >= nA + 2 * p.D) return;
#pragma unroll
    for (int k = 1; k < kColRows; ++k) s += s_sum[k][threadIdx.x];
    if (col < nA) {
        const float A = -expf(p.A_log[col]);
        p.dA_log[col] = (A < -FLT_MAX ? -FLT_MAX : A) * s;   // finite (as load_decay): a sum of zero stays zero; a NaN stays one
    } else if (col < nA + p.D) {
        if (p.dskip) p.dskip[col - nA] = s;
    } else if (p.ddt_bias) {
        p.ddt_bias[col - nA - p.D] = s;
    }
}

}  // namespace kda
