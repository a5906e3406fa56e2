// k_i8_dx.cuh -- gradients through int8 weights:
//
//   dx[m][k] = sum_n g[m][n] w[n][k]     (g = gradient times channel scale)
//
// for one weight matrix, or for gate and up as one contraction over both
// matrices' channels.  g is fp16 with a power of two for each token (below) and
// the codes are exact in fp16, so the products run on tcgen05.mma kind::f16 with
// fp32 sums, 256 k columns x NT tokens over the two SMs of a cluster, and the
// epilogue takes the power of two back.
//
// The codes lie with k along the rows and the contraction across them; the
// operand wants the contraction along its rows, in fp16.  Converter warps turn
// each 64 x 128 block of codes (8 KB, by TMA) into the swizzled 128 x 64 operand:
// a thread takes 8 rows x 4 columns, pairs two rows' bytes of a column with
// one byte permute, and makes them fp16 with one mask and one subtraction:
//   code = fp16(0x6400 | (b ^ 0x80)) - 1152
// (1024 + code + 128: exact).  Lanes are laid out so that both
// the 4-byte reads and the 16-byte writes use all banks.  A weight byte
// crosses HBM once for NT tokens and is never stored wider.
// g in bf16 costs its terms up to 2^-8 of their size (half a step) and brought
// the error of dx to 0.0023 of its norm, where rounding the result alone gives
// 0.0017.  fp16 at the same rate costs 2^-11, if its exponents reach: a power of
// two for each token puts the token's largest |g| into [2^14, 2^15), which leaves
// 28 powers of two below it with all 11 bits and what is smaller still within
// 2^-39 of the largest.  So k_i8_grad_rows makes the operand a token at a time
// (the gated product leaves its scaled gradients in fp32 for it).  Up to 16
// tokens, where the instruction has twice the columns anyway, g comes in two
// fp16 parts (22 bits), as twice the tokens: the first CTA of a pair fetches the
// first parts, the second the second, and the epilogue adds their columns.
//
// Bound by shared memory: for 64 channels x 256 tokens each SM takes 8 KB of
// codes and 16 KB of tokens in, reads the codes, writes and reads 16 KB of
// operand and reads 16 KB of tokens, 80 KB or 640 cycles where the tensor cores
// need 512; 32 tokens take 104 KB for 16 KB of codes, 830 cycles where HBM needs
// 700.  Measured with k_i8_grad_rows, on a cool GPU and in a sustained loop: 2048
// tokens, 4096 x 14336 179 and 215 us, 1.34 and 1.12 PFLOP/s (tensor pipes 74%
// active, clocks down to 1.6 GHz by power; 448 tiles on 74 pairs are six rounds
// and four tiles, so a seventh of the time is a round for these four); 16
// tokens, 8192 x 28672 56 and 61 us, 4.2 and 3.8 TB/s.
//
// Work is handed to the pairs as in k_i8_stream; the fp32 partial sums of a
// cut tile are added in the order of the pieces by the last contributor,
// whoever that is, so results are reproducible.
//
// Roles: warp 0 copies the codes and the last warp the tokens, each as far ahead
// as its own stages allow; warp 1 of the first CTA issues, the EPI warps from 2
// on finish (lane = k column), the rest convert.  Every wait is bounded.
#pragma once
#include "k_i8_stream.cuh"

namespace mpq {

constexpr int I8X_GWARPS = 4;               // warps of a converter group
constexpr int I8X_MAX_EPI = 8;
constexpr int I8X_NC = 64;                  // channels in a stage
constexpr int I8X_RAW = I8X_NC * 128;       // codes of a stage
constexpr int I8X_A = 128 * I8X_NC * 2;     // converted

template <int NT>
struct I8DxCfg {
    // 64-channel blocks in a stage: two while the codes' bytes bound the time
    // (a stage's waits, commit and copies cost each role some 400 cycles,
    // more than the 350 that 8 KB of codes take to arrive), one where the
    // products do and shared memory is needed for tokens.
    static constexpr int U = NT == 256 ? 1 : 2;
    static constexpr int B = NT / 2 * I8X_NC * 2;              // this CTA's tokens, one block
    static constexpr int B_STRIDE = (B + 1023) / 1024 * 1024;
    static constexpr int S = NT == 256 ? 5 : 3;                // operand stages
    static constexpr int R = NT == 256 ? 6 : NT == 128 ? 3 : NT == 64 ? 5 : 6;   // code stages
    static constexpr uint32_t COLS = 2 * NT;                   // double-buffered accumulator
    // Finishing warps, 32 columns each in turn, and converter groups, which
    // take stages in turn: 19 warps leave a thread 96 registers.
    static constexpr int EPI = NT == 32 ? 4 : 8;
    static constexpr int GROUPS = NT == 32 ? 3 : 2;
    static constexpr int PIECES = NT == 32 ? 1 : NT / (8 * EPI);   // 32-column pieces of a finishing warp
    static constexpr int WARPS = 3 + EPI + GROUPS * I8X_GWARPS;
};

template <int NT>
struct I8DxSmem {
    using Cfg = I8DxCfg<NT>;
    uint8_t a[Cfg::S][Cfg::U * I8X_A];      // 1024-aligned
    uint8_t b[Cfg::S][Cfg::U * Cfg::B_STRIDE];
    uint8_t raw[Cfg::R][Cfg::U * I8X_RAW];
    float unscale[Cfg::EPI][Cfg::PIECES * 32];   // of each finishing warp's columns
    uint64_t raw_full[Cfg::R], raw_empty[Cfg::R];
    uint64_t full[Cfg::S], empty[Cfg::S];   // full: both operands of the pair, in the first CTA
    uint64_t d_full[2], d_empty[2], drain;
    uint32_t tmem;
    volatile int abort_flag;
};

struct I8DxParams {
    uint16_t* dx;
    int64_t lddx;
    int M, N, K, nw;
    int split;     // (NT = 32) g in two parts: rows M .. 2 M - 1 hold the second
    const float* unscale;   // one a token
    uint32_t* err;
    uint32_t* counters;
    float* slots;
};

// Bytes j of two rows' words as a pair of fp16 values.
__device__ __forceinline__ uint32_t i8_pair_f16(uint32_t wa, uint32_t wb, int j) {
    const uint32_t t = __byte_perm(wa, wb, (uint32_t)(j | (j << 4) | ((4 + j) << 8) | ((4 + j) << 12)));
    const uint32_t b = (t & 0x00FF00FFu) ^ 0x64806480u;   // 1152 + code
    return h2_bits(__hsub2(bits_h2(b), bits_h2(0x64806480u)));
}

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(I8DxCfg<NT>::WARPS * 32, 1)
k_i8_dx(const __grid_constant__ CUtensorMap wmap0, const __grid_constant__ CUtensorMap wmap1,
        const __grid_constant__ CUtensorMap gmap0, const __grid_constant__ CUtensorMap gmap1, I8DxParams p,
        I8Plan plan) {
    using Cfg = I8DxCfg<NT>;
    constexpr int S = Cfg::S, R = Cfg::R, U = Cfg::U, EPI = Cfg::EPI, GROUPS = Cfg::GROUPS;
    static_assert(R >= S && S >= Cfg::GROUPS, "the converters' parity waits");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    I8DxSmem<NT>& sm = *reinterpret_cast<I8DxSmem<NT>*>(base);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();

    const int NB = (p.N - 1) / (U * I8X_NC) + 1, C = NB * p.nw;   // (N up to 2^31 - 1)
    const bool split = NT == 32 && p.split;
    const int tok = split ? NT / 2 : NT;     // tokens of a tile
    const int64_t TM = (p.M - 1) / tok + 1;
    const int pair = blockIdx.x >> 1;
    const I8Work work(plan, pair, C);
    const int n_segs = work.segs;

    if (tid == 0) {
        for (int s = 0; s < R; ++s) {
            mbar_init(&sm.raw_full[s], 1);
            mbar_init(&sm.raw_empty[s], I8X_GWARPS);
        }
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm.full[s], 2 * I8X_GWARPS + 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.d_full[b], 1);
            mbar_init(&sm.d_empty[b], 2 * Cfg::EPI);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
        i8_tma_prefetch(&wmap0);
        i8_tma_prefetch(&gmap0);
    }
    if (warp == 1) i8_tmem_alloc<true>(&sm.tmem, Cfg::COLS);
    i8_fence_before();
    __syncthreads();
    cluster_sync();
    i8_fence_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();
    pdl_launch_dependents();

    auto timed_out = [&]() {
        set_error(p.err, MPQ_ERR_TIMEOUT);
        sm.abort_flag = 1;
    };
    int armed = 0;   // units whose copies were issued (warp 0: codes, the last warp: tokens)

    if (warp == 0) {
        const bool issuer = elect_one();
        int r = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int j = 0; j < n_segs && ok; ++j) {
            const I8Seg g = work.seg(j);
            const int k0 = (int)(g.tile / TM) * 256 + (int)rank * 128;
            for (int c = g.k0; c < g.k1; ++c) {
                const bool second = c >= NB;   // the second matrix's channels
                ok = i8_wait_warp(&sm.raw_empty[r], ph);
                if (!ok) break;
                if (issuer) {
                    mbar_arrive_expect_tx(&sm.raw_full[r], U * I8X_RAW);
                    if (!kI8WaitTest)
                        i8_tma_load<false>(sm.raw[r], second ? &wmap1 : &wmap0, k0, (second ? c - NB : c) * U * I8X_NC,
                                           smem_u32(&sm.raw_full[r]));
                }
                ++armed;
                if (kI8WaitTest) break;   // armed, no copy
                if (++r == R) { r = 0; ph ^= 1u; }
            }
            if (kI8WaitTest) break;
        }
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else if (warp == Cfg::WARPS - 1) {
        const bool issuer = elect_one();
        const uint32_t full0 = cluster_addr(&sm.full[0], 0);
        int s = 0;
        uint32_t ph = 1;
        bool ok = !kI8WaitTest;
        for (int j = 0; j < n_segs && ok; ++j) {
            const I8Seg g = work.seg(j);
            const int m0 = (int)(g.tile % TM) * tok + (int)rank * (split ? p.M : NT / 2);
            for (int c = g.k0; c < g.k1; ++c) {
                const bool second = c >= NB;
                ok = i8_wait_warp(&sm.empty[s], ph);
                if (!ok) break;
                if (issuer) {
                    // the first CTA's barrier counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * U * Cfg::B);
                    const int n0 = (second ? c - NB : c) * U * I8X_NC;
#pragma unroll
                    for (int b = 0; b < U; ++b)
                        i8_tma_load<true>(sm.b[s] + b * Cfg::B_STRIDE, second ? &gmap1 : &gmap0, n0 + b * I8X_NC, m0,
                                          full0 + 8u * (uint32_t)s);
                }
                ++armed;
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        // the releases of the last stages arrive before the CTA ends
        for (int i = max(0, armed - S); ok && i < armed; ++i)
            ok = i8_wait_warp(&sm.empty[i % S], (uint32_t)(i / S) & 1u);
        if (!ok && issuer && !kI8WaitTest) timed_out();
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = f16_idesc(256, NT);
            const bool issuer = elect_one();
            int s = 0, seg = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int j = 0; j < n_segs && ok; ++j) {
                const I8Seg g = work.seg(j);
                const int n = g.k1 - g.k0, buf = seg & 1;
                ok = i8_wait_warp<true>(&sm.d_empty[buf], ((uint32_t)(seg >> 1) & 1u) ^ 1u);
                if (!ok) break;
                i8_fence_after();
                for (int i = 0; i < n; ++i) {
                    ok = i8_wait_warp<true>(&sm.full[s], ph);
                    if (!ok) break;
                    i8_fence_after();
                    const uint32_t a = smem_u32(sm.a[s]), b = smem_u32(sm.b[s]);
                    if (issuer) {
#pragma unroll
                        for (int q = 0; q < U; ++q)
                            i8_mma4<true, 1>(tmem + (uint32_t)(buf * NT), a + q * I8X_A, b + q * Cfg::B_STRIDE, idesc,
                                             i > 0 || q > 0);
                        i8_commit<true>(&sm.empty[s]);
                        if (i == n - 1) i8_commit<true>(&sm.d_full[buf]);
                    }
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (ok) ++seg;
            }
            // the peer's last arrivals land before this CTA ends
            for (int i = max(0, seg - 2); ok && i < seg; ++i)
                ok = i8_wait_warp<true>(&sm.d_empty[i & 1], (uint32_t)(i >> 1) & 1u);
            if (!ok && issuer) timed_out();
        }
        __syncwarp();
    } else if (warp < 2 + EPI) {
        const int quad = warp & 3, half = (warp - 2) >> 2;   // columns 32 half .., every 8 EPI
        const uint32_t empty_bar = cluster_addr(&sm.d_empty[0], 0);
        float* unscale = sm.unscale[warp - 2];
        for (int seg = 0; seg < n_segs; ++seg) {
            const I8Seg g = work.seg(seg);
            const int buf = seg & 1;
            const int64_t k = (g.tile / TM) * 256 + rank * 128 + quad * 32 + lane, m0 = (g.tile % TM) * tok;
            const int mc = (int)min((int64_t)tok, p.M - m0);
#pragma unroll
            for (int i = 0; i < Cfg::PIECES; ++i) {   // while the tile is multiplied
                const int c = 32 * half + 8 * EPI * i + lane;
                unscale[32 * i + lane] = c < mc ? p.unscale[m0 + c] : 0.f;
            }
            __syncwarp();
            bool ok = !sm.abort_flag && i8_wait(&sm.d_full[buf], (uint32_t)(seg >> 1) & 1u);
            ok = __all_sync(0xffffffffu, ok && !sm.abort_flag);
            if (!ok) {
                if (lane == 0 && !sm.abort_flag) timed_out();
                break;
            }
            i8_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * NT);
            const int c0 = g.c0, c1 = g.c1;
            auto slot_of = [&](int c) {
                return p.slots + ((size_t)(work.slot(c, c0) * 2 + rank) * NT) * 128 + quad * 32 + lane;
            };
            // This CTA's sums of columns c .. c + 31 (both parts).
            auto own_sums = [&](int c, float (&v)[32]) {
                uint32_t t[32];
                i8_tmem_ld32(taddr + (uint32_t)c, t);
                i8_tmem_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(t[i]);
                if (split)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += v[16 + i];   // columns of the second parts
            };
            // A cut tile: when all others have arrived already, this one only
            // adds; else it leaves its part and counts itself in.
            uint32_t* counter = p.counters + (c0 * 2 + rank) * EPI + warp - 2;
            const uint32_t others = (uint32_t)(c1 - c0);
            bool mine = 32 * half < mc;
            if (mine && c0 != c1) {
                uint32_t seen = 0;
                if (lane == 0) seen = i8_load_acquire(counter);
                if (__shfl_sync(0xffffffffu, seen, 0) != others) {
                    float* slot = slot_of(pair);
                    for (int c = 32 * half; c < mc; c += 8 * EPI) {
                        float r[32];
                        own_sums(c, r);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < mc) slot[(c + i) * 128] = r[i];
                    }
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) seen = atomic_add_acq_rel_gpu(counter, 1u);
                    mine = __shfl_sync(0xffffffffu, seen, 0) == others;
                }
                if (mine) {
                    __syncwarp();   // what lane 0 acquired holds for all lanes
                    if (lane == 0) *counter = 0u;   // clean for the next call
                    __threadfence();
                }
            }
            if (mine) {
                for (int c = 32 * half; c < mc; c += 8 * EPI) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                    for (int o = c0; o <= c1; ++o) {   // in the order of the pieces
                        float t[32];
                        if (o == pair) {
                            own_sums(c, t);
                        } else {
                            const float* slot = slot_of(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                t[i] = c + i < mc ? __ldcg(slot + (c + i) * 128) : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += t[i];
                    }
                    const float4* us = reinterpret_cast<const float4*>(unscale + (c - 32 * half) / EPI * 4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 s = us[i];
                        v[4 * i] *= s.x;
                        v[4 * i + 1] *= s.y;
                        v[4 * i + 2] *= s.z;
                        v[4 * i + 3] *= s.w;
                    }
                    if (k < p.K) {
                        uint16_t* dx = p.dx + (m0 + c) * p.lddx + k;
                        const int left = mc - c;
                        if (left >= 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i, dx += p.lddx) *dx = (uint16_t)pack_bf16(v[i], 0.f);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i, dx += p.lddx)
                                if (i < left) *dx = (uint16_t)pack_bf16(v[i], 0.f);
                        }
                    }
                    __syncwarp();
                }
            }
            i8_fence_before();
            __syncwarp();
            if (lane == 0) cluster_arrive(empty_bar + 8u * (uint32_t)buf);
        }
    } else {
        // converters: the groups take the stages in turn, so that several stages'
        // waits, loads and fences overlap.  Warp q of it takes rows 0 .. 31,
        // then 32 .. 63; lane (c, g) the eight rows of block c and the four
        // columns of group (g + 8 c + 8 q) % 32
        const int group = (warp - 2 - EPI) / I8X_GWARPS, q = (warp - 2 - EPI) % I8X_GWARPS, c = lane & 3;
        const int kg = ((lane >> 2) + 8 * c + 8 * q) & 31;
        uint32_t at[4];   // chunk of column 4 kg + j, block c (block c + 4: the other half of the row)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t row = (uint32_t)(4 * kg + j);
            at[j] = (row >> 3) * 1024 + (row & 7) * 128 + (((uint32_t)c ^ (row & 7)) << 4);
        }
        const uint32_t full0 = cluster_addr(&sm.full[0], 0);
        uint32_t n_units = (uint32_t)plan.full * (uint32_t)C;   // stages in all: far below 2^32
        for (int j = plan.full; j < n_segs; ++j) {
            const I8Seg g = work.seg(j);
            n_units += (uint32_t)(g.k1 - g.k0);
        }
        // stage and phase of this group's unit in either ring
        uint32_t r = group, s = group, rph = 0, sph = 1;
        for (uint32_t it = group; it < n_units; it += GROUPS) {
            // The operand stage first: a parity wait can tell a phase only from
            // its neighbour.  Units up to it - S are multiplied once empty[s]
            // says so, so (R >= S) the copy of unit it - R has landed and
            // raw_full[r] is at most one phase behind; asked the other way
            // round, that copy (another group's unit) may still be in flight
            // and the wait would pass a phase early.
            if (!i8_wait_warp(&sm.empty[s], sph) || !i8_wait_warp(&sm.raw_full[r], rph)) {
                if (lane == 0) timed_out();
                break;
            }
#pragma unroll
            for (int b = 0; b < U; ++b) {
                const uint8_t* raw = sm.raw[r] + b * I8X_RAW + 8 * c * 128 + 4 * kg;
                uint32_t in[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        in[h][i] = *reinterpret_cast<const uint32_t*>(raw + (32 * h + i) * 128);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(sm.a[s] + b * I8X_A + (at[j] ^ (uint32_t)(64 * h))) =
                            make_uint4(i8_pair_f16(in[h][0], in[h][1], j), i8_pair_f16(in[h][2], in[h][3], j),
                                       i8_pair_f16(in[h][4], in[h][5], j), i8_pair_f16(in[h][6], in[h][7], j));
            }
            fence_proxy_async_smem();   // to the tensor cores
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.raw_empty[r]);
                cluster_arrive(full0 + 8u * s);
            }
            r += GROUPS;
            if (r >= R) { r -= R; rph ^= 1u; }
            s += GROUPS;
            if (s >= S) { s -= S; sph ^= 1u; }
        }
    }
    __syncthreads();
    if (sm.abort_flag) {
        if (warp == 0)
            for (int i = max(0, armed - R); i < armed; ++i)
                i8_wait_warp(&sm.raw_full[i % R], (uint32_t)(i / R) & 1u);
        if (warp == 1 && rank == 0) {   // every MMA issued so far
            if (elect_one()) i8_commit<true>(&sm.drain);
            i8_wait_warp(&sm.drain, 0u);
        }
        __syncwarp();
        i8_settle();
    }
    i8_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        i8_fence_after();
        i8_tmem_free<true>(tmem, Cfg::COLS);
    }
}

// ---------------------------------------------------------------------------
// The gradients as the product's operand: rows of fp16 in one part or two.
// ---------------------------------------------------------------------------
constexpr int I8G_WARPS = 8;    // of a block with a warp a token

struct I8GradParams {
    const void* src;       // SRC 0, 1: dy in bf16, M x N; 2: scaled fp32 gradients, laid out as g
    int64_t ld;
    const float* s;        // channel scales (SRC 0, 1)
    uint16_t* g;           // fp16 [M][ldg], the up half (SRC 2) at + up_off
    int64_t ldg, up_off;
    int64_t lo_off;        // the second parts, at + lo_off (0: none)
    float* unscale;        // [M]: what brings a token's sums back
    int M, N, cluster;     // tokens, channels; blocks of a token
};

// A warp, a block or a cluster of blocks a token: its values times the channels'
// scales (SRC 2: already done), the largest finite magnitude, and the
// fp16 parts of the values times the power of two that takes that magnitude into
// [2^14, 2^15) (2^126 at most, which leaves smaller values exact or with their 11
// bits all the same).  A thread takes 8 neighbouring columns at a time and keeps
// its first four such units between the two passes; what is beyond them is read
// again.
// SRC 0: rows of dy start at 16-byte blocks.
// Bound by its bytes where they are many (512 tokens, gate and up of 14336: 59 MB
// in, 29 out: 22 us from HBM; with the product's fp32 stores 16 us of 189 in its
// place between the products) and by latency where they are few (1 to 3 us).
template <int SRC, bool WARP>
__global__ void __launch_bounds__(WARP ? I8G_WARPS * 32 : 1024) k_i8_grad_rows(I8GradParams p) {
    constexpr int KEEP = 4;
    __shared__ uint32_t red[32], top_of;
    const int64_t m = WARP ? (int64_t)blockIdx.x * I8G_WARPS + (threadIdx.x >> 5) : blockIdx.x / p.cluster;
    const int first = WARP ? threadIdx.x & 31 : (int)(blockIdx.x % p.cluster * blockDim.x + threadIdx.x);
    const int step = WARP ? 32 : (int)blockDim.x * p.cluster;
    const int per = (p.N - 1) / 8 + 1, units = SRC == 2 ? 2 * per : per;
    const bool s_vec = (reinterpret_cast<uintptr_t>(p.s) & 15) == 0;
    pdl_wait();
    pdl_launch_dependents();
    if (WARP && m >= p.M) return;

    auto offset = [&](int u) { return SRC == 2 && u >= per ? p.up_off + (int64_t)(u - per) * 8 : (int64_t)u * 8; };
    auto load = [&](int u, float (&f)[8]) {
        const int col = (SRC == 2 && u >= per ? u - per : u) * 8;
        const bool whole = p.N - col >= 8;
        if (SRC == 2) {
            const float* x = static_cast<const float*>(p.src) + m * p.ld + offset(u);   // (rows are padded to 64)
            const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            if (!whole)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j >= p.N) f[j] = 0.f;
            return;
        }
        const uint16_t* x = static_cast<const uint16_t*>(p.src) + m * p.ld + col;
        const float* s = p.s + col;
        if (SRC == 0 && whole) {
            I8Elem<true>::unpack(*reinterpret_cast<const uint4*>(x), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = whole || j < p.N - col ? I8Elem<true>::get(x[j]) : 0.f;
        }
        if (s_vec && whole) {
            const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
            f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
            f[4] *= b.x; f[5] *= b.y; f[6] *= b.z; f[7] *= b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (whole || j < p.N - col) f[j] *= s[j];
        }
    };
    uint32_t top = 0;
    auto fold = [&](const float (&f)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t a = __float_as_uint(f[j]) & 0x7FFFFFFFu;
            if (a < 0x7F800000u) top = max(top, a);
        }
    };
    float kept[KEEP][8];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (first + i * step < units) load(first + i * step, kept[i]);
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (first + i * step < units) fold(kept[i]);
    for (int64_t u = (int64_t)first + KEEP * step; !WARP && u < units; u += step) {
        float f[8];
        load((int)u, f);
        fold(f);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (!WARP) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < blockDim.x / 32 ? red[threadIdx.x & 31] : 0u);
    }
    if (!WARP && p.cluster > 1) {
        if (threadIdx.x == 0) top_of = top;
        cluster_sync();
        const uint32_t a = smem_u32(&top_of);
        for (int r = 0; r < p.cluster; ++r) top = max(top, cluster_load(cluster_map(a, (uint32_t)r)));
        cluster_sync();   // the peers have read it
    }

    const int e = (int)(top >> 23), k = e == 0 ? 126 : min(126, 141 - e);   // the largest is in [2^(e - 127), 2^(e - 126))
    const float scale = __uint_as_float((uint32_t)(127 + k) << 23);
    if (first == 0) p.unscale[m] = __uint_as_float((uint32_t)(127 - k) << 23);
    auto put = [&](int u, const float (&f)[8]) {
        uint32_t w[4];
        uint16_t* g = p.g + m * p.ldg + offset(u);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = h2_bits(__floats2half2_rn(f[2 * j] * scale, f[2 * j + 1] * scale));
        *reinterpret_cast<uint4*>(g) = make_uint4(w[0], w[1], w[2], w[3]);
        if (!p.lo_off) return;
        // what that left, rounded again; nothing where it is infinite or NaN (inf - inf would make a NaN of it)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = __low2float(bits_h2(w[j])), y = __high2float(bits_h2(w[j]));
            w[j] = h2_bits(__floats2half2_rn(fabsf(x) < INFINITY ? f[2 * j] * scale - x : 0.f,
                                             fabsf(y) < INFINITY ? f[2 * j + 1] * scale - y : 0.f));
        }
        *reinterpret_cast<uint4*>(g + p.lo_off) = make_uint4(w[0], w[1], w[2], w[3]);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (first + i * step < units) put(first + i * step, kept[i]);
    for (int64_t u = (int64_t)first + KEEP * step; !WARP && u < units; u += step) {
        float f[8];
        load((int)u, f);
        put((int)u, f);
    }
}

}  // namespace mpq
