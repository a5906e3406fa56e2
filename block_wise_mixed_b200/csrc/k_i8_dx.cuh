// k_i8_dx.cuh -- gradients through int8 weights:
//
//   dx[m][k] = sum_n g[m][n] w[n][k]     (g = gradient times channel scale)
//
// for one weight matrix, or for gate and up as one contraction over both
// matrices' channels.  g is bf16 and the codes are exact in bf16, so the
// products run on tcgen05.mma kind::f16 with fp32 sums, 256 k columns x NT
// tokens over the two SMs of a cluster.
//
// The codes lie with k along the rows and the contraction across them; the
// operand wants the contraction along its rows, in bf16.  Converter warps turn
// each 64 x 128 block of codes (8 KB, by TMA) into the swizzled 128 x 64 operand:
// a thread takes 8 rows x 4 columns, pairs two rows' bytes of a column with
// one byte permute, and makes them bf16 with two masks and one subtraction:
//   code = bf16(0x4300 | (b & 0x7F)) - bf16(0x4300 | (b & 0x80))
// (128 + low bits, less 128 or 256: exact).  Lanes are laid out so that both
// the 4-byte reads and the 16-byte writes use all banks.  A weight byte
// crosses HBM once for NT tokens and is never stored wider.
// A bf16 g costs its terms up to 2^-8 of their size (half a step).  Over many
// tokens that brings the error of dx to 0.0023 of its norm, where rounding the
// result alone gives 0.0017; for few tokens and columns there is little to
// average over, and it reached 0.006.  Up to 16 tokens, where the instruction has
// twice the columns anyway, g therefore comes in two bf16 parts (16 bits), as
// twice the tokens: the first CTA of a pair fetches the first parts, the second
// the second, and the epilogue adds their columns (64 tokens so: 62 -> 74 us for
// 8192 x 28672).
//
// Bound by shared memory: for 64 channels x 256 tokens each SM takes 8 KB of
// codes and 16 KB of tokens in, reads the codes, writes and reads 16 KB of
// operand and reads 16 KB of tokens, 80 KB or 640 cycles where the tensor cores
// need 512; 32 tokens take 104 KB for 16 KB of codes, 830 cycles where HBM needs
// 700.  Measured: 2048 tokens, 4096 x 14336 175 us, 1.38 PFLOP/s (tensor pipes
// 73% active, clocks down to 1.6 GHz by power); 16 tokens, 8192 x 28672 56 us,
// 4.2 TB/s.
//
// Work is handed to the pairs as in k_i8_stream; the fp32 partial sums of a
// cut tile are added in the order of the pieces by the last contributor,
// whoever that is, so results are reproducible.
//
// Roles: warp 0 copies the codes and the last warp the tokens, each as far ahead
// as its own stages allow; warp 1 of the first CTA issues, the EPI warps from 2
// on finish (lane = k column), the rest convert.  Every wait is bounded.
#pragma once
#include <cuda_bf16.h>

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
    static constexpr int WARPS = 3 + EPI + GROUPS * I8X_GWARPS;
};

template <int NT>
struct I8DxSmem {
    using Cfg = I8DxCfg<NT>;
    uint8_t a[Cfg::S][Cfg::U * I8X_A];      // 1024-aligned
    uint8_t b[Cfg::S][Cfg::U * Cfg::B_STRIDE];
    uint8_t raw[Cfg::R][Cfg::U * I8X_RAW];
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
    uint32_t* err;
    uint32_t* counters;
    float* slots;
};

// Bytes j of two rows' words as a pair of bf16 values.
__device__ __forceinline__ uint32_t i8_pair_bf16(uint32_t wa, uint32_t wb, int j) {
    const uint32_t t = __byte_perm(wa, wb, (uint32_t)(j | (j << 4) | ((4 + j) << 8) | ((4 + j) << 12)));
    const uint32_t lo = lop_and_or(t, 0x007F007Fu, 0x43004300u), hi = lop_and_or(t, 0x00800080u, 0x43004300u);
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo),
                                     *reinterpret_cast<const __nv_bfloat162*>(&hi));
    return *reinterpret_cast<const uint32_t*>(&d);
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
            constexpr uint32_t idesc = bf16_idesc(256, NT);
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
        for (int seg = 0; seg < n_segs; ++seg) {
            const I8Seg g = work.seg(seg);
            const int buf = seg & 1;
            bool ok = !sm.abort_flag && i8_wait(&sm.d_full[buf], (uint32_t)(seg >> 1) & 1u);
            ok = __all_sync(0xffffffffu, ok && !sm.abort_flag);
            if (!ok) {
                if (lane == 0 && !sm.abort_flag) timed_out();
                break;
            }
            i8_fence_after();
            const int64_t k = (g.tile / TM) * 256 + rank * 128 + quad * 32 + lane, m0 = (g.tile % TM) * tok;
            const int mc = (int)min((int64_t)tok, p.M - m0);
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
                            make_uint4(i8_pair_bf16(in[h][0], in[h][1], j), i8_pair_bf16(in[h][2], in[h][3], j),
                                       i8_pair_bf16(in[h][4], in[h][5], j), i8_pair_bf16(in[h][6], in[h][7], j));
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
// g = dy * scale of its channel in bf16, in one part or two (the operand above).
// ---------------------------------------------------------------------------
// A thread keeps its columns' scales and goes down the rows.
template <bool VEC>
__global__ void __launch_bounds__(256) k_i8_scale_grad(const uint16_t* dy, int64_t lddy, const float* s, uint16_t* g,
                                                       int64_t ldg, int64_t lo_off, int M, int N) {
    constexpr int PER = VEC ? 8 : 2;
    const int n = (blockIdx.x * 256 + threadIdx.x) * PER;   // g's rows are padded to 64
    pdl_wait();
    pdl_launch_dependents();
    if (n >= N) return;
    float sc[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) sc[j] = n + j < N ? s[n + j] : 0.f;
    const bool whole = N - n >= PER;
    for (int64_t m0 = blockIdx.y * 4; m0 < M; m0 += gridDim.y * 4) {
        uint32_t w[4][PER / 2];   // four rows' gradients in flight
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) w[i][j] = 0u;
            if (m0 + i < M) {
                const uint16_t* d = dy + (m0 + i) * lddy + n;
                if (VEC && whole) {
                    const uint4 u = *reinterpret_cast<const uint4*>(d);
                    w[i][0] = u.x;
                    w[i][PER > 2 ? 1 : 0] = u.y;
                    w[i][PER > 4 ? 2 : 0] = u.z;
                    w[i][PER > 6 ? 3 : 0] = u.w;
                } else {
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (n + j < N) w[i][j / 2] |= (uint32_t)d[j] << (16 * (j & 1));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (m0 + i >= M) break;
            uint32_t o[PER / 2], l[PER / 2];
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) {
                const float a = bf16_lo(w[i][j]) * sc[2 * j], b = bf16_hi(w[i][j]) * sc[2 * j + 1];
                o[j] = pack_bf16(a, b);
                l[j] = bf16_rest(a, b, o[j]);
            }
            auto put = [&](uint16_t* at, const uint32_t (&v)[PER / 2]) {
                uint32_t* out = reinterpret_cast<uint32_t*>(at);
                if (VEC) *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[PER > 2 ? 1 : 0], v[PER > 4 ? 2 : 0], v[PER > 6 ? 3 : 0]);
                else *out = v[0];
            };
            uint16_t* at = g + (m0 + i) * ldg + n;
            put(at, o);
            if (lo_off) put(at + lo_off, l);   // the second parts
        }
    }
}

}  // namespace mpq
