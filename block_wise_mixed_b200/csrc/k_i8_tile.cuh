// k_i8_tile.cuh -- int8 products for many tokens: bound by the tensor cores
// (tcgen05.mma kind::i8 over the two SMs of a cluster).
//
//   D[m][n] = sum_k x[m][k] w[n][k]     256 tokens x 256 channels, s32
//
// Each CTA of the pair holds 128 tokens (its TMEM lanes) and fetches half of
// the tile's channels, so a stage moves 32 KB into each SM for 256 x 256 x
// 128 multiply-adds.  Gated: the first CTA fetches 128 gate rows and the
// second the 128 up rows of the same channels, so one instruction makes both
// products, side by side in the same lanes.  The accumulator is double
// buffered (2 x 256 of the 512 TMEM columns): eight warps finish a tile while
// the next one is multiplied.  They pass 32 x 32 pieces through shared memory
// so that a lane holds a channel: its scales stay in registers and stores are
// whole lines.
// Persistent: pair c takes tiles c, c + pairs, ...; the token tiles of a
// channel tile are consecutive, so a wave shares its weights in L2.
//
// Roles of a CTA: warp 0 copies, warp 1 of the first CTA issues the MMAs,
// warps 2-9 finish.  Every wait is bounded.
//
// Measured on a cool GPU and in a sustained loop (clocks down by power): 2048
// tokens, gate and up 14336 x 4096 152 and 177 us, 3.2 and 2.7 P op/s (tensor pipes
// active 80% of the time when cool); 4096 x 14336 79 and 95 us, 3.0 and 2.5 P op/s
// (68%: 128 tiles on 74 pairs take two rounds for 1.73).
#pragma once
#include "k_i8_stream.cuh"

namespace mpq {

constexpr int I8T_WARPS = 10;
constexpr int I8T_EPI = 8;

template <int MODE>
struct I8TileCfg {
    static constexpr int STAGE = 2 * 128 * I8_KC;             // 128 tokens and 128 channels
    static constexpr int PIECES = MODE == 0 ? 1 : 2;          // a (and b) of 32 x 32 outputs
    static constexpr int STAGES = MODE == 0 ? 6 : 5;
};

template <int MODE>
struct I8TileSmem {
    using Cfg = I8TileCfg<MODE>;
    uint8_t st[Cfg::STAGES][Cfg::STAGE];                      // 1024-aligned
    float piece[I8T_EPI][Cfg::PIECES][32 * 32];               // element (r, c) at r * 32 + (c ^ r)
    uint64_t full[Cfg::STAGES], empty[Cfg::STAGES];
    uint64_t d_full[2], d_empty[2], drain;
    uint32_t tmem;
    volatile int abort_flag;
};

template <int MODE, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(I8T_WARPS * 32, 1)
k_i8_tile(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap0,
          const __grid_constant__ CUtensorMap wmap1, I8Product p) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    constexpr int BN = 256 / NW;                              // channels of a tile
    using Cfg = I8TileCfg<MODE>;
    constexpr int S = Cfg::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    I8TileSmem<MODE>& sm = *reinterpret_cast<I8TileSmem<MODE>*>(base);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();

    const int KB = (p.K + I8_KC - 1) / I8_KC;
    const int64_t T = (p.N - 1) / BN + 1, TM = (p.M - 1) / 256 + 1, tiles = T * TM;   // (sizes up to 2^31 - 1)
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.d_full[b], 1);
            mbar_init(&sm.d_empty[b], 2 * I8T_EPI);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
        i8_tma_prefetch(&xmap);
        i8_tma_prefetch(&wmap0);
        if (NW == 2) i8_tma_prefetch(&wmap1);
    }
    if (warp == 1) i8_tmem_alloc<true>(&sm.tmem, 512);
    i8_fence_before();
    __syncthreads();
    cluster_sync();          // the peer's barriers are ready
    i8_fence_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();
    pdl_launch_dependents();

    auto timed_out = [&]() {
        set_error(p.err, MPQ_ERR_TIMEOUT);
        sm.abort_flag = 1;
    };
    int armed = 0;

    if (warp == 0) {
        const bool issuer = elect_one();
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int64_t tile = pair; tile < tiles && ok; tile += pairs) {
            const int m0 = (int)(tile % TM) * 256 + (int)rank * 128;
            const int n0 = (int)(tile / TM) * BN + (NW == 1 ? (int)rank * 128 : 0);
            const CUtensorMap* wmap = NW == 2 && rank == 1 ? &wmap1 : &wmap0;
            for (int kb = 0; kb < KB; ++kb) {
                ok = i8_wait_warp(&sm.empty[s], ph);
                if (!ok) break;
                ++armed;
                if (issuer) {
                    // the first CTA's barrier counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * Cfg::STAGE);
                    if (!kI8WaitTest) {
                        const uint32_t bar = cluster_addr(&sm.full[s], 0);
                        i8_tma_load<true>(sm.st[s], &xmap, kb * I8_KC, m0, bar);
                        i8_tma_load<true>(sm.st[s] + 128 * I8_KC, wmap, kb * I8_KC, n0, bar);
                    }
                }
                if (kI8WaitTest) break;   // armed, no copy
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            if (kI8WaitTest) break;
        }
        // the releases of the last stages arrive before the CTA ends
        for (int i = max(0, armed - S); !kI8WaitTest && ok && i < armed; ++i)
            ok = i8_wait_warp(&sm.empty[i % S], (uint32_t)(i / S) & 1u);
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = i8_idesc(256, 256);
            const bool issuer = elect_one();
            int s = 0, nt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int64_t tile = pair; tile < tiles && ok; tile += pairs) {
                const int buf = nt & 1;
                ok = i8_wait_warp<true>(&sm.d_empty[buf], ((uint32_t)(nt >> 1) & 1u) ^ 1u);
                if (!ok) break;
                i8_fence_after();
                for (int kb = 0; kb < KB; ++kb) {
                    ok = i8_wait_warp(&sm.full[s], ph);
                    if (!ok) break;
                    i8_fence_after();
                    const uint32_t st = smem_u32(sm.st[s]);
                    if (issuer) {
                        i8_mma4<true, 0>(tmem + (uint32_t)(buf * 256), st, st + 128 * I8_KC, idesc, kb > 0);
                        i8_commit<true>(&sm.empty[s]);
                        if (kb == KB - 1) i8_commit<true>(&sm.d_full[buf]);
                    }
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (ok) ++nt;
            }
            // the peer's last arrivals land before this CTA ends
            for (int i = max(0, nt - 2); ok && i < nt; ++i)
                ok = i8_wait_warp<true>(&sm.d_empty[i & 1], (uint32_t)(i >> 1) & 1u);
            if (!ok && issuer) timed_out();
        }
        __syncwarp();
    } else {
        const int e = warp - 2, quad = warp & 3, half = e >> 2;
        float* pa = sm.piece[e][0];
        float* pb = sm.piece[e][Cfg::PIECES - 1];
        const uint32_t empty_bar = cluster_addr(&sm.d_empty[0], 0);
        int nt = 0;
        for (int64_t tile = pair; tile < tiles; tile += pairs, ++nt) {
            const int buf = nt & 1;
            const int64_t m0 = (tile % TM) * 256 + rank * 128 + quad * 32;
            const int64_t n0 = (tile / TM) * BN + half * (BN / 2);
            const int rows = (int)max((int64_t)0, min((int64_t)32, p.M - m0));
            const float xs = lane < rows ? p.xs[m0 + lane] : 0.f;
            bool ok = !sm.abort_flag && i8_wait(&sm.d_full[buf], (uint32_t)(nt >> 1) & 1u);
            ok = __all_sync(0xffffffffu, ok && !sm.abort_flag);
            if (!ok) {
                if (lane == 0 && !sm.abort_flag) timed_out();
                break;
            }
            i8_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * 256 + half * (BN / 2));
#pragma unroll 1
            for (int c = 0; c < BN / 2; c += 32) {
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    i8_tmem_ld32(taddr + (uint32_t)(j * BN + c), r);
                    i8_tmem_wait();
                    float* q = j ? pb : pa;
#pragma unroll
                    for (int i = 0; i < 32; ++i) q[lane * 32 + (i ^ lane)] = __uint_as_float(r[i]);
                }
                if (c + 32 == BN / 2) {   // the accumulator is read: the next tile's MMAs may start
                    i8_fence_before();
                    __syncwarp();
                    if (lane == 0) cluster_arrive(empty_bar + 8u * (uint32_t)buf);
                }
                __syncwarp();
                const int64_t n = n0 + c + lane;
                const bool in = n < p.N;
                const float ws0 = in ? p.ws[0][n] : 0.f, ws1 = NW == 2 && in ? p.ws[1][n] : 0.f;
                I8Column<MODE> col(p, m0, in ? n : 0);
                for (int i0 = 0; i0 < rows; i0 += 8) {
                    const int left = rows - i0;
                    float dh[MODE == 2 ? 8 : 1];
                    if (MODE == 2)
#pragma unroll
                        for (int i = 0; i < 8; ++i) dh[MODE == 2 ? i : 0] = i < left ? col.next_dh() : 0.f;
                    I8Value o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = i0 + i;
                        const int a0 = __float_as_int(pa[r * 32 + (lane ^ r)]);
                        const int a1 = NW == 2 ? __float_as_int(pb[r * 32 + (lane ^ r)]) : 0;
                        o[i] = i8_value<MODE, ACT>(a0, a1, ws0, ws1, __shfl_sync(0xffffffffu, xs, r),
                                                   dh[MODE == 2 ? i : 0]);
                    }
                    if (in) col.put(o, left);
                }
                __syncwarp();
            }
        }
    }
    __syncthreads();
    if (sm.abort_flag) {
        if (warp == 0 && rank == 0)
            for (int i = max(0, armed - S); i < armed; ++i)
                i8_wait_warp(&sm.full[i % S], (uint32_t)(i / S) & 1u);
        if (warp == 1 && rank == 0) {   // every MMA issued so far
            if (elect_one()) i8_commit<true>(&sm.drain);
            i8_wait_warp(&sm.drain, 0u);
        }
        __syncwarp();
        i8_settle();
    }
    i8_fence_before();
    __syncthreads();
    cluster_sync();          // nothing of the pair reaches into a CTA that has ended
    if (warp == 1) {
        i8_fence_after();
        i8_tmem_free<true>(tmem, 512);
    }
}

}  // namespace mpq
