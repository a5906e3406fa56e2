// k_i8_stream.cuh -- int8 products for few tokens: the weights' bytes bound
// the time, so the kernel is a stream of weight tiles through the tensor
// cores (tcgen05.mma kind::i8).
//
//   D[n][m] = sum_k w[n][k] x[m][k]    (128 channels x NT tokens, s32 in TMEM)
//
// The channels take the 128 lanes (the wide side of the instruction) and the
// tokens its columns, so one token costs no more tensor work than NT.  The
// work is the list of (128-channel tile, 128-byte chunk of k) units, cut into
// equal contiguous runs, one a CTA and one CTA an SM, whatever the shape: no
// wave is left half empty and every SM has the same bytes to fetch.  A CTA
// keeps its whole shared memory in flight as TMA copies.
// A tile that is cut gets its partial sums through global memory: every
// contributor writes its own slot, and the last to arrive adds them.  The
// sums are integers, so the result does not depend on the cuts or the order.
// Gated: gate and up tiles ride in the same stage, against the same tokens.
//
// Roles: warp 0 copies, warp 1 issues the MMAs, warps 2-9 read the
// accumulators (two for each TMEM lane quadrant, taking alternate groups of 16
// tokens).  Every wait is bounded.
#pragma once
#include <type_traits>

#include "i8_gate.cuh"
#include "i8_tc.cuh"
#include "k_i8_rows.cuh"

namespace mpq {

constexpr int I8S_EPI = 8;                            // two for each TMEM lane quadrant
constexpr int I8S_WARPS = 2 + I8S_EPI;
constexpr int I8S_MAX_CTAS = 256;                     // counters in the workspace
constexpr int I8_KC = 128;                            // bytes of k in a stage

template <int NT, int NW>
struct I8StreamCfg {
    static constexpr int W_BYTES = 128 * I8_KC;
    static constexpr int X_BYTES = NT * I8_KC;
    static constexpr int STAGE = NW * W_BYTES + X_BYTES;
    static constexpr int STAGES = (204 * 1024) / STAGE;
    static constexpr int BUFS = NW * NT * 2 <= 512 ? 2 : 1;
    static constexpr uint32_t COLS = NW * NT * BUFS < 32 ? 32 : NW * NT * BUFS;
};

template <int NT, int NW>
struct I8StreamSmem {
    using Cfg = I8StreamCfg<NT, NW>;
    uint8_t st[Cfg::STAGES][Cfg::STAGE];              // 1024-aligned
    uint64_t full[Cfg::STAGES], empty[Cfg::STAGES];
    uint64_t d_full[2], d_empty[2], drain;
    uint32_t tmem;
    volatile int abort_flag;
};

struct I8Product {
    const float* xs;
    const float* ws[2];
    void* y;
    int64_t ldy;
    const uint16_t* dh;
    int64_t lddh;
    uint16_t* d[2];      // d_gate, d_up (or null)
    int64_t ldd;
    uint16_t* g;         // scaled gradients [M][ldg], the up half at + up_off
    int64_t ldg, up_off;
    int M, N, K, y_bf16;
    uint32_t* err;
    uint32_t* counters;  // zero between calls
    int32_t* slots;      // partial sums
};

// A column of outputs: channel n of tokens m, m + 1, ..., with the addresses
// counted along (64-bit products for every element cost more than its
// arithmetic).  MODE 0: linear, 1: gated, 2: the gradients of gate and up.
template <int MODE, int ACT>
struct I8Column {
    uint8_t* y;
    const uint16_t* dh;
    uint16_t *d0, *d1, *g;
    int64_t ystep, dhstep, dstep, gstep, up_off;
    float ws0, ws1;
    bool bf16;

    __device__ __forceinline__ I8Column(const I8Product& p, int64_t m, int64_t n, float ws0_, float ws1_)
        : ws0(ws0_), ws1(ws1_) {
        if (MODE < 2) {
            bf16 = p.y_bf16 != 0;
            ystep = p.ldy * (bf16 ? 2 : 4);
            y = static_cast<uint8_t*>(p.y) + m * ystep + n * (bf16 ? 2 : 4);
        } else {
            dhstep = p.lddh;
            dh = p.dh + m * dhstep + n;
            dstep = p.ldd;
            d0 = p.d[0] ? p.d[0] + m * dstep + n : nullptr;
            d1 = p.d[0] ? p.d[1] + m * dstep + n : nullptr;
            gstep = p.ldg;
            g = p.g + m * gstep + n;
            up_off = p.up_off;
        }
    }
    __device__ __forceinline__ float load_dh() const { return MODE == 2 ? I8Elem<true>::get(*dh) : 0.f; }
    __device__ __forceinline__ void next_dh() { if (MODE == 2) dh += dhstep; }
    __device__ __forceinline__ void next() {
        if (MODE < 2) {
            y += ystep;
        } else {
            if (d0) { d0 += dstep; d1 += dstep; }
            g += gstep;
        }
    }
    __device__ __forceinline__ void put(int acc0, int acc1, float xs, float dhv) const {
        const float a = ((float)acc0 * ws0) * xs;
        float v = a;
        if (MODE > 0) {
            const float b = ((float)acc1 * ws1) * xs;
            const Gate gt = gate_eval<ACT>(a);
            if (MODE == 2) {
                const float dg = dhv * b * gt.grad, du = dhv * gt.act;
                if (d0) {
                    *d0 = (uint16_t)pack_bf16(dg, 0.f);
                    *d1 = (uint16_t)pack_bf16(du, 0.f);
                }
                g[0] = (uint16_t)pack_bf16(dg * ws0, 0.f);
                g[up_off] = (uint16_t)pack_bf16(du * ws1, 0.f);
                return;
            }
            v = gt.act * b;
        }
        if (bf16) *reinterpret_cast<uint16_t*>(y) = (uint16_t)pack_bf16(v, 0.f);
        else *reinterpret_cast<float*>(y) = v;
    }
};

// Unit u belongs to CTA u * G / units (rounded down the same way as the
// runs' ends): run c is [c * units / G, (c + 1) * units / G).
__device__ __forceinline__ int64_t i8_run_start(int64_t c, int64_t units, int64_t G) { return c * units / G; }
__device__ __forceinline__ int64_t i8_run_of(int64_t u, int64_t units, int64_t G) {
    return ((u + 1) * G - 1) / units;
}

template <int NT, int MODE, int ACT>
__global__ void __launch_bounds__(I8S_WARPS * 32, 1)
k_i8_stream(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap0,
            const __grid_constant__ CUtensorMap wmap1, I8Product p) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    using Cfg = I8StreamCfg<NT, NW>;
    constexpr int S = Cfg::STAGES, BUFS = Cfg::BUFS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    I8StreamSmem<NT, NW>& sm = *reinterpret_cast<I8StreamSmem<NT, NW>*>(base);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int KB = (p.K + I8_KC - 1) / I8_KC;
    const int T = (p.N + 127) / 128, TM = (p.M + NT - 1) / NT;
    const int64_t units = (int64_t)TM * T * KB, G = gridDim.x, cta = blockIdx.x;
    const int64_t u0 = i8_run_start(cta, units, G), u1 = i8_run_start(cta + 1, units, G);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.d_full[b], 1);
            mbar_init(&sm.d_empty[b], I8S_EPI);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
        i8_tma_prefetch(&xmap);
        i8_tma_prefetch(&wmap0);
        if (NW == 2) i8_tma_prefetch(&wmap1);
    }
    if (warp == 1) i8_tmem_alloc<false>(&sm.tmem, Cfg::COLS);
    i8_fence_before();
    __syncthreads();
    i8_fence_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();
    pdl_launch_dependents();

    auto timed_out = [&]() {
        set_error(p.err, MPQ_ERR_TIMEOUT);
        sm.abort_flag = 1;
    };
    int armed = 0, segs = 0;

    if (warp == 0) {
        const bool issuer = elect_one();
        const int64_t tile = u0 / KB;
        int kb = (int)(u0 - tile * KB), t = (int)(tile % T), mt = (int)(tile / T), s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int64_t u = u0; u < u1; ++u) {
            ok = i8_wait_warp(&sm.empty[s], ph);
            if (!ok) break;
            ++armed;
            if (issuer) {
                mbar_arrive_expect_tx(&sm.full[s], Cfg::STAGE);
                if (!kI8WaitTest) {
                    const uint32_t bar = smem_u32(&sm.full[s]);
                    const int kc = kb * I8_KC;
                    i8_tma_load<false>(sm.st[s], &wmap0, kc, t * 128, bar);
                    if (NW == 2) i8_tma_load<false>(sm.st[s] + Cfg::W_BYTES, &wmap1, kc, t * 128, bar);
                    i8_tma_load<false>(sm.st[s] + NW * Cfg::W_BYTES, &xmap, kc, mt * NT, bar);
                }
            }
            if (kI8WaitTest) break;   // armed, no copy
            if (++s == S) { s = 0; ph ^= 1u; }
            if (++kb == KB) {   // the next tile
                kb = 0;
                if (++t == T) { t = 0; ++mt; }
            }
        }
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t idesc = i8_idesc(128, NT);
        const bool issuer = elect_one();
        int s = 0;
        uint32_t ph = 0;
        int64_t next = (u0 / KB + 1) * KB;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok; next += KB) {
            const int n = (int)(min(u1, next) - u);
            const int buf = segs % BUFS;
            ok = i8_wait_warp(&sm.d_empty[buf], ((uint32_t)(segs / BUFS) & 1u) ^ 1u);
            if (!ok) break;
            i8_fence_after();
            for (int i = 0; i < n; ++i) {
                ok = i8_wait_warp(&sm.full[s], ph);
                if (!ok) break;
                i8_fence_after();
                const uint32_t st = smem_u32(sm.st[s]);
                if (issuer) {
#pragma unroll
                    for (int j = 0; j < NW; ++j)
                        i8_mma4<false, 0>(tmem + (uint32_t)((buf * NW + j) * NT), st + j * Cfg::W_BYTES,
                                          st + NW * Cfg::W_BYTES, idesc, i > 0);
                    i8_commit<false>(&sm.empty[s]);
                    if (i == n - 1) i8_commit<false>(&sm.d_full[buf]);
                }
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            if (ok) ++segs;
            u += n;
        }
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        int seg = 0;
        for (int64_t u = u0; u < u1; ++seg) {
            const int64_t tile = u / KB, t0 = tile * KB, t1 = t0 + KB;
            const int64_t end = min(u1, t1);
            const int buf = seg % BUFS;
            const int n = (int)(tile % T) * 128 + quad * 32 + lane, m0 = (int)(tile / T) * NT;
            const int mc = min(NT, p.M - m0);
            const bool in = n < p.N;
            const float ws0 = in ? p.ws[0][n] : 0.f, ws1 = NW == 2 && in ? p.ws[1][n] : 0.f;
            bool ok = !sm.abort_flag && i8_wait(&sm.d_full[buf], (uint32_t)(seg / BUFS) & 1u);
            ok = __all_sync(0xffffffffu, ok && !sm.abort_flag);
            if (!ok) {
                if (lane == 0 && !sm.abort_flag) timed_out();
                break;
            }
            i8_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * NW * NT);
            // contributors c0 .. c1; this CTA's slot: 1 for the tile that
            // starts inside its run, 0 for the one that began before it
            const int64_t c0 = i8_run_of(t0, units, G), c1 = i8_run_of(t1 - 1, units, G);
            auto slot_of = [&](int64_t c) {
                return p.slots + ((c * 2 + (c == c0 ? 1 : 0)) * NW * NT) * 128 + quad * 32 + lane;
            };
            // A cut tile: when all others have arrived already, this one only
            // adds; else it leaves its part and counts itself in.
            uint32_t* counter = p.counters + c0 * I8S_EPI + warp - 2;
            const uint32_t others = (uint32_t)(c1 - c0);
            bool mine = 16 * half < mc;   // this warp writes the results
            if (mine && c0 != c1) {
                uint32_t seen = 0;
                if (lane == 0) seen = i8_load_acquire(counter);
                if (__shfl_sync(0xffffffffu, seen, 0) != others) {
                    int32_t* slot = slot_of(cta);
                    for (int c = 16 * half; c < mc; c += 32) {
#pragma unroll
                        for (int j = 0; j < NW; ++j) {
                            uint32_t r[16];
                            i8_tmem_ld16(taddr + (uint32_t)(j * NT + c), r);
                            i8_tmem_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c + i < mc) slot[(j * NT + c + i) * 128] = (int)r[i];
                        }
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
            // Columns c .. c + CW - 1: the sums, then the outputs.  Loads come
            // first (a store may alias them for all the compiler knows, and
            // each would wait for the one before), Q contributors' at a time.
            auto finish = [&](auto cw, auto qn, int c) {
                constexpr int CW = decltype(cw)::value, Q = decltype(qn)::value;
                const int left = mc - c;
                float xs[CW], dh[MODE == 2 ? CW : 1];
#pragma unroll
                for (int i = 0; i < CW; ++i) xs[i] = i < left ? p.xs[m0 + c + i] : 0.f;
                I8Column<MODE, ACT> col(p, m0 + c, in ? n : 0, ws0, ws1);
                if (MODE == 2)
#pragma unroll
                    for (int i = 0; i < CW; ++i)
                        if (i < left) { dh[MODE == 2 ? i : 0] = col.load_dh(); col.next_dh(); }
                int acc[NW][CW];
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    uint32_t r[CW];
                    if (CW == 16) i8_tmem_ld16(taddr + (uint32_t)(j * NT + c), r);
                    else i8_tmem_ld8(taddr + (uint32_t)(j * NT + c), r);
                    i8_tmem_wait();
#pragma unroll
                    for (int i = 0; i < CW; ++i) acc[j][i] = (int)r[i];
                }
                if (c0 != c1)
                    for (int64_t o = c0; o <= c1; o += Q) {
                        int t[Q][NW][CW];
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            const bool add = o + q <= c1 && o + q != cta;
                            const int32_t* slot = slot_of(o + q);
#pragma unroll
                            for (int j = 0; j < NW; ++j)
#pragma unroll
                                for (int i = 0; i < CW; ++i)
                                    t[q][j][i] = add && i < left ? __ldcg(slot + (j * NT + c + i) * 128) : 0;
                        }
#pragma unroll
                        for (int q = 0; q < Q; ++q)
#pragma unroll
                            for (int j = 0; j < NW; ++j)
#pragma unroll
                                for (int i = 0; i < CW; ++i) acc[j][i] += t[q][j][i];
                    }
                if (in) {
#pragma unroll
                    for (int i = 0; i < CW; ++i)
                        if (i < left) {
                            col.put(acc[0][i], acc[NW - 1][i], xs[i], dh[MODE == 2 ? i : 0]);
                            col.next();
                        }
                }
                __syncwarp();
            };
            if (mine) {
                if (mc <= 8) finish(std::integral_constant<int, 8>{}, std::integral_constant<int, 4 / NW>{}, 0);
                else
                    for (int c = 16 * half; c < mc; c += 32)
                        finish(std::integral_constant<int, 16>{}, std::integral_constant<int, 2 / NW>{}, c);
            }
            i8_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.d_empty[buf]);
            u = end;
        }
    }
    // copies and MMAs in flight land before shared memory and TMEM are given
    // up (after an abort they may be; else this is already so)
    __syncthreads();
    if (sm.abort_flag) {
        if (warp == 0)
            for (int i = max(0, armed - S); i < armed; ++i)
                i8_wait_warp(&sm.full[i % S], (uint32_t)(i / S) & 1u);
        if (warp == 1) {   // every MMA issued so far
            if (elect_one()) i8_commit<false>(&sm.drain);
            i8_wait_warp(&sm.drain, 0u);
        }
    }
    i8_fence_before();
    __syncthreads();
    if (warp == 1) {
        i8_fence_after();
        i8_tmem_free<false>(tmem, Cfg::COLS);
    }
}

}  // namespace mpq
