// k_i8_stream.cuh -- int8 products for few tokens: the weights' bytes bound
// the time, so the kernel is a stream of weight tiles through the tensor
// cores (tcgen05.mma kind::i8).
//
//   D[n][m] = sum_k w[n][k] x[m][k]    (128 channels x NT tokens, s32 in TMEM)
//
// The channels take the 128 lanes (the wide side of the instruction) and the
// tokens its columns, so one token costs no more tensor work than NT.  A CTA
// keeps its whole shared memory in flight as TMA copies, one CTA an SM.
//
// Work (I8Plan): every CTA takes whole tiles, a round of them at a time.  When
// the tiles leave at least two CTAs for each, they are cut along k into equal
// pieces: the CTAs of a cluster where that is the whole call, each leaving its
// sums in its own shared memory (the stages are free by then) and all sharing
// out the columns to read one another's parts; else through global memory, a
// slot for every contributor, and the last to arrive adds them (one token, 1024 x
// 8192: 9.9 us with slots, 7.4 as clusters).  Sums are integers, so the result
// depends neither on the cuts nor on the order.  A last round with more tiles
// than that stays whole, since half of the SMs still draw nearly all of HBM's
// bandwidth (gate and up 14336 x 4096, 112 tiles: 64 tokens 36 us cut into equal
// shares, 24 whole), unless its idle time is worth more than the cuts; then its
// chunks are dealt out in equal runs, and a run may cross into the next tile.
// Gated: gate and up tiles ride in the same stage, against the same tokens.
//
// Roles: warp 0 copies, warp 1 issues the MMAs, warps 2-17 read the
// accumulators (four for each TMEM lane quadrant, each taking every fourth group
// of eight tokens: a group costs mostly latency).  Every wait is bounded.
//
// Measured: 16 tokens through 28672 x 8192 40 us, 5.9 TB/s (floor 36: HBM); one
// token through gate and up 14336 x 4096 21.7 us, 5.4 TB/s (floor 18), through
// 4096 x 4096 8.1 us (floor 2.6: launch, first bytes and the adding up remain).
#pragma once
#include "i8_gate.cuh"
#include "i8_tc.cuh"
#include "k_i8_rows.cuh"

namespace mpq {

constexpr int I8S_EPI = 16;                           // four for each TMEM lane quadrant
constexpr int I8S_WARPS = 2 + I8S_EPI;
constexpr int I8_KC = 128;                            // bytes of k in a chunk

template <int NT, int NW>
struct I8StreamCfg {
    // 128-byte chunks of k in a stage: two of one matrix (a stage's waits,
    // copies and commit cost each role some 400 cycles, as much as 18 KB take
    // to arrive), one of two.
    static constexpr int U = NW == 1 ? 2 : 1;
    static constexpr int W_BYTES = 128 * I8_KC;
    static constexpr int X_BYTES = NT * I8_KC;
    static constexpr int STAGE = U * (NW * W_BYTES + X_BYTES);
    static constexpr int STAGES = (204 * 1024) / STAGE;
    static constexpr int BUFS = NW * NT * 2 <= 512 ? 2 : 1;
    static constexpr uint32_t COLS = NW * NT * BUFS < 32 ? 32 : NW * NT * BUFS;
};

template <int NT, int NW>
struct I8StreamSmem {
    using Cfg = I8StreamCfg<NT, NW>;
    uint8_t st[Cfg::STAGES][Cfg::STAGE];              // 1024-aligned
    uint64_t full[Cfg::STAGES], empty[Cfg::STAGES];
    uint64_t d_full[2], d_empty[2], drain, parts;
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
    float* g;            // scaled gradients [M][ldg], the up half at + up_off
    int64_t ldg, up_off;
    int M, N, K, y_bf16;
    uint32_t* err;
    uint32_t* counters;  // zero between calls
    int32_t* slots;      // partial sums
};

// What a sum (or a pair of sums) becomes.  MODE 0: the product, 1: the gated
// product, 2: the gradients of gate and up, plain (v) and scaled (g).
struct I8Value {
    float v, v1, g, g1;
};
template <int MODE, int ACT>
__device__ __forceinline__ I8Value i8_value(int acc0, int acc1, float ws0, float ws1, float xs, float dh) {
    I8Value o{};
    o.v = ((float)acc0 * ws0) * xs;
    if (MODE > 0) {
        const float b = ((float)acc1 * ws1) * xs;
        const Gate gt = gate_eval<ACT>(o.v);
        if (MODE == 1) {
            o.v = gt.act * b;
        } else {
            o.v = dh * b * gt.grad;
            o.v1 = dh * gt.act;
            o.g = o.v * ws0;
            o.g1 = o.v1 * ws1;
        }
    }
    return o;
}

// A column of outputs: channel n of tokens m, m + 1, ..., with the addresses
// counted along (64-bit products for every element cost more than its
// arithmetic).
template <int MODE>
struct I8Column {
    uint8_t* y;
    const uint16_t* dh;
    uint16_t *d0, *d1;
    float* g;
    int64_t ystep, dhstep, dstep, gstep, up_off;
    bool bf16;

    __device__ __forceinline__ I8Column(const I8Product& p, int64_t m, int64_t n) {
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
    __device__ __forceinline__ float next_dh() {
        const float v = I8Elem<true>::get(*dh);
        dh += dhstep;
        return v;
    }
    // The first `left` of N values.  Values are computed before, without a
    // branch between them, so that their latencies overlap.
    template <int N>
    __device__ __forceinline__ void put(const I8Value (&o)[N], int left) {
        if (MODE < 2) {
            if (bf16) {
#pragma unroll
                for (int i = 0; i < N; ++i, y += ystep)
                    if (i < left) *reinterpret_cast<uint16_t*>(y) = (uint16_t)pack_bf16(o[i].v, 0.f);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i, y += ystep)
                    if (i < left) *reinterpret_cast<float*>(y) = o[i].v;
            }
            return;
        }
        if (d0) {
#pragma unroll
            for (int i = 0; i < N; ++i, d0 += dstep, d1 += dstep)
                if (i < left) {
                    *d0 = (uint16_t)pack_bf16(o[i].v, 0.f);
                    *d1 = (uint16_t)pack_bf16(o[i].v1, 0.f);
                }
        }
#pragma unroll
        for (int i = 0; i < N; ++i, g += gstep)
            if (i < left) {
                g[0] = o[i].g;
                g[up_off] = o[i].g1;
            }
    }
};

// The work of `workers` CTAs or pairs: `full` rounds of whole tiles, then the
// `rem` tiles left, in `cuts` equal pieces each (worker w: piece w), or with
// cuts = 0 as equal runs over all their chunks.
struct I8Plan {
    int full, rem, cuts, workers;
    int cluster;   // the pieces of a tile are the CTAs of a cluster (k_i8_stream, full = 0)
};
// A worker's j-th segment: a tile, its chunks [k0, k1), and the contributors
// c0 .. c1 to that tile.
struct I8Seg {
    int64_t tile;
    int k0, k1, c0, c1;
};
struct I8Work {
    const I8Plan& p;
    int w, chunks, segs;
    int64_t u0, u1;   // the run (cuts = 0)
    __device__ __forceinline__ I8Work(const I8Plan& plan, int worker, int chunks_) : p(plan), w(worker), chunks(chunks_) {
        segs = p.full;
        u0 = u1 = 0;
        if (p.cuts > 0) {
            segs += w < p.rem * p.cuts ? 1 : 0;
        } else {
            const int64_t units = (int64_t)p.rem * chunks;
            u0 = w * units / p.workers;
            u1 = (w + 1) * units / p.workers;
            if (u1 > u0) segs += (int)((u1 - 1) / chunks - u0 / chunks) + 1;
        }
    }
    // the worker whose run holds unit u
    __device__ __forceinline__ int run_of(int64_t u) const {
        return (int)(((u + 1) * p.workers - 1) / ((int64_t)p.rem * chunks));
    }
    __device__ __forceinline__ I8Seg seg(int j) const {
        I8Seg s;
        if (j < p.full) {
            s.tile = (int64_t)j * p.workers + w;
            s.k0 = 0;
            s.k1 = chunks;
            s.c0 = s.c1 = w;
            return s;
        }
        if (p.cuts > 0) {
            const int t = w / p.cuts, piece = w - t * p.cuts;
            s.tile = (int64_t)p.full * p.workers + t;
            s.k0 = (int)((int64_t)piece * chunks / p.cuts);
            s.k1 = (int)((int64_t)(piece + 1) * chunks / p.cuts);
            s.c0 = t * p.cuts;
            s.c1 = s.c0 + p.cuts - 1;
            return s;
        }
        const int64_t t = u0 / chunks + (j - p.full), t0 = t * chunks;
        s.tile = (int64_t)p.full * p.workers + t;
        s.k0 = (int)(max(u0, t0) - t0);
        s.k1 = (int)(min(u1, t0 + chunks) - t0);
        s.c0 = run_of(t0);
        s.c1 = run_of(t0 + chunks - 1);
        return s;
    }
    // Worker c's slot for a tile with first contributor c0: a run has two, one
    // for the tile it enters in the middle and one for the tile it starts.
    __device__ __forceinline__ int slot(int c, int c0) const { return p.cuts > 0 ? c : 2 * c + (c == c0 ? 1 : 0); }
};

template <int NT, int MODE, int ACT>
__global__ void __launch_bounds__(I8S_WARPS * 32, 1)
k_i8_stream(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap0,
            const __grid_constant__ CUtensorMap wmap1, I8Product p, I8Plan plan) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    using Cfg = I8StreamCfg<NT, NW>;
    constexpr int S = Cfg::STAGES, BUFS = Cfg::BUFS, U = Cfg::U;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    I8StreamSmem<NT, NW>& sm = *reinterpret_cast<I8StreamSmem<NT, NW>*>(base);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int KB = (p.K + U * I8_KC - 1) / (U * I8_KC);   // stages of a tile
    const int T = (p.N + 127) / 128, cta = blockIdx.x;
    const I8Work work(plan, cta, KB);
    const int n_segs = work.segs;

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
        mbar_init(&sm.parts, (uint32_t)(max(plan.cuts, 1) * I8S_EPI));
        sm.abort_flag = 0;
        fence_mbar_init();
        i8_tma_prefetch(&xmap);
        i8_tma_prefetch(&wmap0);
        if (NW == 2) i8_tma_prefetch(&wmap1);
    }
    if (warp == 1) i8_tmem_alloc<false>(&sm.tmem, Cfg::COLS);
    i8_fence_before();
    __syncthreads();
    if (plan.cluster) cluster_sync();   // the peers' barriers are ready
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
        for (int j = 0; j < n_segs && ok; ++j) {
            const I8Seg g = work.seg(j);
            const int n0 = (int)(g.tile % T) * 128, m0 = (int)(g.tile / T) * NT;
            for (int kb = g.k0; kb < g.k1; ++kb) {
                ok = i8_wait_warp(&sm.empty[s], ph);
                if (!ok) break;
                ++armed;
                if (issuer) {
                    mbar_arrive_expect_tx(&sm.full[s], Cfg::STAGE);
                    if (!kI8WaitTest) {
                        const uint32_t bar = smem_u32(&sm.full[s]);
#pragma unroll
                        for (int q = 0; q < U; ++q) {   // (a chunk behind the last reads as zeros)
                            const int kc = (kb * U + q) * I8_KC;
                            uint8_t* w = sm.st[s] + q * NW * Cfg::W_BYTES;
                            i8_tma_load<false>(w, &wmap0, kc, n0, bar);
                            if (NW == 2) i8_tma_load<false>(w + Cfg::W_BYTES, &wmap1, kc, n0, bar);
                            i8_tma_load<false>(sm.st[s] + U * NW * Cfg::W_BYTES + q * Cfg::X_BYTES, &xmap, kc, m0, bar);
                        }
                    }
                }
                if (kI8WaitTest) break;   // armed, no copy
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            if (kI8WaitTest) break;
        }
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t idesc = i8_idesc(128, NT);
        const bool issuer = elect_one();
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int j = 0; j < n_segs && ok; ++j) {
            const I8Seg g = work.seg(j);
            const int n = g.k1 - g.k0, buf = j % BUFS;
            ok = i8_wait_warp(&sm.d_empty[buf], ((uint32_t)(j / BUFS) & 1u) ^ 1u);
            if (!ok) break;
            i8_fence_after();
            for (int i = 0; i < n; ++i) {
                ok = i8_wait_warp(&sm.full[s], ph);
                if (!ok) break;
                i8_fence_after();
                const uint32_t st = smem_u32(sm.st[s]);
                if (issuer) {
#pragma unroll
                    for (int q = 0; q < U; ++q)
#pragma unroll
                        for (int j = 0; j < NW; ++j)
                            i8_mma4<false, 0>(tmem + (uint32_t)((buf * NW + j) * NT), st + (q * NW + j) * Cfg::W_BYTES,
                                              st + U * NW * Cfg::W_BYTES + q * Cfg::X_BYTES, idesc, i > 0 || q > 0);
                    i8_commit<false>(&sm.empty[s]);
                    if (i == n - 1) i8_commit<false>(&sm.d_full[buf]);
                }
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok && issuer) timed_out();
        __syncwarp();
    } else {
        const int quad = warp & 3, part = (warp - 2) >> 2;
        for (int seg = 0; seg < n_segs; ++seg) {
            const I8Seg g = work.seg(seg);
            const int buf = seg % BUFS;
            const int n = (int)(g.tile % T) * 128 + quad * 32 + lane, m0 = (int)(g.tile / T) * NT;
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
            const int c0 = g.c0, c1 = g.c1;
            auto slot_of = [&](int c) {
                return p.slots + (size_t)work.slot(c, c0) * (NW * NT * 128) + quad * 32 + lane;
            };
            // This CTA's sums of columns c .. c + 7, and the outputs of eight
            // columns.  What the outputs need is loaded first (a store may
            // alias it for all the compiler knows, and each load would wait
            // for the store before).
            auto own_sums = [&](int c, uint32_t (&r)[NW][8]) {
#pragma unroll
                for (int j = 0; j < NW; ++j) i8_tmem_ld8(taddr + (uint32_t)(j * NT + c), r[j]);
                i8_tmem_wait();
            };
            auto finish = [&](int c, auto&& sums) {
                const int left = mc - c;
                float xs[8], dh[MODE == 2 ? 8 : 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) xs[i] = i < left ? p.xs[m0 + c + i] : 0.f;
                I8Column<MODE> col(p, m0 + c, in ? n : 0);
                if (MODE == 2)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dh[MODE == 2 ? i : 0] = i < left ? col.next_dh() : 0.f;
                int acc[NW][8] = {};
                sums(c, left, acc);
                I8Value o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = i8_value<MODE, ACT>(acc[0][i], acc[NW - 1][i], ws0, ws1, xs[i], dh[MODE == 2 ? i : 0]);
                if (in) col.put(o, left);
                __syncwarp();
            };
            if (c0 != c1 && plan.cluster) {
                // columns go to part + lane of [NW NT][128] words in every CTA's first stages
                const uint32_t part0 = smem_u32(sm.st[0]) + (uint32_t)(quad * 32 + lane) * 4u;
                for (int c = 8 * part; c < mc; c += 32) {
                    uint32_t r[NW][8];
                    own_sums(c, r);
#pragma unroll
                    for (int j = 0; j < NW; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(part0 + (uint32_t)(j * NT + c + i) * 512u), "r"(r[j][i])
                                         : "memory");
                }
                __syncwarp();
                if (lane < plan.cuts) cluster_arrive_release(cluster_addr(&sm.parts, (uint32_t)lane));
                if (!__all_sync(0xffffffffu, i8_wait<true>(&sm.parts, 0u))) {
                    if (lane == 0) timed_out();
                    break;
                }
                const int rank = cta - c0, step = 8 * plan.cuts;
                for (int c = 8 * rank + step * part; c < mc; c += 4 * step)
                    finish(c, [&](int c, int, int (&acc)[NW][8]) {
                        for (int o = 0; o < plan.cuts; o += 4 / NW) {   // some peers' loads in flight
                            uint32_t t[4 / NW][NW][8];
#pragma unroll
                            for (int q = 0; q < 4 / NW; ++q) {
                                const uint32_t peer = cluster_map(part0, (uint32_t)min(o + q, plan.cuts - 1));
#pragma unroll
                                for (int j = 0; j < NW; ++j)
#pragma unroll
                                    for (int i = 0; i < 8; ++i) t[q][j][i] = cluster_load(peer + (uint32_t)(j * NT + c + i) * 512u);
                            }
#pragma unroll
                            for (int q = 0; q < 4 / NW; ++q)
                                if (o + q < plan.cuts)
#pragma unroll
                                    for (int j = 0; j < NW; ++j)
#pragma unroll
                                        for (int i = 0; i < 8; ++i) acc[j][i] += (int)t[q][j][i];
                        }
                    });
            } else {
                // A tile cut between CTAs that are no cluster: when all others
                // have arrived already, this one only adds; else it leaves its
                // part and counts itself in.
                uint32_t* counter = p.counters + c0 * I8S_EPI + warp - 2;
                const uint32_t others = (uint32_t)(c1 - c0);
                bool mine = 8 * part < mc;   // this warp writes the results
                if (mine && c0 != c1) {
                    uint32_t seen = 0;
                    if (lane == 0) seen = i8_load_acquire(counter);
                    if (__shfl_sync(0xffffffffu, seen, 0) != others) {
                        int32_t* slot = slot_of(cta);
                        for (int c = 8 * part; c < mc; c += 32) {
                            uint32_t r[NW][8];
                            own_sums(c, r);
#pragma unroll
                            for (int j = 0; j < NW; ++j)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (c + i < mc) slot[(j * NT + c + i) * 128] = (int)r[j][i];
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
                for (int c = 8 * part; mine && c < mc; c += 32)
                    finish(c, [&](int c, int left, int (&acc)[NW][8]) {
                        if (c0 != c1)
                            for (int o = c0; o <= c1; o += 2) {   // two contributors' loads in flight
                                int t[2][NW][8];
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    const bool add = o + q <= c1 && o + q != cta;
                                    const int32_t* slot = slot_of(o + q);
#pragma unroll
                                    for (int j = 0; j < NW; ++j)
#pragma unroll
                                        for (int i = 0; i < 8; ++i)
                                            t[q][j][i] = add && i < left ? __ldcg(slot + (j * NT + c + i) * 128) : 0;
                                }
#pragma unroll
                                for (int q = 0; q < 2; ++q)
#pragma unroll
                                    for (int j = 0; j < NW; ++j)
#pragma unroll
                                        for (int i = 0; i < 8; ++i) acc[j][i] += t[q][j][i];
                            }
                        uint32_t r[NW][8];
                        own_sums(c, r);
#pragma unroll
                        for (int j = 0; j < NW; ++j)
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[j][i] += (int)r[j][i];
                    });
            }
            i8_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.d_empty[buf]);
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
    if (sm.abort_flag && plan.cluster) i8_settle();
    i8_fence_before();
    __syncthreads();
    if (plan.cluster) cluster_sync();   // nobody reads this CTA's part any more
    if (warp == 1) {
        i8_fence_after();
        i8_tmem_free<false>(tmem, Cfg::COLS);
    }
}

}  // namespace mpq
