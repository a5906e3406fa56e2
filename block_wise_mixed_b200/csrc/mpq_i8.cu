// mpq_i8.cu -- the C ABI of the 8-bit integer operators (include/mpq.h):
// argument checks, workspace layout and launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/mpq.h"
#include "common.cuh"
#include "i8_gate.cuh"
#include "k_i8_dx.cuh"
#include "k_i8_rows.cuh"
#include "k_i8_stream.cuh"
#include "k_i8_tile.cuh"

using namespace mpq;

namespace {

constexpr int kSMs = 148;

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

mpq_status check_i8(const mpq_i8* q) {
    if (!q) return MPQ_ERR_ARG;
    if (q->rows < 0 || q->cols < 1 || q->cols > MPQ_I8_MAX_COLS) return MPQ_ERR_SHAPE;
    if (q->ld < q->cols || q->ld % 16 != 0 || q->ld >= ((int64_t)1 << 40)) return MPQ_ERR_ARG;
    if (q->rows == 0) return MPQ_OK;
    if (!q->codes || !q->scales || !aligned(q->codes, 16) || !aligned(q->scales, 4)) return MPQ_ERR_ARG;
    return MPQ_OK;
}

inline uintptr_t elem_size(mpq_ydtype dt) { return dt == MPQ_Y_BF16 ? 2 : 4; }
inline bool dtype_ok(mpq_ydtype dt) { return dt == MPQ_Y_F32 || dt == MPQ_Y_BF16; }
inline bool act_ok(mpq_act a) { return a == MPQ_ACT_SILU || a == MPQ_ACT_GELU_TANH; }

// A rows x cols array of elements of `size` bytes, ld elements a row.
mpq_status check_array(const void* p, uintptr_t size, int64_t ld, int64_t cols) {
    if (!p || !aligned(p, size) || ld < cols) return MPQ_ERR_ARG;
    return MPQ_OK;
}

mpq_status check_ws(const void* ws, size_t have, size_t need) {
    return !ws || !aligned(ws, 256) || have < need ? MPQ_ERR_WORKSPACE : MPQ_OK;
}

// Every launch may overlap the end of the kernel before it (programmatic
// dependent launch).  The kernels read and write global memory only after
// griddepcontrol.wait, and let their dependents start only after it.
template <typename... KArgs, typename... Args>
mpq_status launch_cluster(int cluster, void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, void* stream,
                          Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = static_cast<cudaStream_t>(stream);
    c.attrs = attr;
    c.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, std::forward<Args>(args)...) == cudaSuccess ? MPQ_OK : MPQ_ERR_CUDA;
}
template <typename... KArgs, typename... Args>
mpq_status launch(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, void* stream, Args&&... args) {
    return launch_cluster(0, kernel, grid, threads, smem, stream, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
template <bool BF16, bool SHIFT, int G, int VPT, bool LONG = false>
mpq_status quantize_run(const I8RowsParams& p, void* stream) {
    constexpr int threads = G >= 128 ? G : 128;
    static const int resident = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_i8_quantize<BF16, SHIFT, G, VPT, LONG>, threads, 0) ==
                       cudaSuccess && n > 0 ? n : 1;
    }();
    const int64_t blocks = std::min<int64_t>(div_up(p.rows, threads / G), (int64_t)kSMs * resident);
    return launch(k_i8_quantize<BF16, SHIFT, G, VPT, LONG>, dim3((unsigned)blocks), threads, 0, stream, p);
}

// Threads a row: as few as hold it in four 16-byte blocks each (rows of 1000
// bf16: 4.3 us for 4096 of them, 7.0 with eight), eight from 32 KB on; for a few
// rows, as many as have a block to load.
template <bool BF16, bool SHIFT>
mpq_status quantize_launch(const I8RowsParams& p, void* stream) {
    const int64_t warps = div_up(div_up(p.cols, I8Elem<BF16>::PER) + (SHIFT ? 1 : 0), SHIFT ? 31 : 32);
    const int64_t per = p.rows <= kSMs ? 1 : 4;
    if (warps > 16 * 8) return quantize_run<BF16, SHIFT, 512, 8, true>(p, stream);
    if (warps > 16 * 4) return quantize_run<BF16, SHIFT, 512, 8>(p, stream);
    if (warps > 8 * per) return quantize_run<BF16, SHIFT, 512, 4>(p, stream);
    if (warps > 4 * per) return quantize_run<BF16, SHIFT, 256, 4>(p, stream);
    if (warps > per) return quantize_run<BF16, SHIFT, 128, 4>(p, stream);
    return quantize_run<BF16, SHIFT, 32, 4>(p, stream);
}

}  // namespace

extern "C" {

mpq_status mpq_i8_quantize(const void* x_dev, mpq_ydtype dt, int64_t ldx, const mpq_i8* out, void* stream) {
    mpq_status st = check_i8(out);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(dt)) return MPQ_ERR_ARG;
    if (out->rows == 0) return MPQ_OK;
    const uintptr_t es = elem_size(dt);
    st = check_array(x_dev, es, ldx, out->cols);
    if (st != MPQ_OK) return st;
    I8RowsParams p{};
    p.x = x_dev;
    p.codes = const_cast<int8_t*>(out->codes);
    p.scales = const_cast<float*>(out->scales);
    p.ldx = ldx;
    p.ldc = out->ld;
    p.rows = out->rows;
    p.cols = out->cols;
    const bool vec = aligned(x_dev, 16) && (out->rows == 1 || ldx * (int64_t)es % 16 == 0) &&
                     out->cols * (int64_t)es % 16 == 0;   // rows are whole 16-byte blocks
    if (dt == MPQ_Y_BF16) return vec ? quantize_launch<true, false>(p, stream) : quantize_launch<true, true>(p, stream);
    return vec ? quantize_launch<false, false>(p, stream) : quantize_launch<false, true>(p, stream);
}

mpq_status mpq_i8_dequantize(const mpq_i8* q, void* x_dev, mpq_ydtype dt, int64_t ldx, void* stream) {
    mpq_status st = check_i8(q);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(dt)) return MPQ_ERR_ARG;
    if (q->rows == 0) return MPQ_OK;
    const uintptr_t es = elem_size(dt);
    st = check_array(x_dev, es, ldx, q->cols);
    if (st != MPQ_OK) return st;
    I8RowsParams p{};
    p.y = x_dev;
    p.codes = const_cast<int8_t*>(q->codes);
    p.scales = const_cast<float*>(q->scales);
    p.ldx = ldx;
    p.ldc = q->ld;
    p.rows = q->rows;
    p.cols = q->cols;
    const bool vec = aligned(x_dev, 16) && (q->rows == 1 || ldx * (int64_t)es % 16 == 0);
    const int64_t per = 256 * (vec ? 4 * 16 / (int64_t)es : 32);   // a block's columns in one round
    const dim3 grid((unsigned)q->rows, (unsigned)div_up(q->cols, per));
    if (dt == MPQ_Y_BF16) return vec ? launch(k_i8_dequantize<true, true>, grid, 256, 0, stream, p)
                                     : launch(k_i8_dequantize<true, false>, grid, 256, 0, stream, p);
    return vec ? launch(k_i8_dequantize<false, true>, grid, 256, 0, stream, p)
               : launch(k_i8_dequantize<false, false>, grid, 256, 0, stream, p);
}

}  // extern "C"

namespace {

constexpr int kPairs = kSMs / 2;
// Workspace: the error word, the counters (zero between calls), then scratch
// that a call writes before it reads.  The zeroed part has one size for all
// mpq_i8_* calls, so one workspace serves them all, one after another.
constexpr size_t kErrBytes = 256;
constexpr size_t kI8ZeroBytes = MPQ_I8_WS_ZERO;   // I8S_EPI counters for each CTA (a pair: 2 I8X_EPI)
constexpr size_t kCounterBytes = kI8ZeroBytes - kErrBytes;
static_assert(kSMs * I8S_EPI * 4 <= kCounterBytes && kPairs * 2 * I8X_MAX_EPI * 4 <= kCounterBytes &&
              kI8ZeroBytes % 256 == 0, "counters");

inline bool shape_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 1 && K >= 1 && K <= MPQ_I8_MAX_COLS;
}

// Pieces that a tile of `chunks` stages may be cut into: a stage costs about as
// long as the last contributor takes to add 14 columns of one more partial sum,
// so n pieces cost chunks / n + n cols / 14, least at n = sqrt(14 chunks / cols).
inline int64_t max_cuts(int64_t chunks, int64_t cols) {
    return std::max<int64_t>(1, (int64_t)std::ceil(std::sqrt(14.0 * (double)chunks / (double)cols)));
}
// What it costs to add up a tile between the CTAs of a cluster.
inline double cluster_fix_us(int64_t cols) { return 2.0 + 0.02 * (double)cols; }

// chunk_us: a stage's time; fix_us: what adding up a tile that is cut through
// global memory costs.  Cuts, or equal runs, only where the time they take off
// is worth more (measured: 16-token gradient of 8192 x 28672, 112 tiles on 74
// pairs: 55 us in runs, 62 whole; one token through 14336 x 4096: 16.8 us in runs,
// 13.6 whole).
I8Plan make_plan(int64_t tiles, int64_t chunks, int64_t cols, int workers, double chunk_us, double fix_us,
                 bool clusters) {
    I8Plan p{};
    p.full = (int)(tiles / workers);
    p.rem = (int)(tiles % workers);
    p.cuts = 1;
    const double tile_us = (double)chunks * chunk_us;
    if (clusters && p.full == 0 && p.rem > 0 && workers / p.rem >= 2) {   // (no tiles: an empty batch)
        // All clusters at once: the occupancy query gives 74, 45, 33, 26, 22, 15
        // and 15 clusters of 2 to 8 CTAs; a few less here, as a second wave
        // costs more than smaller clusters (2048 x 2048: 10.7 us in 16 of 8).
        static const int kFit[9] = {0, 0, 72, 44, 32, 24, 20, 14, 14};
        int n = (int)std::min<int64_t>({workers / p.rem, chunks, 8});
        while (n > 1 && kFit[n] < p.rem) --n;
        if (n > 1 && tile_us * (n - 1) / n > cluster_fix_us(cols)) {
            p.cuts = n;
            p.cluster = 1;
            p.workers = p.rem * n;
            return p;
        }
    }
    if (p.rem) {
        const int n = (int)std::min<int64_t>({workers / p.rem, chunks, max_cuts(chunks, cols)});
        if (n > 1 && tile_us * (n - 1) / n > fix_us) p.cuts = n;
        if (workers / p.rem == 1 && tile_us * (workers - p.rem) / workers > fix_us) p.cuts = 0;
    }
    p.workers = p.full || p.cuts == 0 ? workers : p.rem * p.cuts;
    return p;
}

// Stages of the worker that has most.
inline double stages_each(const I8Plan& p, int64_t chunks, int workers) {
    return (double)p.full * chunks +
           (p.rem == 0 ? 0.0 : p.cuts == 0 ? (double)p.rem * chunks / workers : (double)chunks / p.cuts);
}

// Which kernel makes a product, and how.
struct ProductPlan {
    int nt;        // tokens per tile of k_i8_stream; 0: k_i8_tile
    I8Plan work;   // (k_i8_stream)
};
// The smaller estimate, in us, fitted to what was measured on shapes from 1 to
// 512 tokens and 1000 to 28672 channels: a stage of k_i8_stream takes 0.0078 a
// KB, 0.30 at least (two chunks of one matrix), or 0.0115 a KB (one of two),
// unless the weights take longer (6.2 TB/s from HBM, half as long from L2 for
// each further tile of tokens); adding cut tiles up costs
// what make_plan says; k_i8_tile takes 0.36 a chunk of its 256 x 256 tiles and
// a quarter more than HBM's time.  Few tokens per tile make more tiles where
// there are few channels (128 tokens, 4096 x 4096: 9.8 us with 32, 14.5 with 16,
// 10.9 with 64 or 128), many read the weights once (64 tokens, 14336 x 4096:
// 28.6 us with 16, 14.3 with 64).
ProductPlan product_plan(int64_t M, int64_t N, int64_t K, int nw) {
    const int u = nw == 1 ? I8StreamCfg<16, 1>::U : I8StreamCfg<16, 2>::U;
    const int64_t chunks = div_up(K, u * I8_KC);
    const int64_t tiles = div_up(M, 256) * div_up(N, 256 / nw);
    ProductPlan best{0, {}};
    const double hbm_us = (double)N * (double)K * nw / 6.2e6;
    double best_us = 7.0 + std::max(1.25 * hbm_us, (double)(div_up(tiles, kPairs) * div_up(K, I8_KC)) * 0.36);
    for (int nt = 16; nt <= 128; nt *= 2) {
        if (nt > 16 && nt >= 2 * M) break;
        const int64_t t = div_up(M, nt) * div_up(N, 128), cols = std::min<int64_t>(M, nt) * nw;
        if (t > 16 * kSMs) continue;   // far into k_i8_tile's range
        const double kb = (double)(u * (16 * nw + nt / 8));
        const double stage_us = nw == 1 ? std::max(0.30, 0.0078 * kb) : 0.0115 * kb;
        const double fix_us = 5.0 + 0.08 * cols;
        const I8Plan p = make_plan(t, chunks, cols, kSMs, stage_us, fix_us, true);
        const double each = stages_each(p, chunks, kSMs);
        const double read_us = hbm_us * (1.0 + 0.5 * (double)(div_up(M, nt) - 1));
        const double us = std::max(read_us, each * stage_us) + 4.0 + 0.02 * cols +
                          (p.cuts == 1 ? 0.0 : p.cluster ? cluster_fix_us(cols) : fix_us);
        if (us < best_us) {
            best_us = us;
            best = {nt, p};
        }
    }
    return best;
}

// Tokens per tile of the gradient kernel, and its work.  As above: a stage takes
// 0.42, 0.45 or 0.55 us (two 64-channel blocks, 32, 64 or 128 tokens) or 0.34
// (one block, 256 tokens); adding up a cut tile 5 + 0.045 a column (256 tokens,
// 4096 x 4096: 29 us in tiles of 256 cut in four, 24 in whole tiles of 64).
struct DxPlan {
    int nt;
    I8Plan work;
};
// Gradients in two fp16 parts up to here (see k_i8_dx.cuh): tiles of 32 columns
// then hold 16 tokens.
constexpr int kDxSplitM = 16;
inline int grad_parts(int64_t M) { return M <= kDxSplitM ? 2 : 1; }

DxPlan dx_plan(int64_t M, int64_t N, int64_t K, int nw) {
    static const double kStage[4] = {0.42, 0.45, 0.55, 0.34};
    DxPlan best{};
    double best_us = 0.0;
    for (int i = 0; i < 4; ++i) {
        const int nt = 32 << i, u = nt == 256 ? I8DxCfg<256>::U : I8DxCfg<32>::U;
        const int64_t tok = nt / grad_parts(M);
        if (i > 0 && tok >= 2 * M) break;
        const int64_t chunks = div_up(N, I8X_NC * u) * nw, cols = std::min<int64_t>(M, tok);
        const double fix_us = 5.0 + 0.045 * cols;
        const I8Plan p = make_plan(div_up(M, tok) * div_up(K, 256), chunks, cols, kPairs, kStage[i], fix_us, false);
        const double us = stages_each(p, chunks, kPairs) * kStage[i] + 0.02 * cols + (p.cuts == 1 ? 0.0 : fix_us);
        if (i == 0 || us < best_us) {
            best_us = us;
            best = {nt, p};
        }
    }
    return best;
}
inline int64_t plan_slots(const I8Plan& p) {
    return p.cuts == 0 ? 2 * p.workers : p.cuts == 1 || p.cluster ? 0 : (int64_t)p.rem * p.cuts;
}

// Partial sums: 128 lanes x NT columns a slot.
inline size_t product_slots(int64_t M, int64_t N, int64_t K, int nw) {
    const ProductPlan p = product_plan(M, N, K, nw);
    return p.nt == 0 ? 0 : (size_t)plan_slots(p.work) * nw * p.nt * 128 * 4;
}
inline size_t dx_slots(int64_t M, int64_t N, int64_t K, int nw) {
    const DxPlan p = dx_plan(M, N, K, nw);
    return (size_t)plan_slots(p.work) * 2 * p.nt * 128 * 4;
}

// The most slots that any call of up to M tokens takes: equal runs (two for each
// worker) of the widest tiles that M allows.
inline size_t product_slots_upto(int64_t M, int nw) {
    int64_t nt = 16;
    while (nt < 128 && nt < M) nt *= 2;
    return (size_t)2 * kSMs * nw * nt * 128 * 4;
}
inline size_t dx_slots_upto(int64_t M) {
    int64_t nt = 32;
    while (nt < 256 && nt < M) nt *= 2;
    return (size_t)2 * kPairs * 2 * nt * 128 * 4;
}
// Rows of gradients (in two parts up to kDxSplitM tokens).
inline size_t grad_rows_upto(int64_t M) {
    return (size_t)std::max<int64_t>(M, 2 * std::min<int64_t>(M, kDxSplitM));
}

inline int64_t grad_ld(int64_t n) { return div_up(n, 64) * 64; }

struct I8Ws {
    uint32_t* err;
    uint32_t* counters;
    void* slots;
    uint16_t* grads;     // the gradient product's fp16 operand
    float* grads32;      // the gated product's scaled gradients
    float* unscale;      // one a token
    size_t bytes;
};
I8Ws carve(void* ws, size_t slots, size_t grads, size_t grads32, size_t unscale) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    I8Ws w{};
    const size_t after = kI8ZeroBytes + round256(slots), after16 = after + round256(grads),
                 after32 = after16 + round256(grads32);
    w.bytes = after32 + round256(unscale);
    if (!b) return w;
    w.err = reinterpret_cast<uint32_t*>(b);
    w.counters = reinterpret_cast<uint32_t*>(b + kErrBytes);
    w.slots = b + kI8ZeroBytes;
    w.grads = reinterpret_cast<uint16_t*>(b + after);
    w.grads32 = reinterpret_cast<float*>(b + after16);
    w.unscale = reinterpret_cast<float*>(b + after32);
    return w;
}

I8Ws ws_product(void* ws, int64_t M, int64_t N, int64_t K, int nw) {
    return carve(ws, product_slots(M, N, K, nw), 0, 0, 0);
}
// nw matrices: the product's slots (gated) and the gradient's share their place.
I8Ws ws_backward(void* ws, int64_t M, int64_t N, int64_t K, int nw) {
    const size_t ps = nw == 2 ? product_slots(M, N, K, 2) : 0;
    const size_t row = (size_t)grad_ld(N) * (size_t)nw;
    return carve(ws, std::max(ps, dx_slots(M, N, K, nw)), (size_t)M * grad_parts(M) * row * 2,
                 nw == 2 ? (size_t)M * row * 4 : 0, (size_t)M * 4);
}

// For any call of up to M tokens: the layouts above with the most that a part may take.
size_t bytes_product(int64_t M, int nw) { return carve(nullptr, product_slots_upto(M, nw), 0, 0, 0).bytes; }
size_t bytes_backward(int64_t M, int64_t N, int nw) {
    const size_t ps = nw == 2 ? product_slots_upto(M, 2) : 0, row = (size_t)grad_ld(N) * (size_t)nw;
    return carve(nullptr, std::max(ps, dx_slots_upto(M)), grad_rows_upto(M) * row * 2, nw == 2 ? (size_t)M * row * 4 : 0,
                 (size_t)M * 4).bytes;
}

// x and the weights of a product: common columns, at least one channel.
mpq_status check_product(const mpq_i8* x, const mpq_i8* const* w, int nw) {
    mpq_status st = check_i8(x);
    if (st != MPQ_OK) return st;
    for (int i = 0; i < nw; ++i) {
        st = check_i8(w[i]);
        if (st != MPQ_OK) return st;
        if (w[i]->cols != x->cols || w[i]->rows < 1 || w[i]->rows != w[0]->rows) return MPQ_ERR_SHAPE;
    }
    return MPQ_OK;
}

// ---------------------------------------------------------------------------
// tensor maps
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// rows x cols elements, ld bytes a row, boxes of box_rows x 128 bytes; what
// lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* ptr, bool f16, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              bool swizzle) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {f16 ? 64u : 128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
               const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_map(CUtensorMap* map, const mpq_i8* q, int box_rows, bool swizzle) {
    return make_map(map, q->codes, false, q->rows, q->cols, q->ld, box_rows, swizzle);
}

// Launches with all the shared memory a kernel asks for (raised once per device).
template <auto Kernel, typename... Args>
mpq_status launch_big(int cluster, dim3 grid, int threads, size_t smem, void* stream, Args&&... args) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MPQ_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return MPQ_ERR_CUDA;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_cluster(cluster, Kernel, grid, threads, smem, stream, std::forward<Args>(args)...);
}

template <int NT, int MODE, int ACT>
mpq_status stream_run(const mpq_i8* x, const mpq_i8* const* w, const I8Product& p, const I8Plan& plan, void* stream) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    CUtensorMap xm, w0, w1;
    if (!make_map(&xm, x, NT, true) || !make_map(&w0, w[0], 128, true) || !make_map(&w1, w[NW - 1], 128, true))
        return MPQ_ERR_CUDA;
    return launch_big<k_i8_stream<NT, MODE, ACT>>(plan.cluster ? plan.cuts : 0, dim3((unsigned)plan.workers), I8S_WARPS * 32,
                                                  sizeof(I8StreamSmem<NT, NW>) + 1024, stream, xm, w0, w1, p, plan);
}

template <int MODE, int ACT>
mpq_status tile_run(const mpq_i8* x, const mpq_i8* const* w, const I8Product& p, void* stream) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    CUtensorMap xm, w0, w1;
    if (!make_map(&xm, x, 128, true) || !make_map(&w0, w[0], 128, true) || !make_map(&w1, w[NW - 1], 128, true))
        return MPQ_ERR_CUDA;
    const int64_t tiles = div_up(p.M, 256) * div_up(p.N, 256 / NW);
    return launch_big<k_i8_tile<MODE, ACT>>(0, dim3((unsigned)(2 * std::min<int64_t>(kPairs, tiles))), I8T_WARPS * 32,
                                            sizeof(I8TileSmem<MODE>) + 1024, stream, xm, w0, w1, p);
}

template <int MODE, int ACT>
mpq_status product_run(const mpq_i8* x, const mpq_i8* const* w, I8Product& p, const I8Ws& ws, void* stream) {
    p.xs = x->scales;
    p.ws[0] = w[0]->scales;
    p.ws[1] = MODE == 0 ? nullptr : w[1]->scales;
    p.M = x->rows;
    p.N = w[0]->rows;
    p.K = x->cols;
    p.err = ws.err;
    p.counters = ws.counters;
    p.slots = static_cast<int32_t*>(ws.slots);
    const ProductPlan plan = product_plan(p.M, p.N, p.K, MODE == 0 ? 1 : 2);
    switch (plan.nt) {
        case 0: return tile_run<MODE, ACT>(x, w, p, stream);
        case 16: return stream_run<16, MODE, ACT>(x, w, p, plan.work, stream);
        case 32: return stream_run<32, MODE, ACT>(x, w, p, plan.work, stream);
        case 64: return stream_run<64, MODE, ACT>(x, w, p, plan.work, stream);
        default: return stream_run<128, MODE, ACT>(x, w, p, plan.work, stream);
    }
}

template <int NT>
mpq_status dx_run(const mpq_i8* const* w, int nw, const uint16_t* g, int64_t ldg, int64_t up_off, I8DxParams& p,
                  const I8Plan& plan, void* stream) {
    CUtensorMap w0, w1, g0, g1;
    if (!make_map(&w0, w[0], I8DxCfg<NT>::U * I8X_NC, false) || !make_map(&w1, w[nw - 1], I8DxCfg<NT>::U * I8X_NC, false) ||
        !make_map(&g0, g, true, (int64_t)p.M * grad_parts(p.M), p.N, ldg * 2, NT / 2, true) ||
        !make_map(&g1, g + (nw - 1) * up_off, true, (int64_t)p.M * grad_parts(p.M), p.N, ldg * 2, NT / 2, true))
        return MPQ_ERR_CUDA;
    return launch_big<k_i8_dx<NT>>(0, dim3((unsigned)(2 * plan.workers)), I8DxCfg<NT>::WARPS * 32, sizeof(I8DxSmem<NT>) + 1024,
                                   stream, w0, w1, g0, g1, p, plan);
}

// The operand of the gradient product from `src` (SRC as in k_i8_grad_rows).  Many
// short tokens take a warp each (3840 of 64 channels, whole gradient: 9.4 us, 12.2
// with blocks; 64 of 1024: 18.6, 15.5 with blocks).  For others a thread takes
// one unit of 8 columns if all blocks are resident so, else two to four (256
// tokens of 4096 channels: 22.8 us, 25.6 with four; 125 of 18560: 50.5 us with
// two blocks a token in two waves, 47.1 with one); more than 1024 threads a token
// are a cluster, and so are more than 256 where the gradients are more than L2
// holds and smaller blocks keep HBM busier (2240 tokens, gate and up of 22528:
// 583 us, 619 with 1024 threads).
template <int SRC>
mpq_status grad_rows_run(I8GradParams& p, const I8Ws& ws, int64_t M, int64_t N, int64_t ldg, void* stream) {
    p.g = ws.grads;
    p.ldg = ldg;
    p.lo_off = grad_parts(M) == 2 ? M * ldg : 0;
    p.unscale = ws.unscale;
    p.M = (int)M;
    p.N = (int)N;
    const int64_t units = div_up(N, 8) * (SRC == 2 ? 2 : 1);
    if (units <= 4 * 32 && M >= 8 * kSMs)
        return launch(k_i8_grad_rows<SRC, true>, dim3((unsigned)div_up(M, I8G_WARPS)), I8G_WARPS * 32, 0, stream, p);
    const int most = M * units * 8 * (SRC == 2 ? 4 : 2) > (int64_t)126 << 20 ? 8 : 32;   // warps of a block
    int threads = 0;
    for (int each = 1; each <= 4; ++each) {
        const int64_t warps = div_up(units, 32 * each);
        p.cluster = 1;
        while (p.cluster < 8 && p.cluster * most < warps) p.cluster *= 2;
        threads = (int)std::min<int64_t>(1024, div_up(warps, p.cluster) * 32);
        if (M * p.cluster <= (int64_t)kSMs * (1024 / threads)) break;
    }
    return launch_cluster(p.cluster > 1 ? p.cluster : 0, k_i8_grad_rows<SRC, false>, dim3((unsigned)(M * p.cluster)), threads,
                          0, stream, p);
}

mpq_status dx_run(const mpq_i8* const* w, int nw, const uint16_t* g, int64_t ldg, int64_t up_off, int64_t M,
                  void* dx_dev, int64_t lddx, const I8Ws& ws, void* stream) {
    I8DxParams p{};
    p.dx = static_cast<uint16_t*>(dx_dev);
    p.lddx = lddx;
    p.M = (int)M;
    p.N = w[0]->rows;
    p.K = w[0]->cols;
    p.nw = nw;
    p.split = grad_parts(M) == 2;
    p.unscale = ws.unscale;
    p.err = ws.err;
    p.counters = ws.counters;
    p.slots = static_cast<float*>(ws.slots);
    const DxPlan plan = dx_plan(M, p.N, p.K, nw);
    switch (plan.nt) {
        case 32: return dx_run<32>(w, nw, g, ldg, up_off, p, plan.work, stream);
        case 64: return dx_run<64>(w, nw, g, ldg, up_off, p, plan.work, stream);
        case 128: return dx_run<128>(w, nw, g, ldg, up_off, p, plan.work, stream);
        default: return dx_run<256>(w, nw, g, ldg, up_off, p, plan.work, stream);
    }
}

}  // namespace

extern "C" {

size_t mpq_i8_linear_workspace_size(int32_t M, int32_t N, int32_t K) {
    return shape_ok(M, N, K) ? bytes_product(M, 1) : 0;
}
size_t mpq_i8_gated_workspace_size(int32_t M, int32_t F, int32_t K) {
    return shape_ok(M, F, K) ? bytes_product(M, 2) : 0;
}
size_t mpq_i8_linear_backward_workspace_size(int32_t M, int32_t N, int32_t K) {
    return shape_ok(M, N, K) ? bytes_backward(M, N, 1) : 0;
}
size_t mpq_i8_gated_backward_workspace_size(int32_t M, int32_t F, int32_t K) {
    return shape_ok(M, F, K) ? bytes_backward(M, F, 2) : 0;
}

mpq_status mpq_i8_plan(mpq_i8_op op, int32_t M, int32_t N, int32_t K, mpq_i8_work* out) {
    if (!out || op < MPQ_I8_LINEAR || op > MPQ_I8_GATED_BACKWARD) return MPQ_ERR_ARG;
    if (M < 1 || !shape_ok(M, N, K)) return MPQ_ERR_SHAPE;
    out[0] = out[1] = mpq_i8_work{};
    const int nw = op == MPQ_I8_GATED || op == MPQ_I8_GATED_BACKWARD ? 2 : 1;
    auto fill = [](mpq_i8_work& o, int kernel, int columns, const I8Plan& p, size_t slots) {
        o = {kernel, columns, p.workers, p.full, p.rem, p.cuts, p.cluster, slots};
    };
    if (op != MPQ_I8_LINEAR_BACKWARD) {
        const ProductPlan p = product_plan(M, N, K, nw);
        if (p.nt) {
            fill(out[0], MPQ_I8_KERNEL_STREAM, p.nt, p.work, product_slots(M, N, K, nw));
        } else {
            const int64_t tiles = div_up(M, 256) * div_up(N, 256 / nw);
            const int workers = (int)std::min<int64_t>(kPairs, tiles);
            fill(out[0], MPQ_I8_KERNEL_TILE, 256, {(int)(tiles / workers), (int)(tiles % workers), 1, workers, 0}, 0);
        }
    }
    if (op >= MPQ_I8_LINEAR_BACKWARD) {
        const DxPlan p = dx_plan(M, N, K, nw);
        fill(out[1], MPQ_I8_KERNEL_DX, p.nt, p.work, dx_slots(M, N, K, nw));
    }
    return MPQ_OK;
}

mpq_status mpq_i8_linear(const mpq_i8* x, const mpq_i8* w, void* y_dev, mpq_ydtype ydt, int64_t ldy, void* ws,
                         size_t ws_bytes, void* stream) {
    const mpq_i8* wl[1] = {w};
    mpq_status st = check_product(x, wl, 1);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(ydt)) return MPQ_ERR_ARG;
    if (x->rows == 0) return MPQ_OK;
    const I8Ws k = ws_product(ws, x->rows, w->rows, x->cols, 1);
    st = check_array(y_dev, elem_size(ydt), ldy, w->rows);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, bytes_product(x->rows, 1));
    if (st != MPQ_OK) return st;
    I8Product p{};
    p.y = y_dev;
    p.ldy = ldy;
    p.y_bf16 = ydt == MPQ_Y_BF16;
    return product_run<0, MPQ_ACT_SILU>(x, wl, p, k, stream);
}

mpq_status mpq_i8_gated(const mpq_i8* x, const mpq_i8* w_gate, const mpq_i8* w_up, mpq_act act, void* h_dev,
                        mpq_ydtype ydt, int64_t ldh, void* ws, size_t ws_bytes, void* stream) {
    const mpq_i8* wl[2] = {w_gate, w_up};
    mpq_status st = check_product(x, wl, 2);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(ydt) || !act_ok(act)) return MPQ_ERR_ARG;
    if (x->rows == 0) return MPQ_OK;
    const I8Ws k = ws_product(ws, x->rows, w_gate->rows, x->cols, 2);
    st = check_array(h_dev, elem_size(ydt), ldh, w_gate->rows);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, bytes_product(x->rows, 2));
    if (st != MPQ_OK) return st;
    I8Product p{};
    p.y = h_dev;
    p.ldy = ldh;
    p.y_bf16 = ydt == MPQ_Y_BF16;
    return act == MPQ_ACT_SILU ? product_run<1, MPQ_ACT_SILU>(x, wl, p, k, stream)
                               : product_run<1, MPQ_ACT_GELU_TANH>(x, wl, p, k, stream);
}

mpq_status mpq_i8_linear_backward(const mpq_i8* w, const void* dy_dev, int32_t M, int64_t lddy, void* dx_dev,
                                  int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
    mpq_status st = check_i8(w);
    if (st != MPQ_OK) return st;
    if (M < 0 || w->rows < 1) return MPQ_ERR_SHAPE;
    if (M == 0) return MPQ_OK;
    const I8Ws k = ws_backward(ws, M, w->rows, w->cols, 1);
    st = check_array(dy_dev, 2, lddy, w->rows);
    if (st == MPQ_OK) st = check_array(dx_dev, 2, lddx, w->cols);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, bytes_backward(M, w->rows, 1));
    if (st != MPQ_OK) return st;
    const int64_t ldg = grad_ld(w->rows);
    const bool vec = aligned(dy_dev, 16) && (M == 1 || lddy % 8 == 0);
    I8GradParams g{};
    g.src = dy_dev;
    g.ld = lddy;
    g.s = w->scales;
    st = vec ? grad_rows_run<0>(g, k, M, w->rows, ldg, stream) : grad_rows_run<1>(g, k, M, w->rows, ldg, stream);
    if (st != MPQ_OK) return st;
    return dx_run(&w, 1, k.grads, ldg, 0, M, dx_dev, lddx, k, stream);
}

mpq_status mpq_i8_gated_backward(const mpq_i8* x, const mpq_i8* w_gate, const mpq_i8* w_up, mpq_act act,
                                 const void* dh_dev, int64_t lddh, void* d_gate_dev, void* d_up_dev, int64_t ldd,
                                 void* dx_dev, int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
    const mpq_i8* wl[2] = {w_gate, w_up};
    mpq_status st = check_product(x, wl, 2);
    if (st != MPQ_OK) return st;
    if (!act_ok(act) || (d_gate_dev == nullptr) != (d_up_dev == nullptr)) return MPQ_ERR_ARG;
    if (x->rows == 0) return MPQ_OK;
    const int64_t F = w_gate->rows;
    const I8Ws k = ws_backward(ws, x->rows, F, x->cols, 2);
    st = check_array(dh_dev, 2, lddh, F);
    if (st == MPQ_OK && d_gate_dev) st = check_array(d_gate_dev, 2, ldd, F);
    if (st == MPQ_OK && d_up_dev) st = check_array(d_up_dev, 2, ldd, F);
    if (st == MPQ_OK) st = check_array(dx_dev, 2, lddx, x->cols);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, bytes_backward(x->rows, F, 2));
    if (st != MPQ_OK) return st;
    I8Product p{};
    p.dh = static_cast<const uint16_t*>(dh_dev);
    p.lddh = lddh;
    p.d[0] = static_cast<uint16_t*>(d_gate_dev);
    p.d[1] = static_cast<uint16_t*>(d_up_dev);
    p.ldd = ldd;
    p.g = k.grads32;
    p.up_off = grad_ld(F);
    p.ldg = 2 * p.up_off;
    st = act == MPQ_ACT_SILU ? product_run<2, MPQ_ACT_SILU>(x, wl, p, k, stream)
                             : product_run<2, MPQ_ACT_GELU_TANH>(x, wl, p, k, stream);
    if (st != MPQ_OK) return st;
    I8GradParams g{};
    g.src = k.grads32;
    g.ld = p.ldg;
    g.up_off = p.up_off;
    st = grad_rows_run<2>(g, k, x->rows, F, p.ldg, stream);
    if (st != MPQ_OK) return st;
    return dx_run(wl, 2, k.grads, p.ldg, p.up_off, x->rows, dx_dev, lddx, k, stream);
}

}  // extern "C"
