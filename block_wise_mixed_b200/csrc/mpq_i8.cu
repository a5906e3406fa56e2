// mpq_i8.cu -- the C ABI of the 8-bit integer operators (include/mpq.h):
// argument checks, workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mpq.h"
#include "common.cuh"
#include "i8_gate.cuh"
#include "k_i8_rows.cuh"
#include "k_i8_simple.cuh"

using namespace mpq;

namespace {

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

mpq_status check_i8(const mpq_i8* q) {
    if (!q) return MPQ_ERR_ARG;
    if (q->rows < 0 || q->cols < 1 || q->cols > MPQ_I8_MAX_COLS) return MPQ_ERR_SHAPE;
    if (q->ld < q->cols || q->ld % 16 != 0) return MPQ_ERR_ARG;
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
mpq_status launch(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, void* stream, Args&&... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = static_cast<cudaStream_t>(stream);
    c.attrs = pdl;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, std::forward<Args>(args)...) == cudaSuccess ? MPQ_OK : MPQ_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
template <bool BF16, bool VEC>
mpq_status quantize_launch(const I8RowsParams& p, void* stream) {
    constexpr int PER = VEC ? I8Elem<BF16>::PER : 1;
    constexpr int VPT = VEC ? 8 : 32;   // loads kept by a thread (32 registers)
    const int64_t units = p.cols / PER;
    // a few rows: as many threads a row as have a load to make
    const bool few = p.rows <= 148;
    if (units > 512 * VPT) return launch(k_i8_quantize<BF16, VEC, 512, VPT, true>, dim3(p.rows), 512, 0, stream, p);
    if (units > 128 * VPT || (few && units > 128))
        return launch(k_i8_quantize<BF16, VEC, 512, VPT, false>, dim3(p.rows), 512, 0, stream, p);
    if (units > 32 * VPT || (few && units > 32))
        return launch(k_i8_quantize<BF16, VEC, 128, VPT, false>, dim3(p.rows), 128, 0, stream, p);
    return launch(k_i8_quantize<BF16, VEC, 32, VPT, false>, dim3((unsigned)div_up(p.rows, 4)), 128, 0, stream, p);
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
    const bool vec = aligned(x_dev, 16) && (out->rows == 1 || ldx * (int64_t)es % 16 == 0);
    if (dt == MPQ_Y_BF16) return vec ? quantize_launch<true, true>(p, stream) : quantize_launch<true, false>(p, stream);
    return vec ? quantize_launch<false, true>(p, stream) : quantize_launch<false, false>(p, stream);
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
    const int64_t per = 256 * (vec ? 16 * 2 : 8);
    const dim3 grid((unsigned)q->rows, (unsigned)div_up(q->cols, q->rows <= 148 ? per / (vec ? 2 : 8) : per));
    if (dt == MPQ_Y_BF16) return vec ? launch(k_i8_dequantize<true, true>, grid, 256, 0, stream, p)
                                     : launch(k_i8_dequantize<true, false>, grid, 256, 0, stream, p);
    return vec ? launch(k_i8_dequantize<false, true>, grid, 256, 0, stream, p)
               : launch(k_i8_dequantize<false, false>, grid, 256, 0, stream, p);
}

}  // extern "C"

namespace {

// Workspace: the error word, the counters (zero between calls), then scratch
// that a call writes before it reads.  The zeroed part has one size for all
// mpq_i8_* calls, so one workspace serves them all, one after another.
constexpr size_t kI8ZeroBytes = 256;

inline bool shape_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 1 && K >= 1 && K <= MPQ_I8_MAX_COLS;
}

inline int64_t grad_ld(int64_t n) { return div_up(n, 64) * 64; }

inline size_t i8_ws_bytes(int64_t M, int64_t N, int64_t K, int grads) {
    if (!shape_ok(M, N, K)) return 0;
    return round256(kI8ZeroBytes + (size_t)M * (size_t)grad_ld(N) * 2 * (size_t)grads);
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

I8GemmParams gemm_params(const mpq_i8* x, const mpq_i8* const* w, int nw) {
    I8GemmParams p{};
    p.x = x->codes;
    p.xs = x->scales;
    p.ldx = x->ld;
    for (int i = 0; i < nw; ++i) {
        p.w[i] = w[i]->codes;
        p.ws[i] = w[i]->scales;
        p.ldw[i] = w[i]->ld;
    }
    p.M = x->rows;
    p.N = w[0]->rows;
    p.K = x->cols;
    return p;
}

template <int MODE>
mpq_status gemm_run(const I8GemmParams& p, mpq_act act, void* stream) {
    const dim3 grid((unsigned)div_up(p.N, 64), (unsigned)div_up(p.M, 64));
    if (grid.y > 65535) return MPQ_ERR_SHAPE;
    return act == MPQ_ACT_SILU ? launch(k_i8_simple<MODE, MPQ_ACT_SILU>, grid, 256, 0, stream, p)
                               : launch(k_i8_simple<MODE, MPQ_ACT_GELU_TANH>, grid, 256, 0, stream, p);
}

mpq_status dx_run(const I8DxParams& p, void* stream) {
    const dim3 grid((unsigned)div_up(p.K, 64), (unsigned)div_up(p.M, 64));
    if (grid.y > 65535) return MPQ_ERR_SHAPE;
    return launch(k_i8_dx_simple, grid, 256, 0, stream, p);
}

}  // namespace

extern "C" {

size_t mpq_i8_linear_workspace_size(int32_t M, int32_t N, int32_t K) { return i8_ws_bytes(M, N, K, 0); }
size_t mpq_i8_gated_workspace_size(int32_t M, int32_t F, int32_t K) { return i8_ws_bytes(M, F, K, 0); }
size_t mpq_i8_linear_backward_workspace_size(int32_t M, int32_t N, int32_t K) { return i8_ws_bytes(M, N, K, 1); }
size_t mpq_i8_gated_backward_workspace_size(int32_t M, int32_t F, int32_t K) { return i8_ws_bytes(M, F, K, 2); }

mpq_status mpq_i8_linear(const mpq_i8* x, const mpq_i8* w, void* y_dev, mpq_ydtype ydt, int64_t ldy, void* ws,
                         size_t ws_bytes, void* stream) {
    const mpq_i8* wl[1] = {w};
    mpq_status st = check_product(x, wl, 1);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(ydt)) return MPQ_ERR_ARG;
    if (x->rows == 0) return MPQ_OK;
    st = check_array(y_dev, elem_size(ydt), ldy, w->rows);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, mpq_i8_linear_workspace_size(x->rows, w->rows, x->cols));
    if (st != MPQ_OK) return st;
    I8GemmParams p = gemm_params(x, wl, 1);
    p.y = y_dev;
    p.ldy = ldy;
    p.y_bf16 = ydt == MPQ_Y_BF16;
    return gemm_run<0>(p, MPQ_ACT_SILU, stream);
}

mpq_status mpq_i8_gated(const mpq_i8* x, const mpq_i8* w_gate, const mpq_i8* w_up, mpq_act act, void* h_dev,
                        mpq_ydtype ydt, int64_t ldh, void* ws, size_t ws_bytes, void* stream) {
    const mpq_i8* wl[2] = {w_gate, w_up};
    mpq_status st = check_product(x, wl, 2);
    if (st != MPQ_OK) return st;
    if (!dtype_ok(ydt) || !act_ok(act)) return MPQ_ERR_ARG;
    if (x->rows == 0) return MPQ_OK;
    st = check_array(h_dev, elem_size(ydt), ldh, w_gate->rows);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, mpq_i8_gated_workspace_size(x->rows, w_gate->rows, x->cols));
    if (st != MPQ_OK) return st;
    I8GemmParams p = gemm_params(x, wl, 2);
    p.y = h_dev;
    p.ldy = ldh;
    p.y_bf16 = ydt == MPQ_Y_BF16;
    return gemm_run<1>(p, act, stream);
}

mpq_status mpq_i8_linear_backward(const mpq_i8* w, const void* dy_dev, int32_t M, int64_t lddy, void* dx_dev,
                                  int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
    mpq_status st = check_i8(w);
    if (st != MPQ_OK) return st;
    if (M < 0 || w->rows < 1) return MPQ_ERR_SHAPE;
    if (M == 0) return MPQ_OK;
    st = check_array(dy_dev, 2, lddy, w->rows);
    if (st == MPQ_OK) st = check_array(dx_dev, 2, lddx, w->cols);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, mpq_i8_linear_backward_workspace_size(M, w->rows, w->cols));
    if (st != MPQ_OK) return st;
    uint16_t* g = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kI8ZeroBytes);
    const int64_t ldg = grad_ld(w->rows);
    const unsigned blocks = (unsigned)std::min<int64_t>(div_up((int64_t)M * w->rows, 256), 148 * 8);
    st = launch(k_i8_scale_grad, dim3(blocks), 256, 0, stream, static_cast<const uint16_t*>(dy_dev), lddy, w->scales,
                g, ldg, M, w->rows);
    if (st != MPQ_OK) return st;
    I8DxParams d{};
    d.g = g;
    d.ldg = ldg;
    d.w[0] = w->codes;
    d.ldw[0] = w->ld;
    d.dx = static_cast<uint16_t*>(dx_dev);
    d.lddx = lddx;
    d.M = M;
    d.N = w->rows;
    d.K = w->cols;
    d.nw = 1;
    return dx_run(d, stream);
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
    st = check_array(dh_dev, 2, lddh, F);
    if (st == MPQ_OK && d_gate_dev) st = check_array(d_gate_dev, 2, ldd, F);
    if (st == MPQ_OK && d_up_dev) st = check_array(d_up_dev, 2, ldd, F);
    if (st == MPQ_OK) st = check_array(dx_dev, 2, lddx, x->cols);
    if (st == MPQ_OK) st = check_ws(ws, ws_bytes, mpq_i8_gated_backward_workspace_size(x->rows, (int32_t)F, x->cols));
    if (st != MPQ_OK) return st;
    I8GemmParams p = gemm_params(x, wl, 2);
    p.dh = static_cast<const uint16_t*>(dh_dev);
    p.lddh = lddh;
    p.d[0] = static_cast<uint16_t*>(d_gate_dev);
    p.d[1] = static_cast<uint16_t*>(d_up_dev);
    p.ldd = ldd;
    p.g = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kI8ZeroBytes);
    p.up_off = grad_ld(F);
    p.ldg = 2 * p.up_off;
    st = gemm_run<2>(p, act, stream);
    if (st != MPQ_OK) return st;
    I8DxParams d{};
    d.g = p.g;
    d.ldg = p.ldg;
    d.up_off = p.up_off;
    d.w[0] = w_gate->codes;
    d.w[1] = w_up->codes;
    d.ldw[0] = w_gate->ld;
    d.ldw[1] = w_up->ld;
    d.dx = static_cast<uint16_t*>(dx_dev);
    d.lddx = lddx;
    d.M = x->rows;
    d.N = (int)F;
    d.K = x->cols;
    d.nw = 2;
    return dx_run(d, stream);
}

}  // extern "C"
