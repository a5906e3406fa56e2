// k_i8_simple.cuh -- the int8 products and their gradients as plain tiled
// kernels: 64 x 64 outputs a CTA, 4 x 4 a thread, operands staged in shared
// memory 64 bytes (or 16 rows) of the contraction at a time.
#pragma once
#include "common.cuh"
#include "i8_gate.cuh"
#include "k_i8_rows.cuh"

namespace mpq {

struct I8GemmParams {
    const int8_t* x;
    const int8_t* w[2];
    const float* xs;
    const float* ws[2];
    int64_t ldx, ldw[2];
    void* y;
    int64_t ldy;
    const uint16_t* dh;
    int64_t lddh;
    uint16_t* d[2];      // d_gate, d_up (or null)
    int64_t ldd;
    uint16_t* g;         // scaled gradients [M][ldg], up at + up_off
    int64_t ldg, up_off;
    int M, N, K, y_bf16;
};

__device__ __forceinline__ void store_out(void* y, int64_t i, float v, int bf16) {
    if (bf16) static_cast<uint16_t*>(y)[i] = (uint16_t)pack_bf16(v, 0.f);
    else static_cast<float*>(y)[i] = v;
}

// MODE 0: linear, 1: gated, 2: gated backward's gradients.
template <int MODE, int ACT>
__global__ void __launch_bounds__(256) k_i8_simple(I8GemmParams p) {
    constexpr int NW = MODE == 0 ? 1 : 2;
    __shared__ int sx[64][17], sw[NW][64][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    pdl_wait();
    pdl_launch_dependents();
    int acc[NW][4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i >> 4, c = i & 15, k = k0 + 4 * c;
            auto word = [&](const int8_t* base, int64_t ld, int64_t row, int64_t rows) {
                uint32_t v = 0;
                if (row < rows && k < p.K) {   // the pitch is a multiple of 16: the word is inside the row
                    v = *reinterpret_cast<const uint32_t*>(base + row * ld + k);
                    if (p.K - k < 4) v &= (1u << (8 * (p.K - k))) - 1u;
                }
                return (int)v;
            };
            sx[r][c] = word(p.x, p.ldx, m0 + r, p.M);
            for (int j = 0; j < NW; ++j) sw[j][r][c] = word(p.w[j], p.ldw[j], n0 + r, p.N);
        }
        __syncthreads();
        for (int c = 0; c < 16; ++c)
            for (int j = 0; j < NW; ++j)
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        acc[j][a][b] = __dp4a(sx[ty + 16 * a][c], sw[j][tx + 16 * b][c], acc[j][a][b]);
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t m = m0 + ty + 16 * a, n = n0 + tx + 16 * b;
            if (m >= p.M || n >= p.N) continue;
            const float s = p.xs[m];
            float v[NW];
            for (int j = 0; j < NW; ++j) v[j] = ((float)acc[j][a][b] * p.ws[j][n]) * s;
            if (MODE == 0) {
                store_out(p.y, m * p.ldy + n, v[0], p.y_bf16);
            } else {
                const Gate g = gate_eval<ACT>(v[0]);
                if (MODE == 1) {
                    store_out(p.y, m * p.ldy + n, g.act * v[NW - 1], p.y_bf16);
                } else {
                    const float dh = I8Elem<true>::get(p.dh[m * p.lddh + n]);
                    const float dg = dh * v[NW - 1] * g.grad, du = dh * g.act;
                    if (p.d[0]) {
                        p.d[0][m * p.ldd + n] = (uint16_t)pack_bf16(dg, 0.f);
                        p.d[1][m * p.ldd + n] = (uint16_t)pack_bf16(du, 0.f);
                    }
                    p.g[m * p.ldg + n] = (uint16_t)pack_bf16(dg * p.ws[0][n], 0.f);
                    p.g[m * p.ldg + p.up_off + n] = (uint16_t)pack_bf16(du * p.ws[NW - 1][n], 0.f);
                }
            }
        }
}

// dy * scale of its channel, rounded to bf16.
__global__ void __launch_bounds__(256) k_i8_scale_grad(const uint16_t* dy, int64_t lddy, const float* s, uint16_t* g,
                                                       int64_t ldg, int M, int N) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)M * N; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / N, n = i % N;
        g[m * ldg + n] = (uint16_t)pack_bf16(I8Elem<true>::get(dy[m * lddy + n]) * s[n], 0.f);
    }
}

struct I8DxParams {
    const uint16_t* g;
    int64_t ldg, up_off;
    const int8_t* w[2];
    int64_t ldw[2];
    uint16_t* dx;
    int64_t lddx;
    int M, N, K, nw;
};

__global__ void __launch_bounds__(256) k_i8_dx_simple(I8DxParams p) {
    __shared__ float sg[16][65], sw[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, k0 = (int64_t)blockIdx.x * 64;
    pdl_wait();
    pdl_launch_dependents();
    float acc[4][4] = {};
    for (int j = 0; j < p.nw; ++j)
        for (int n0 = 0; n0 < p.N; n0 += 16) {
            for (int i = threadIdx.x; i < 64 * 16; i += 256) {
                const int r = i >> 4, c = i & 15;
                sg[c][r] = m0 + r < p.M && n0 + c < p.N
                               ? I8Elem<true>::get(p.g[(m0 + r) * p.ldg + j * p.up_off + n0 + c]) : 0.f;
                const int r2 = i & 63, c2 = i >> 6;
                sw[c2][r2] = k0 + r2 < p.K && n0 + c2 < p.N ? (float)p.w[j][(n0 + c2) * p.ldw[j] + k0 + r2] : 0.f;
            }
            __syncthreads();
            for (int c = 0; c < 16; ++c)
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        acc[a][b] = fmaf(sg[c][ty + 16 * a], sw[c][tx + 16 * b], acc[a][b]);
            __syncthreads();
        }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t m = m0 + ty + 16 * a, k = k0 + tx + 16 * b;
            if (m < p.M && k < p.K) p.dx[m * p.lddx + k] = (uint16_t)pack_bf16(acc[a][b], 0.f);
        }
}

}  // namespace mpq
