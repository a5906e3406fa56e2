// k_i8_rows.cuh -- rows of fp32 or bf16 values to int8 codes with one scale
// a row, and back.
//
//   amax = max |x|,  s = max(fl32(amax / 127), 2^-126)  (1 for a zero row),
//   q = the integer nearest to the exact quotient x / s (ties to even).
//
// The quotient is not divided out: q0 = rint(x * fl32(1/s)) is within one of
// the answer (|x / s| <= 127 (1 + 2^-24), relative error of the product below
// 2^-22), and r = fma(-q0, s, x) is exact -- x and q0 s are multiples of a
// half of s's last place and |r| < (1/2 + 2^-14) s fits 24 of those -- so
// comparing 2 r with s settles the rounding, ties included, without a
// division per element (s / 2 would lose a bit where it is subnormal).
//
// Memory-bound: a row is read once and kept in registers between the maximum
// and the codes (rows longer than the group's registers are read again).
// G threads work on a row, so that short rows fill warps and a single long
// row (one token) still has every thread's load in flight at once.  Rows
// whose address is not 16-byte aligned (odd widths) take one element a
// thread instead of 16 bytes.
#pragma once
#include "common.cuh"

namespace mpq {

struct I8RowsParams {
    const void* x;     // quantize: in
    void* y;           // dequantize: out
    int8_t* codes;
    float* scales;
    int64_t ldx, ldc;  // elements, bytes
    int rows, cols;
};

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two floats to packed bf16, round to nearest even (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

template <bool BF16>
struct I8Elem;
template <>
struct I8Elem<true> {
    using T = uint16_t;
    static constexpr int PER = 8;   // elements in 16 bytes
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(w[i]); f[2 * i + 1] = bf16_hi(w[i]); }
    }
};
template <>
struct I8Elem<false> {
    using T = float;
    static constexpr int PER = 4;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
};

// max of |v| that keeps NaN: bit patterns of non-negative floats compare as
// integers, infinities above every number and NaN above infinity.
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, float v) {
    return max(m, __float_as_uint(v) & 0x7FFFFFFFu);
}

struct I8Scale {
    float s, inv;
    bool finite;
};
__device__ __forceinline__ I8Scale i8_scale(uint32_t amax) {
    I8Scale k;
    k.finite = amax < 0x7F800000u;
    k.s = amax == 0u ? 1.f : fmaxf(__fdiv_rn(__uint_as_float(amax), 127.f), 1.17549435e-38f);
    k.inv = __frcp_rn(k.s);
    if (!k.finite) k.s = __uint_as_float(0x7FC00000u);
    return k;
}

__device__ __forceinline__ int i8_code(float v, const I8Scale& k) {
    if (!k.finite) return 0;
    const float q0 = rintf(v * k.inv);
    const float r = fmaf(-q0, k.s, v), r2 = r + r;
    int q = (int)q0;
    // beyond half a step, or at half a step from an odd code: one further
    if (r2 > k.s || (r2 == k.s && (q & 1))) q += 1;
    else if (r2 < -k.s || (r2 == -k.s && (q & 1))) q -= 1;
    return q;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t m, uint32_t* red, int group, int t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (G > 32) {
        constexpr int W = G / 32;
        if ((t & 31) == 0) red[group * W + (t >> 5)] = m;
        __syncthreads();
        m = red[group * W];
#pragma unroll
        for (int i = 1; i < W; ++i) m = max(m, red[group * W + i]);
    }
    return m;
}

// One group of G threads a row; VPT loads a thread are kept (VEC: 16 bytes
// each, else one element).  LONG: rows beyond G * VPT loads, read twice.
template <bool BF16, bool VEC, int G, int VPT, bool LONG>
__global__ void __launch_bounds__(G > 128 ? G : 128) k_i8_quantize(I8RowsParams p) {
    using E = I8Elem<BF16>;
    using T = typename E::T;
    constexpr int THREADS = G > 128 ? G : 128;
    constexpr int PER = VEC ? E::PER : 1;
    __shared__ uint32_t red[THREADS / 32];
    const int group = threadIdx.x / G, t = threadIdx.x % G;
    const int64_t row = (int64_t)blockIdx.x * (THREADS / G) + group;
    const bool live = row < p.rows;
    const int units = p.cols / PER, tail0 = units * PER;   // whole loads, then single elements
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    int8_t* codes = p.codes + row * p.ldc;
    pdl_wait();
    pdl_launch_dependents();

    uint4 kept[VEC ? VPT : 1];
    float kept1[VEC ? 1 : VPT];
    uint32_t m = 0;
    float tail = 0.f;
    auto fold = [&](const uint4& u) {
        float f[E::PER];
        E::unpack(u, f);
#pragma unroll
        for (int j = 0; j < E::PER; ++j) m = amax_bits(m, f[j]);
    };
    if (live) {
        if (VEC) {
            if (!LONG) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    kept[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (t + i * G < units) kept[i] = reinterpret_cast<const uint4*>(x)[t + i * G];
                }
#pragma unroll
                for (int i = 0; i < VPT; ++i) fold(kept[i]);
            } else {
#pragma unroll 4
                for (int u = t; u < units; u += G) fold(reinterpret_cast<const uint4*>(x)[u]);
            }
            if (t < p.cols - tail0) {
                tail = E::get(x[tail0 + t]);
                m = amax_bits(m, tail);
            }
        } else if (!LONG) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) kept1[i] = t + i * G < units ? E::get(x[t + i * G]) : 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) m = amax_bits(m, kept1[i]);
        } else {
#pragma unroll 8
            for (int u = t; u < units; u += G) m = amax_bits(m, E::get(x[u]));
        }
    }
    m = group_max<G>(m, red, group, t);
    if (!live) return;
    const I8Scale k = i8_scale(m);
    if (t == 0) p.scales[row] = k.s;

    auto put = [&](int u, const uint4& v) {
        float f[E::PER];
        E::unpack(v, f);
        uint32_t w[E::PER / 4];
#pragma unroll
        for (int j = 0; j < E::PER / 4; ++j) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = (uint32_t)i8_code(f[4 * j + i], k);
            w[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
        if (BF16) *reinterpret_cast<uint2*>(codes + (size_t)u * 8) = make_uint2(w[0], w[E::PER / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(codes + (size_t)u * 4) = w[0];
    };
    if (VEC) {
        if (!LONG) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (t + i * G < units) put(t + i * G, kept[i]);
        } else {
#pragma unroll 2
            for (int u = t; u < units; u += G) put(u, reinterpret_cast<const uint4*>(x)[u]);
        }
        if (t < p.cols - tail0) codes[tail0 + t] = (int8_t)i8_code(tail, k);
    } else if (!LONG) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (t + i * G < units) codes[t + i * G] = (int8_t)i8_code(kept1[i], k);
    } else {
#pragma unroll 4
        for (int u = t; u < units; u += G) codes[u] = (int8_t)i8_code(E::get(x[u]), k);
    }
}

// x = code * scale.  Sixteen codes a thread (VEC: 16-byte aligned rows of x),
// or one.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) k_i8_dequantize(I8RowsParams p) {
    using T = typename I8Elem<BF16>::T;
    const int64_t row = blockIdx.x;
    const int8_t* codes = p.codes + row * p.ldc;
    T* y = static_cast<T*>(p.y) + row * p.ldx;
    pdl_wait();
    pdl_launch_dependents();
    const float s = p.scales[row];
    auto one = [&](int c) {
        const float v = (float)codes[c] * s;
        if (BF16) reinterpret_cast<uint16_t*>(y)[c] = (uint16_t)pack_bf16(v, 0.f);
        else reinterpret_cast<float*>(y)[c] = v;
    };
    const int t = blockIdx.y * 256 + threadIdx.x, step = gridDim.y * 256;
    if (!VEC) {
#pragma unroll 8
        for (int c = t; c < p.cols; c += step) one(c);
        return;
    }
    const int units = p.cols / 16;
#pragma unroll 2
    for (int u = t; u < units; u += step) {
        const uint4 q = *reinterpret_cast<const uint4*>(codes + (size_t)u * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * s;
        uint4* o = reinterpret_cast<uint4*>(y + (size_t)u * 16);
        if (BF16) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                o[i] = make_uint4(pack_bf16(f[8 * i], f[8 * i + 1]), pack_bf16(f[8 * i + 2], f[8 * i + 3]),
                                  pack_bf16(f[8 * i + 4], f[8 * i + 5]), pack_bf16(f[8 * i + 6], f[8 * i + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                  __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
        }
    }
    for (int c = units * 16 + t; c < p.cols; c += step) one(c);
}

}  // namespace mpq
