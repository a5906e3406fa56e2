// k_i8_rows.cuh -- rows of fp32 or bf16 values to int8 codes with one scale
// a row, and back.
//
//   amax = max |x|,  s = max(fl32(amax / 127), 2^-126)  (1 for a zero row),
//   q = the integer nearest to the exact quotient x / s (ties to even).
//
// The quotient is not divided out.  With M = 1.5 * 2^23 and inv = 1/s to 1 ulp,
//   t = fma(x, inv, M)              M + q0, q0 within one of the answer
//   r = fma(M - t, s, x)            x - q0 s, exact: both are multiples of half
//                                   of s's last place, |r| < (1/2 + 2^-14) s
//   d = 2 |r| - s                   exact near 0, a multiple of s's last place
//   e = fma(d, 0.75 inv, 0.5)       below, at, or above 1/2 as |r| is below,
//                                   at, or above s / 2 (|d| > 2^-24 s if not 0,
//                                   and 0.75 * 2^-24 does not round to 1/2)
//   t = t + copysign(e, r)          rounds the way the exact quotient does, ties
//                                   to even; |e| < 1/2 changes nothing
// and the code is the low byte of t.  Exact ties are common for bf16 (one
// element in 200: both values have 8 bits), so they are not left to a branch:
// a branch for the rare elements was taken by most warps and cost 28672 x
// 8192 bf16 160 us where this costs 120.
//
// Memory-bound: a row is read once and kept in registers between the maximum
// and the codes (rows longer than the group's registers are read again).
// G threads work on a row, so that short rows fill warps and a single long
// row (one token) still has every thread's load in flight at once.
// Loads are 16 bytes at any alignment: a row that starts or ends inside a
// 16-byte block (odd widths) is read in the blocks that cover it, and the codes
// are shifted into place with the next lane's (SHIFT; a warp then advances by
// 31 blocks, its last lane only serving its neighbour).
//
// Measured: 2048 x 14336 fp32 25 us (5.8 TB/s), 2047 x 14335 32 us (4.6 TB/s);
// 28672 x 8192 bf16 120 us (5.9 TB/s); back 25, 27 and 105 us (5.5-6.7 TB/s).
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
    static __device__ __forceinline__ uint4 guarded(const uint16_t* x, int lo, int hi) {   // elements [lo, hi) of a block
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= lo && j < hi) w[j >> 1] |= (uint32_t)x[j] << (16 * (j & 1));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
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
    static __device__ __forceinline__ uint4 guarded(const float* x, int lo, int hi) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j >= lo && j < hi) w[j] = __float_as_uint(x[j]);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
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
    float s, inv, inv75;   // scale, 1 / s and 0.75 / s
    bool finite;
};
__device__ __forceinline__ I8Scale i8_scale(uint32_t amax) {
    I8Scale k;
    k.finite = amax < 0x7F800000u;
    k.s = amax == 0u ? 1.f : fmaxf(__fdiv_rn(__uint_as_float(amax), 127.f), 1.17549435e-38f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(k.inv) : "f"(k.s));   // 1 ulp; s and 1/s are normal numbers
    k.inv75 = 0.75f * k.inv;
    if (!k.finite) k.s = __uint_as_float(0x7FC00000u);
    return k;
}

// The code of one element in the low byte (of a finite row).
__device__ __forceinline__ uint32_t i8_code(float x, const I8Scale& k) {
    constexpr float kMagic = 12582912.f;   // 1.5 * 2^23
    const float t = fmaf(x, k.inv, kMagic);
    const float r = fmaf(kMagic - t, k.s, x);
    const float d = (fabsf(r) + fabsf(r)) - k.s;
    return __float_as_uint(t + copysignf(fmaf(d, k.inv75, 0.5f), r));
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The maximum over the G threads of a row; red: a 16-byte aligned word a warp.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t m, uint32_t* red, int t) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (G > 32) {
        if ((t & 31) == 0) red[t >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < G / 128; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(red)[i];
            m = max(m, max(max(v.x, v.y), max(v.z, v.w)));
        }
    }
    return m;
}

// A row as the 16-byte blocks that cover it: elements off .. end - 1 of the
// array at x.  Without SHIFT rows are whole blocks; with it the first and the
// last block may hold elements of the gap or the rows beside, which `mask`
// takes out (before the array's start and behind its end nothing is read).
template <bool BF16, bool SHIFT>
struct I8Row {
    using E = I8Elem<BF16>;
    using T = typename E::T;
    const T* x;
    int off, end, blocks;
    bool edge0, edge1;   // the first block starts before the array, the last one ends behind it
    __device__ __forceinline__ I8Row(const I8RowsParams& p, int64_t row) {
        x = static_cast<const T*>(p.x) + row * p.ldx;
        off = SHIFT ? (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)) : 0;
        x -= off;
        end = off + p.cols;
        blocks = row < p.rows ? (end + E::PER - 1) / E::PER : 0;
        // (of few columns, several rows lie in the array's first or last block)
        edge0 = SHIFT && row * p.ldx < off;
        edge1 = SHIFT && (p.rows - 1 - row) * p.ldx + end < (int64_t)blocks * E::PER;
    }
    __device__ __forceinline__ uint4 load(int b) const {
        if (b >= blocks) return make_uint4(0u, 0u, 0u, 0u);
        if ((edge0 && b == 0) || (edge1 && b == blocks - 1))
            return E::guarded(x + (size_t)b * E::PER, b == 0 ? off : 0, min(E::PER, end - b * E::PER));
        return *reinterpret_cast<const uint4*>(x + (size_t)b * E::PER);
    }
    __device__ __forceinline__ void mask(int b, uint4& v) const {
        if (!SHIFT) return;
        const int lo = b == 0 ? off : 0, hi = end - b * E::PER;
        if (lo == 0 && hi >= E::PER) return;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < E::PER; ++j)
            if (j < lo || j >= hi) w[j * (int)sizeof(T) / 4] &= BF16 ? (j & 1 ? 0x0000FFFFu : 0xFFFF0000u) : 0u;
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// One group of G threads a row, VPT 16-byte blocks kept by a thread.  LONG:
// rows of more blocks, read twice.  The grid is what is resident, and a group
// asks for its next row before it works on the one that has arrived (a block
// a row instead spent a third of its time starting and waiting).
template <bool BF16, bool SHIFT, int G, int VPT, bool LONG>
__global__ void __launch_bounds__(G > 128 ? G : 128) k_i8_quantize(I8RowsParams p) {
    using E = I8Elem<BF16>;
    using Row = I8Row<BF16, SHIFT>;
    constexpr int THREADS = G > 128 ? G : 128, PER = E::PER, GROUPS = THREADS / G, K = LONG ? 1 : VPT;
    constexpr int STEP = SHIFT ? G / 32 * 31 : G;              // blocks of a round
    __shared__ __align__(16) uint32_t red[2][THREADS / 32];
    const int t = threadIdx.x % G, lane = threadIdx.x & 31;
    const int first = SHIFT ? t / 32 * 31 + lane : t;          // this thread's block of the first round
    const int64_t row0 = (int64_t)blockIdx.x * GROUPS + threadIdx.x / G, step = (int64_t)gridDim.x * GROUPS;
    pdl_wait();
    pdl_launch_dependents();

    auto load_row = [&](const Row& r, uint4 (&v)[K]) {
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = r.load(first + i * STEP);
    };
    uint4 next[K];
    if (!LONG) load_row(Row(p, row0), next);
    int round = 0;
    for (int64_t row = row0; row < p.rows; row += step, round ^= 1) {
        const Row r(p, row);
        uint32_t m = 0, m2 = 0;   // m2: two bf16 magnitudes
        auto fold = [&](const uint4& u) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (BF16) m2 = __vmaxu2(m2, w[j] & 0x7FFF7FFFu);
                else m = max(m, w[j] & 0x7FFFFFFFu);
            }
        };
        uint4 kept[K];
        if (!LONG) {
#pragma unroll
            for (int i = 0; i < K; ++i) kept[i] = next[i];
            if (row + step < p.rows) load_row(Row(p, row + step), next);
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int b = first + i * STEP;
                if (SHIFT && (i == 0 || b >= r.blocks - 1)) r.mask(b, kept[i]);
                fold(kept[i]);
            }
        } else {
#pragma unroll 4
            for (int b = first; b < r.blocks; b += STEP) {
                uint4 v = r.load(b);
                r.mask(b, v);
                fold(v);
            }
        }
        if (BF16) m = max(m, max(m2 << 16, m2 & 0xFFFF0000u));
        m = group_max<G>(m, red[round], t);
        const I8Scale k = i8_scale(m);
        if (t == 0) p.scales[row] = k.s;

        int8_t* codes = p.codes + row * p.ldc;
        const uint32_t finite = k.finite ? 0xFFFFFFFFu : 0u;
        uint32_t part[2] = {0u, 0u};   // codes of a partial block of columns
        int part_col = -1;
        auto put = [&](int b, const uint4& v) {
            float f[PER];
            E::unpack(v, f);
            uint32_t c[PER], w[2];
    #pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = i8_code(f[i], k);
            w[0] = pack_bytes(c[0], c[1], c[2], c[3]) & finite;
            w[1] = BF16 ? pack_bytes(c[PER - 4], c[PER - 3], c[PER - 2], c[PER - 1]) & finite : 0u;
            if (SHIFT) {   // columns PER b ..: this block's codes from `off` on, then the next block's first
                const uint32_t n0 = __shfl_down_sync(0xffffffffu, w[0], 1);
                if (BF16) {
                    const uint32_t n1 = __shfl_down_sync(0xffffffffu, w[1], 1);
                    const uint32_t q[4] = {w[0], w[1], n0, n1};
                    const bool far = r.off >= 4;
                    const uint32_t q0 = far ? q[1] : q[0], q1 = far ? q[2] : q[1], q2 = far ? q[3] : q[2];
                    w[0] = __funnelshift_r(q0, q1, 8 * (r.off & 3));
                    w[1] = __funnelshift_r(q1, q2, 8 * (r.off & 3));
                } else {
                    w[0] = __funnelshift_r(w[0], n0, 8 * r.off);
                }
            }
            const int col = b * PER, left = p.cols - col;
            if (left <= 0 || (SHIFT && lane == 31)) return;
            if (left >= PER) {
                if (BF16) *reinterpret_cast<uint2*>(codes + col) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t*>(codes + col) = w[0];
            } else {
                part[0] = w[0];
                part[1] = w[1];
                part_col = col;
            }
        };
        if (!LONG) {
#pragma unroll
            for (int i = 0; i < K; ++i) put(first + i * STEP, kept[i]);
        } else {   // whole warps go round together (the shuffles)
#pragma unroll 2
            for (int b = first; b - lane < r.blocks; b += STEP) put(b, r.load(b));
        }
        if (part_col >= 0) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (part_col + j < p.cols) codes[part_col + j] = (int8_t)(part[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// Word w (codes 4 w .. 4 w + 3) of a row of `cols` codes; bytes behind the last
// column read as zero and are not touched.
__host__ __device__ __forceinline__ uint32_t i8_codes_word(const int8_t* codes, int w, int cols) {
    const int left = cols - 4 * w;
    if (left >= 4) return reinterpret_cast<const uint32_t*>(codes)[w];
    uint32_t v = 0u;
    for (int j = 0; j < left; ++j) v |= (uint32_t)(uint8_t)codes[4 * w + j] << (8 * j);
    return v;
}

// x = code * scale.  VEC (16-byte aligned rows of x): 16 bytes of x a thread,
// four times.  Otherwise a warp takes 128 codes as 32 words and deals them
// out, so that lane l stores elements 32 j + l: whole lines at any alignment,
// and eight words a lane in flight.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) k_i8_dequantize(I8RowsParams p) {
    using T = typename I8Elem<BF16>::T;
    const int64_t row = blockIdx.x;
    const int8_t* codes = p.codes + row * p.ldc;
    T* y = static_cast<T*>(p.y) + row * p.ldx;
    pdl_wait();
    pdl_launch_dependents();
    const float s = p.scales[row];
    auto store = [&](int c, int q) {
        const float v = (float)q * s;
        if (BF16) reinterpret_cast<uint16_t*>(y)[c] = (uint16_t)pack_bf16(v, 0.f);
        else reinterpret_cast<float*>(y)[c] = v;
    };
    if (!VEC) {
        const int lane = threadIdx.x & 31, words = (p.cols + 3) / 4;
        const int per = 8 * 32;   // words of a warp's piece
        for (int w0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * per; w0 < words; w0 += gridDim.y * 8 * per) {
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = i8_codes_word(codes, w0 + 32 * i + lane, p.cols);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t word = __shfl_sync(0xffffffffu, r[i], 8 * j + (lane >> 2));
                    const int c = 4 * (w0 + 32 * i) + 32 * j + lane;
                    if (c < p.cols) store(c, (int8_t)(word >> (8 * (lane & 3))));
                }
        }
        return;
    }
    constexpr int PER = I8Elem<BF16>::PER;
    const int units = p.cols / PER, step = gridDim.y * 256 * 4;
    for (int u0 = blockIdx.y * 256 * 4 + threadIdx.x; u0 < units; u0 += step) {
        uint32_t w[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = u0 + i * 256;
            w[i][0] = w[i][1] = 0u;
            if (u < units) {
                if (BF16) {
                    const uint2 q = *reinterpret_cast<const uint2*>(codes + (size_t)u * 8);
                    w[i][0] = q.x;
                    w[i][1] = q.y;
                } else {
                    w[i][0] = *reinterpret_cast<const uint32_t*>(codes + (size_t)u * 4);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = u0 + i * 256;
            if (u >= units) break;
            float f[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) f[j] = (float)(int8_t)(w[i][j >> 2] >> (8 * (j & 3))) * s;
            *reinterpret_cast<uint4*>(y + (size_t)u * PER) =
                BF16 ? make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[PER - 4], f[PER - 3]),
                                  pack_bf16(f[PER - 2], f[PER - 1]))
                     : make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                  __float_as_uint(f[3]));
        }
    }
    if (blockIdx.y == 0 && threadIdx.x < p.cols - units * PER)
        store(units * PER + threadIdx.x, codes[units * PER + threadIdx.x]);
}

}  // namespace mpq
