// layer_mat.h -- 16 x 16 matrix-core tiles of the scan over heads.
//
// Operand layout of a product with 32 values of k (a wavefront of 4 groups g
// of 16 lanes l): lane (g, l) holds 8 values of k of row (or column) l.  Which
// 8 does not matter as long as both operands agree, and three orders occur:
//   row       k = 8g .. 8g+7                     (16 neighbouring bytes)
//   row_perm  k = 4g .. 4g+3, 16+4g .. 16+4g+3   (two pieces of 8 bytes)
//   col_perm  the same k, read down a column of a matrix stored by rows of k
// A result tile has rows 4g .. 4g+3 of column l in lane (g, l): two result
// tiles one above the other are an operand in the permuted order, with no
// data moved between lanes.
#pragma once

#include "layer_common.h"

namespace ssm {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

template <class IO>
struct Mat;

template <>
struct Mat<BF16> {
    using E = uint16_t;
    using Frag = bf8;
    static constexpr int kTerms = 3;    // bf16 values that hold a float32: 3 x 8 bits
    static constexpr int kPad = 8;      // elements behind a row in LDS: 16 bytes
    union Bits { Frag f; uint32_t u[4]; uint2 d[2]; uint4 q; s4v s[2]; };
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ Frag row(const E *p, int g) {
        Bits b;
        b.q = *reinterpret_cast<const uint4 *>(p + 8 * g);
        return b.f;
    }
    static __device__ __forceinline__ Frag row_perm(const E *p, int g) {
        Bits b;
        b.d[0] = *reinterpret_cast<const uint2 *>(p + 4 * g);
        b.d[1] = *reinterpret_cast<const uint2 *>(p + 16 + 4 * g);
        return b.f;
    }
    // m: row k = 0, column 0 of the tile; LDS transposes 4 x 16 values a group
    static __device__ __forceinline__ Frag col_perm(const E *m, int stride, int g, int l) {
        using L3 = __attribute__((address_space(3))) s4v;
        const E *p = m + (4 * g + (l >> 2)) * stride + 4 * (l & 3);
        Bits b;
        b.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L3 *)(p));
        b.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L3 *)(p + 16 * stride));
        return b.f;
    }
    static __device__ __forceinline__ Frag pack(const float (&v)[8]) {
        Bits b;
        b.q = Seg<BF16>::pack(v);
        return b.f;
    }
    static __device__ __forceinline__ void unpack(Frag f, float (&v)[8]) {
        Bits b;
        b.f = f;
        Seg<BF16>::unpack(b.q, v);
    }
    // v becomes what packing it left out
    static __device__ __forceinline__ Frag take(float (&v)[8]) {
        const Frag f = pack(v);
        float r[8];
        unpack(f, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] -= r[i];
        return f;
    }
};

template <>
struct Mat<F32> {
    using E = float;
    typedef float Frag __attribute__((ext_vector_type(8)));
    static constexpr int kTerms = 1;
    static constexpr int kPad = 4;
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag two(const E *p, const E *q) {
        const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(q);
        return Frag{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    static __device__ __forceinline__ Frag row(const E *p, int g) { return two(p + 8 * g, p + 8 * g + 4); }
    static __device__ __forceinline__ Frag row_perm(const E *p, int g) { return two(p + 4 * g, p + 16 + 4 * g); }
    static __device__ __forceinline__ Frag col_perm(const E *m, int stride, int g, int l) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = m[(4 * g + (j & 3) + 16 * (j >> 2)) * stride + l];
        return f;
    }
    static __device__ __forceinline__ Frag pack(const float (&v)[8]) {
        return Frag{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    }
    static __device__ __forceinline__ void unpack(Frag f, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
    static __device__ __forceinline__ Frag take(float (&v)[8]) { return pack(v); }
};

// ----------------------------------------------------------- chunks of tokens
struct Chunk {
    int64_t b, t;       // batch row, first token
    int n;              // tokens, 0: none
    int64_t row;        // sequence (row of the states)
    bool first, last;
};

// Chunk c (0 .. nc - 1) of batch row b.
__device__ __forceinline__ Chunk chunk_at(const HeadsArgs &a, int64_t b, int64_t c) {
    Chunk k;
    k.b = b;
    if (a.cu) {
        const HeadsEntry e = a.table[c];
        k.t = e.t; k.n = e.n; k.row = e.row;
        k.first = e.flags & kFirst; k.last = e.flags & kLast;
    } else {
        k.t = c * a.Q;
        const int64_t left = a.L - k.t;
        k.n = static_cast<int>(left < a.Q ? left : a.Q);
        k.row = b;
        k.first = c == 0;
        k.last = c == a.nc - 1;
    }
    return k;
}

// Rows of a chunk into LDS: dst[t][c] = src[t * stride + c] for t < n, c < cols,
// zeros up to Q rows and `width` columns.  vec: 16-byte pieces.
template <class IO, int Q>
__device__ __forceinline__ void stage_rows(typename IO::T *dst, int ld, const typename IO::T *src,
                                           int64_t stride, int n, int cols, int width, bool vec) {
    using T = typename IO::T;
    constexpr int V = Seg<IO>::VW;
    using Vec = typename Seg<IO>::V;
    if (vec) {
        const int per = width / V;
        for (int i = threadIdx.x; i < Q * per; i += blockDim.x) {
            const int t = i / per, c = (i % per) * V;
            Vec v{};
            if (t < n && c < cols) v = *reinterpret_cast<const Vec *>(src + t * stride + c);
            *reinterpret_cast<Vec *>(dst + t * ld + c) = v;
        }
    } else {
        for (int i = threadIdx.x; i < Q * width; i += blockDim.x) {
            const int t = i / width, c = i % width;
            dst[t * ld + c] = t < n && c < cols ? src[t * stride + c] : T(0);
        }
    }
}

// The step size of one token of one head (0 behind the chunk's end).
template <class IO>
__device__ __forceinline__ float step_size(const HeadsArgs &a, const Chunk &k, int t, int64_t h) {
    if (t >= k.n) return 0.0f;
    float v = IO::load(static_cast<const typename IO::T *>(a.delta) + k.b * a.dt_b + (k.t + t) * a.dt_t, h);
    if (a.bias) v += a.bias[h];
    // once a token and head: log1pf and expf, whose errors do not add up in dA
    return a.softplus ? fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))) : v;
}

// Inclusive sum over the lanes of a wavefront, in 64 bits: differences of
// these sums are the exponents, and in 32 bits the chunk's later ones would
// lose 1e-6 of the decay.
__device__ __forceinline__ double lane_prefix(double v) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double w = __shfl_up(v, o, 64);
        if (l >= o) v += w;
    }
    return v;
}

// 2^x of an exponent in 64 bits: what its rounding to float leaves out comes
// back as a factor 1 + lo ln 2.
__device__ __forceinline__ float exp2_d(double x) {
    const float hi = static_cast<float>(x), lo = static_cast<float>(x - hi);
    const float e = exp2_hw(hi);
    return __builtin_fmaf(e * kLn2, lo, e);
}

// Host: whether rows of `src` can be read in 16-byte pieces.
template <class IO>
__host__ __device__ inline bool vec_rows(const void *src, int64_t b, int64_t t, int64_t piece) {
    constexpr int V = Seg<IO>::VW;
    return reinterpret_cast<uintptr_t>(src) % 16 == 0 && b % V == 0 && t % V == 0 && piece % V == 0;
}

}  // namespace ssm
