// layer_mat.h -- 16 x 16 matrix-core tiles of the scan over heads.
//
// Operand layout of a product with 32 values of k (a wavefront of 4 groups g
// of 16 lanes l): lane (g, l) holds 8 values of k of row (or column) l.  Which
// 8 does not matter as long as both operands agree; here k = 4g .. 4g+3 and
// 16+4g .. 16+4g+3 (the permuted order), read along a row (row_perm) or down a
// column of a matrix stored by rows of k (col_perm).  16-bit rows are kept in
// the permuted order in LDS (pos): one read of 16 bytes instead of two of 8,
// which run at half the rate at every distance of the rows (measured: 31 .. 37
// against 66 cycles for the four wavefronts' 4 KB).
// A result tile has rows 4g .. 4g+3 of column l in lane (g, l): two result
// tiles one above the other are an operand in the permuted order, with no
// data moved between lanes.
#pragma once

#include "layer_common.h"

namespace ssm {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void store16(f4 v, Rsrc to, uint32_t off, int more) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), to, off, more, 0);
}

// The kernel's arguments read again: what a loop needs rarely, or only the end
// does, takes no scalar registers (or lanes of a vector one) until then.  The
// arguments are the kernel's first.
typedef const __attribute__((address_space(4))) HeadsArgs *ArgsAgain;
__device__ __forceinline__ ArgsAgain args_again() {
    ArgsAgain p = (ArgsAgain)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// A number known while compiling, for lambdas.
template <int I>
struct Int { static constexpr int value = I; };

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
    // where column c of a row kept in the permuted order lies; whole tiles of
    // 16 columns: the tile's first value is at pos, the next fours at pos + 8
    static __device__ __forceinline__ constexpr int pos(int c) {
        return (c & ~31) + (c >> 2 & 3) * 8 + (c >> 4 & 1) * 4 + (c & 3);
    }
    static __device__ __forceinline__ Frag row_perm(const E *p, int g) {
        Bits b;
        b.q = *reinterpret_cast<const uint4 *>(p + 8 * g);
        return b.f;
    }
    // columns c .. c + 7 (c a multiple of 8) into a row kept in that order
    template <class Vec>
    static __device__ __forceinline__ void put_perm(E *row, int c, const Vec &v) {
        uint2 h[2];
        __builtin_memcpy(h, &v, 16);
        *reinterpret_cast<uint2 *>(row + pos(c)) = h[0];
        *reinterpret_cast<uint2 *>(row + pos(c + 4)) = h[1];
    }
    template <class Vec>
    static __device__ __forceinline__ Vec get_perm(const E *row, int c) {
        const uint2 h[2] = {*reinterpret_cast<const uint2 *>(row + pos(c)),
                            *reinterpret_cast<const uint2 *>(row + pos(c + 4))};
        Vec v;
        __builtin_memcpy(&v, h, 16);
        return v;
    }
    // m: row k = 0 and column 0 of the tile; LDS transposes 4 x 16 values a
    // group.  FOUR: distance of the tile's fours of columns, 8 in rows kept
    // in the permuted order.
    template <int FOUR = 4>
    static __device__ __forceinline__ Frag col_perm(const E *m, int stride, int g, int l) {
        using L3 = __attribute__((address_space(3))) s4v;
        const E *p = m + (4 * g + (l >> 2)) * stride + FOUR * (l & 3);
        Bits b;
        b.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L3 *)(p));
        b.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L3 *)(p + 16 * stride));
        return b.f;
    }
    static __device__ __forceinline__ f4 fours(const E *p) {
        const uint2 d = *reinterpret_cast<const uint2 *>(p);
        return f4{__uint_as_float(d.x << 16), __uint_as_float(d.x & 0xffff0000u),
                  __uint_as_float(d.y << 16), __uint_as_float(d.y & 0xffff0000u)};
    }
    static __device__ __forceinline__ Frag pack(const float (&v)[8]) {
        Bits b;
        b.q = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        return b.f;
    }
    static __device__ __forceinline__ void unpack(Frag f, float (&v)[8]) {
        Bits b;
        b.f = f;
        Seg<BF16>::unpack(b.q, v);
    }
    // half an operand (one result tile) in LDS: 8 bytes a lane
    using Half = uint2;
    static __device__ __forceinline__ Half half(f4 v) {
        return make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
    }
    static __device__ __forceinline__ void store(Half h, Rsrc to, uint32_t off, int more) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(u2{h.x, h.y}, to, off, more, 0);
    }
    static __device__ __forceinline__ Half none() { return make_uint2(0, 0); }
    // What the rounding of v to h left of the float32 bits, in 16 bits: with h
    // all of v again.  (A tie rounded down leaves 0x8000, one too many: 2^-24.)
    static __device__ __forceinline__ Half rest(f4 v, Half h) {
        auto two = [](float a, float b, uint32_t h2) {
            const int x = min(static_cast<int>(__float_as_uint(a) - (h2 << 16)), 0x7fff);
            const int y = min(static_cast<int>(__float_as_uint(b) - (h2 & 0xffff0000u)), 0x7fff);
            return __builtin_amdgcn_perm(static_cast<uint32_t>(y), static_cast<uint32_t>(x), 0x05040100);
        };
        return make_uint2(two(v.x, v.y, h.x), two(v.z, v.w, h.y));
    }
    // two values of h and what their rounding left
    static __device__ __forceinline__ void whole(uint32_t h, uint32_t r, float &a, float &b) {
        a = __uint_as_float((h << 16) + static_cast<uint32_t>(static_cast<int>(r << 16) >> 16));
        b = __uint_as_float((h & 0xffff0000u) + static_cast<uint32_t>(static_cast<int>(r) >> 16));
    }
    static __device__ __forceinline__ Frag join(Half a, Half b) {
        Bits x;
        x.d[0] = a;
        x.d[1] = b;
        return x.f;
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
    static __device__ __forceinline__ constexpr int pos(int c) { return c; }
    static __device__ __forceinline__ Frag row_perm(const E *p, int g) {
        const f4 a = *reinterpret_cast<const f4 *>(p + 4 * g), b = *reinterpret_cast<const f4 *>(p + 16 + 4 * g);
        return Frag{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    template <class Vec>
    static __device__ __forceinline__ void put_perm(E *row, int c, const Vec &v) {
        *reinterpret_cast<Vec *>(row + c) = v;
    }
    template <class Vec>
    static __device__ __forceinline__ Vec get_perm(const E *row, int c) {
        return *reinterpret_cast<const Vec *>(row + c);
    }
    template <int FOUR = 4>
    static __device__ __forceinline__ Frag col_perm(const E *m, int stride, int g, int l) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = m[(4 * g + (j & 3) + 16 * (j >> 2)) * stride + l];
        return f;
    }
    static __device__ __forceinline__ f4 fours(const E *p) { return *reinterpret_cast<const f4 *>(p); }
    static __device__ __forceinline__ Frag pack(const float (&v)[8]) {
        return Frag{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    }
    static __device__ __forceinline__ void unpack(Frag f, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
    using Half = f4;
    static __device__ __forceinline__ Half half(f4 v) { return v; }
    static __device__ __forceinline__ void store(Half h, Rsrc to, uint32_t off, int more) {
        store16(h, to, off, more);
    }
    static __device__ __forceinline__ Half none() { return f4{0.0f, 0.0f, 0.0f, 0.0f}; }
    static __device__ __forceinline__ Frag join(Half a, Half b) {
        return Frag{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
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

// Workgroup id -> position: the ids of one XCD (id % 8) become neighbours, so
// that the heads that share B and C share an L2.
__device__ __forceinline__ int64_t by_xcd(int64_t id, int64_t total) {
    const int64_t x = id & 7, q = total >> 3, r = total & 7;
    return x * q + (x < r ? x : r) + (id >> 3);
}

// Inclusive sum over the lanes of a wavefront, in 64 bits: differences of
// these sums are the exponents, and in 32 bits the chunk's later ones would
// lose 1e-6 of the decay.  Four DPP shifts within 16 lanes, then the two
// broadcasts of a row's last lane to the rows behind it.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, false);
    return v + __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);   // 0.0 where nothing comes
}
__device__ __forceinline__ double lane_prefix(double v) {
    v = dpp_add<0x111, 0xf>(v);     // row_shr:1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);     // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xc>(v);     // row_bcast:31 into rows 2 and 3
    return v;
}
// The value of one lane, for all.
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
    return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

// a + b over the groups of 16 lanes, two values at once: lane group 0 and 2 of
// a where 16, the lower half of a where 32 lanes change places with b's.
__device__ __forceinline__ float swap16_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap32_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sums over the four groups of lanes: v[q] of tile q -> lane (g, l) has tile
// g's (of two tiles g % 2's), column l.
template <int TT>
__device__ __forceinline__ float group_sums(const float (&v)[TT]) {
    const float a = swap16_add(v[0], v[1]);
    if constexpr (TT == 2) return swap32_add(a, a);
    else return swap32_add(a, swap16_add(v[2], v[3]));
}

// 2^x of an exponent in 64 bits: what its rounding to float leaves out comes
// back as a factor 1 + lo ln 2.
__device__ __forceinline__ float exp2_d(double x) {
    const float hi = static_cast<float>(x), lo = static_cast<float>(x - hi);
    const float e = exp2_hw(hi);
    return __builtin_fmaf(e * kLn2, lo, e);
}

// softplus to an ulp or two, as ssm_common.h's but with the exponent in 64 bits:
// dA adds up the step sizes' errors over all tokens.
__device__ __forceinline__ float softplus_exact(float x) {
    const float e = exp2_d(static_cast<double>(-fabsf(x)) * 1.4426950408889634);
    const float s = 1.0f + e;
    return fmaxf(x, 0.0f) + __builtin_fmaf(log2_hw(s), kLn2, (1.0f - s) + e);
}

// Host: whether rows of `src` can be read in 16-byte pieces.
template <class IO>
__host__ __device__ inline bool vec_rows(const void *src, int64_t b, int64_t t, int64_t piece) {
    constexpr int V = Seg<IO>::VW;
    return reinterpret_cast<uintptr_t>(src) % 16 == 0 && b % V == 0 && t % V == 0 && piece % V == 0;
}

}  // namespace ssm
