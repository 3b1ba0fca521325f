// layer_common.h -- device helpers shared by the layer operators.
#pragma once

#include "layer_launch.h"
#include "ssm_common.h"

namespace ssm {

// Two values to bfloat16 in one instruction, nearest even.  (The header's
// conversion of two becomes two instructions, a shift and an or: 348 against
// 310 us of the backward walks at 4 x 2048 x 80 heads.)
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// VW consecutive values of a row as they lie in memory (one access of up to
// 16 bytes), and as floats.
template <class IO, int VW>
struct Piece {
    using T = typename IO::T;
    static constexpr int kBytes = VW * sizeof(T);
    uint32_t raw[(kBytes + 3) / 4];
    __device__ __forceinline__ void load(const T *p) {
        __builtin_memcpy(raw, __builtin_assume_aligned(p, kBytes < 16 ? kBytes : 16), kBytes);
    }
    __device__ __forceinline__ void get(float (&o)[VW]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VW; ++i) o[i] = __uint_as_float(raw[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VW; ++i)
                o[i] = __uint_as_float(i & 1 ? raw[i / 2] & 0xffff0000u : raw[i / 2] << 16);
        }
    }
};

template <class IO, int VW>
__device__ __forceinline__ void load_vec(const typename IO::T *p, float (&o)[VW]) {
    Piece<IO, VW> v;
    v.load(p);
    v.get(o);
}

template <class IO, int VW>
__device__ __forceinline__ void store_vec(typename IO::T *p, const float (&o)[VW]) {
    if constexpr (VW == 1) {
        IO::store(p, 0, o[0]);
    } else if constexpr (sizeof(typename IO::T) == 2) {
        uint32_t raw[VW / 2];
#pragma unroll
        for (int i = 0; i < VW; i += 2) raw[i / 2] = pack2(o[i], o[i + 1]);
        __builtin_memcpy(__builtin_assume_aligned(p, VW * 2), raw, VW * 2);
    } else {
#pragma unroll
        for (int i = 0; i < VW; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
}

__device__ __forceinline__ float sigmoid_f32(float v) {
    return rcp_hw(1.0f + exp2_hw(-v * kLog2e));
}

// Offset r of a packed batch, inside 0 .. L whatever the table holds.
__device__ __forceinline__ int64_t seq_at(const int32_t *cu, int64_t r, int64_t L) {
    const int64_t v = cu[r];
    return v < 0 ? 0 : v > L ? L : v;
}

// The sequence that holds token t: the last r with cu[r] <= t (so empty
// sequences before it are passed over); -1 if t lies before the first.
__device__ __forceinline__ int64_t seq_of(const int32_t *cu, int64_t n, int64_t t, int64_t L) {
    int64_t lo = -1, hi = n;      // cu[lo] <= t < cu[hi], in the mind's eye
    while (hi - lo > 1) {
        const int64_t m = (lo + hi) >> 1;
        if (seq_at(cu, m, L) <= t) lo = m; else hi = m;
    }
    return lo;
}

}  // namespace ssm
