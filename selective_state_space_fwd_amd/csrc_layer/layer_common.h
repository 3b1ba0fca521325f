// layer_common.h -- device helpers shared by the layer operators.
#pragma once

#include "layer_launch.h"
#include "ssm_common.h"

namespace ssm {

// VW consecutive values of a row as floats: one 16-byte access (8 for VW = 4
// of 16 bits), or single elements for VW = 1.
template <class IO, int VW>
__device__ __forceinline__ void load_vec(const typename IO::T *p, float (&o)[VW]) {
    if constexpr (VW == 1) {
        o[0] = IO::load(p, 0);
    } else if constexpr (sizeof(typename IO::T) == 2) {
        static_assert(VW == 8, "eight 16-bit values");
        Seg<BF16>::unpack(*reinterpret_cast<const uint4 *>(p), o);
    } else {
#pragma unroll
        for (int i = 0; i < VW; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            o[i] = v.x; o[i + 1] = v.y; o[i + 2] = v.z; o[i + 3] = v.w;
        }
    }
}

template <class IO, int VW>
__device__ __forceinline__ void store_vec(typename IO::T *p, const float (&o)[VW]) {
    if constexpr (VW == 1) {
        IO::store(p, 0, o[0]);
    } else if constexpr (sizeof(typename IO::T) == 2) {
        static_assert(VW == 8, "eight 16-bit values");
        *reinterpret_cast<uint4 *>(p) = Seg<BF16>::pack(o);
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
