// layer_norm.hip -- root-mean-square norm over groups of a row, with the
// residual's addition in front, the gate silu(z), and an output in 8 bits
// with one scale a block:
//   s = x + residual;  g = s silu(z);  y = g / sqrt(mean g^2 + eps) * weight
//   q = e4m3(y * 448 / max|y|),  scale = max|y| / 448
// Every value is read and written once: HBM bounds it.  A workgroup holds one
// group of a row in registers, so the statistic (float32) and the scale need
// no second read, and there are as many workgroups as groups: walking rows with
// the next one on its way, as the gradients do, has fewer bytes in flight (gated,
// 8 bits, 16384 x 5120: 118 against 100 us).  Measured: gated, 8 bits, 16384 x 5120, 422 MB in 95 us
// (4.4 TB/s; the copy's rate would be 81); gated gradients, 8192 x 5120 in two
// groups, 420 MB in 84 us (5.0 TB/s) and 5 for dweight's partial rows, where the
// copy's rate would be 81; 4 rows of 2560: 4 us, a launch.
#include "layer_common.h"

namespace ssm {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// e4m3 bits of four values, round to nearest even, magnitudes above 448 kept
// at 448 (NaN stays NaN).
__device__ __forceinline__ float clamp8(float v) { return fabsf(v) > 448.0f ? copysignf(448.0f, v) : v; }
__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(clamp8(a), clamp8(b), 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(clamp8(c), clamp8(d), v, true);
}

// A block's scale and its values, for its largest magnitude m.  A block of
// zeros (or below 2^-100, where 448 / m overflows) has scale 0.
__device__ __forceinline__ float scale8(float m) { return m < 0x1p-100f ? 0.0f : m / 448.0f; }
template <int VW>
__device__ __forceinline__ void store8(uint8_t *q, const float (&v)[VW], float m) {
    const float inv = m < 0x1p-100f ? 0.0f : 448.0f / m;
    if constexpr (VW == 1) {
        *q = static_cast<uint8_t>(pack8(v[0] * inv, 0.0f, 0.0f, 0.0f));
    } else {
        uint32_t o[VW / 4];
#pragma unroll
        for (int i = 0; i < VW; i += 4)
            o[i / 4] = pack8(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv);
        __builtin_memcpy(__builtin_assume_aligned(q, VW), o, VW);
    }
}

// The largest magnitude, as bits: those of non-negative floats order as the
// floats do, NaN above all.
template <int VW>
__device__ __forceinline__ uint32_t vec_max(const float (&v)[VW]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VW; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}
// Over the 16 lanes of a row, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, m, 0x121, 0xf, 0xf, false)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, m, 0x122, 0xf, 0xf, false)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, m, 0x124, 0xf, 0xf, false)));
    return max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, m, 0x128, 0xf, 0xf, false)));
}

template <class IO, class RT, int VW, int NV>
__global__ __launch_bounds__(512) void norm_fwd_kernel(NormArgs a) {
    using T = typename IO::T;
    extern __shared__ uint32_t lds[];           // 8 sums, then the blocks' largest magnitudes
    float *red = reinterpret_cast<float *>(lds);
    uint32_t *most = lds + 8;
    const int nw = blockDim.x >> 6, tid = threadIdx.x;
    const int64_t ng = a.d / a.group;
    const int64_t row = blockIdx.x / ng, g0 = (blockIdx.x % ng) * a.group;
    const int nblk = a.block ? static_cast<int>((a.group + a.block - 1) / a.block) : 0;
    const bool lanes = VW > 1 && a.block == 16 * VW;    // a block is a row of 16 lanes
    for (int i = tid; i < nblk; i += blockDim.x) most[i] = 0;

    float v[NV][VW], wt[NV][VW];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
#pragma unroll
        for (int i = 0; i < VW; ++i) v[k][i] = 0.0f;
        if (e < a.group) {
            const int64_t c = g0 + e;
            load_vec<IO, VW>(static_cast<const T *>(a.x) + row * a.x_row + c, v[k]);
            load_vec<F32, VW>(a.weight + c, wt[k]);     // on its way before the sum is known
            if (a.residual) {
                float r[VW];
                load_vec<RT, VW>(static_cast<const typename RT::T *>(a.residual) + row * a.res_row + c, r);
#pragma unroll
                for (int i = 0; i < VW; ++i) v[k][i] += r[i];
                typename RT::T *o = static_cast<typename RT::T *>(a.residual_out) + row * a.d + c;
                store_vec<RT, VW>(o, v[k]);
                // the norm is of the sum as it is kept (the backward reads that)
                if constexpr (sizeof(typename RT::T) == 2) {
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        uint16_t h;
                        BF16::store(&h, 0, v[k][i]);
                        v[k][i] = BF16::load(&h, 0);
                    }
                }
            }
            if (a.z) {
                float z[VW];
                load_vec<IO, VW>(static_cast<const T *>(a.z) + row * a.z_row + c, z);
#pragma unroll
                for (int i = 0; i < VW; ++i) v[k][i] *= silu_f32(z[i]);
            }
#pragma unroll
            for (int i = 0; i < VW; ++i) sum = __builtin_fmaf(v[k][i], v[k][i], sum);
        }
    }
    sum = wave_sum(sum);
    if (nw > 1) {
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < nw; ++w) sum += red[w];
    } else if (nblk) {
        __syncthreads();                        // the cleared magnitudes
    }
    const float rs = 1.0f / sqrtf(sum / static_cast<float>(a.group) + a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
        if (e < a.group) {
#pragma unroll
            for (int i = 0; i < VW; ++i) v[k][i] = v[k][i] * rs * wt[k][i];
            if (!nblk) {
                store_vec<IO, VW>(static_cast<T *>(a.y) + row * a.d + g0 + e, v[k]);
            } else if (!lanes) {
                atomicMax(most + e / a.block, vec_max<VW>(v[k]));   // no order changes a maximum
            }
        }
    }
    if (!nblk) return;
    if (lanes) {
        uint8_t *q = static_cast<uint8_t *>(a.y) + row * a.d + g0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
            const uint32_t m = row_max(vec_max<VW>(v[k]));
            if (e >= a.group) continue;
            store8<VW>(q + e, v[k], __uint_as_float(m));
            if ((tid & 15) == 0)
                a.scale[(row * ng + g0 / a.group) * nblk + e / a.block] = scale8(__uint_as_float(m));
        }
        return;
    }
    __syncthreads();
    uint8_t *q = static_cast<uint8_t *>(a.y) + row * a.d + g0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
        if (e < a.group) store8<VW>(q + e, v[k], __uint_as_float(most[e / a.block]));
    }
    for (int i = tid; i < nblk; i += blockDim.x) {
        a.scale[(row * ng + g0 / a.group) * nblk + i] = scale8(__uint_as_float(most[i]));
    }
}

// Gradients.  n = g rs, dn = dy weight: dg = rs (dn - n mean(dn n)), with
// mean(dn n) = rs mean(dn g), so both sums are taken in one pass over the row.
// A workgroup walks rows nblk apart of one group and keeps dweight of its
// columns in registers: one partial row of dweight a workgroup.
template <class IO, class RT, int VW, int NV>
__global__ __launch_bounds__(512) void norm_bwd_kernel(NormArgs a) {
    using T = typename IO::T;
    using R = typename RT::T;
    __shared__ float red[2][2][8];
    const int nw = blockDim.x >> 6, tid = threadIdx.x;
    const int64_t ng = a.d / a.group, g0 = blockIdx.x % ng * a.group, first = blockIdx.x / ng;
    float dw[NV][VW];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VW; ++i) dw[k][i] = 0.0f;
    // The next row on its way while this one is summed, and the weight kept,
    // where there are registers for it (two vectors a lane: 84 against 99 us at
    // 8192 x 5120 in two gated groups).
    constexpr bool AHEAD = NV * VW <= 16;
    Piece<RT, VW> xn[AHEAD ? NV : 1];
    Piece<IO, VW> yn[AHEAD ? NV : 1], zn[AHEAD ? NV : 1];
    float wk[AHEAD ? NV : 1][VW];
    auto fetch = [&](int k, int64_t row, int64_t c) {
        xn[k].load(static_cast<const R *>(a.x) + row * a.x_row + c);
        yn[k].load(static_cast<const T *>(a.dy) + row * a.dy_row + c);
        if (a.z) zn[k].load(static_cast<const T *>(a.z) + row * a.z_row + c);
    };
    auto weight = [&](int k, int64_t e, float (&w)[VW]) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < VW; ++i) w[i] = wk[k][i];
        } else {
            load_vec<F32, VW>(a.weight + g0 + e, w);
        }
    };
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
            if (e >= a.group) continue;
            load_vec<F32, VW>(a.weight + g0 + e, wk[k]);
            fetch(k, first, g0 + e);           // nblk <= rows
        }
    }
    int par = 0;
    for (int64_t row = first; row < a.rows; row += a.nblk, par ^= 1) {
        float s[NV][VW], z[NV][VW], dy[NV][VW], gate[NV][VW];
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
#pragma unroll
            for (int i = 0; i < VW; ++i) { s[k][i] = 0.0f; z[k][i] = 0.0f; dy[k][i] = 0.0f; gate[k][i] = 1.0f; }
            if (e < a.group) {
                float w[VW];
                if constexpr (AHEAD) {
                    xn[k].get(s[k]);
                    yn[k].get(dy[k]);
                } else {
                    load_vec<RT, VW>(static_cast<const R *>(a.x) + row * a.x_row + g0 + e, s[k]);
                    load_vec<IO, VW>(static_cast<const T *>(a.dy) + row * a.dy_row + g0 + e, dy[k]);
                }
                weight(k, e, w);
                if (a.z) {
                    if constexpr (AHEAD) zn[k].get(z[k]);
                    else load_vec<IO, VW>(static_cast<const T *>(a.z) + row * a.z_row + g0 + e, z[k]);
#pragma unroll
                    for (int i = 0; i < VW; ++i) gate[k][i] = silu_f32(z[k][i]);
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const float g = s[k][i] * gate[k][i];
                    sq = __builtin_fmaf(g, g, sq);
                    dot = __builtin_fmaf(dy[k][i] * w[i], g, dot);
                }
            }
        }
        if constexpr (AHEAD) {
            if (row + a.nblk < a.rows)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
                    if (e < a.group) fetch(k, row + a.nblk, g0 + e);
                }
        }
        sq = wave_sum(sq);
        dot = wave_sum(dot);
        if (nw > 1) {
            if ((tid & 63) == 0) { red[par][0][tid >> 6] = sq; red[par][1][tid >> 6] = dot; }
            __syncthreads();    // the next row writes the other half
            sq = dot = 0.0f;
            for (int w = 0; w < nw; ++w) { sq += red[par][0][w]; dot += red[par][1][w]; }
        }
        const float m = 1.0f / static_cast<float>(a.group);
        const float rs = 1.0f / sqrtf(sq * m + a.eps);
        const float k2 = rs * rs * m * dot;     // rs mean(dn n), per g
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
            if (e < a.group) {
                const int64_t c = g0 + e;
                float w[VW], dx[VW], dz[VW], dr[VW];
                weight(k, e, w);
                if (a.dresidual)
                    load_vec<RT, VW>(static_cast<const R *>(a.dresidual) + row * a.d + c, dr);
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const float g = s[k][i] * gate[k][i];
                    const float dg = rs * (dy[k][i] * w[i] - k2 * g);
                    dw[k][i] = __builtin_fmaf(dy[k][i], g * rs, dw[k][i]);
                    dx[i] = dg * gate[k][i];
                    if (a.dresidual) dx[i] += dr[i];
                    const float sg = sigmoid_f32(z[k][i]);
                    dz[i] = dg * s[k][i] * sg * __builtin_fmaf(z[k][i], 1.0f - sg, 1.0f);
                }
                store_vec<RT, VW>(static_cast<R *>(a.dx) + row * a.d + c, dx);
                if (a.z) store_vec<IO, VW>(static_cast<T *>(a.dz) + row * a.d + c, dz);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t e = (static_cast<int64_t>(k) * blockDim.x + tid) * VW;
        if (e < a.group) store_vec<F32, VW>(a.part + first * a.d + g0 + e, dw[k]);
    }
}

// dweight: the workgroups' partial rows, added in a fixed order: 32 columns by
// 16 lanes, each every 16th row, then the 16 in a tree.
__global__ __launch_bounds__(512) void norm_reduce_kernel(NormArgs a) {
    __shared__ float sum[16][33];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float v = 0.0f;
    if (c < a.d) {
#pragma unroll 8
        for (int64_t r = w; r < a.nblk; r += 16) v += a.part[r * a.d + c];
    }
    sum[w][x] = v;
    for (int n = 8; n > 0; n >>= 1) {
        __syncthreads();
        if (w < n) sum[w][x] += sum[w + n][x];
    }
    if (w == 0 && c < a.d) a.dweight[c] = sum[0][x];
}

// ------------------------------------------------------------------ launch
static bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 16-byte accesses need whole vectors in a group (and a block) and aligned rows.
static bool norm_vec(const NormArgs &a, int V) {
    bool ok = a.group % V == 0 && al16(a.weight) && al16(a.x) && a.x_row % V == 0;
    ok = ok && al16(a.z) && (!a.z || a.z_row % V == 0);
    ok = ok && al16(a.residual) && (!a.residual || a.res_row % V == 0) && al16(a.residual_out);
    ok = ok && al16(a.dy) && (!a.dy || a.dy_row % V == 0) && al16(a.dresidual);
    ok = ok && al16(a.y) && al16(a.dx) && al16(a.dz) && al16(a.part);
    return ok && a.block % V == 0;
}

int64_t norm_bwd_blocks(int64_t rows, int64_t d, int64_t group) {
    const int64_t ng = d / group, want = 1024 / ng < 64 ? 64 : 1024 / ng;
    return rows < want ? rows : want;
}

template <class IO, class RT, int VW, int NV>
static hipError_t norm_go(const NormArgs &a, bool bwd, int threads, hipStream_t s) {
    const int64_t ng = a.d / a.group;
    if (!bwd) {
        const int64_t nblk = a.block ? (a.group + a.block - 1) / a.block : 0;
        hipLaunchKernelGGL((norm_fwd_kernel<IO, RT, VW, NV>),
                           dim3(static_cast<unsigned>(a.rows * ng)), dim3(threads),
                           static_cast<unsigned>(4 * (8 + nblk)), s, a);
        return hipGetLastError();
    }
    if (a.nblk > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<IO, RT, VW, NV>),
                           dim3(static_cast<unsigned>(a.nblk * ng)),
                           dim3(threads), 0, s, a);
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)), dim3(512),
                       0, s, a);
    return hipGetLastError();
}

template <class IO, class RT, int VW>
static hipError_t norm_vw(const NormArgs &a, bool bwd, hipStream_t s) {
    // Vectors a lane holds: one up to 256 vectors a group, then the least that
    // keeps the workgroup within 512 lanes.  (8192 rows of 5120 and of 8192 in
    // bfloat16, two vectors a lane against four: 30 and 43 against 31 and 45 us,
    // gradients 98 and 113 against 102 and 141.)
    const int64_t nvec = (a.group + VW - 1) / VW;
    const int nv = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : nvec <= 4096 ? 8 : 32;
    const int threads = static_cast<int>(((nvec + nv - 1) / nv + 63) / 64 * 64);
    if (nv == 1) return norm_go<IO, RT, VW, 1>(a, bwd, threads, s);
    if (nv == 2) return norm_go<IO, RT, VW, 2>(a, bwd, threads, s);
    if constexpr (VW <= 8)
        if (nv == 4) return norm_go<IO, RT, VW, 4>(a, bwd, threads, s);
    if constexpr (VW <= 4)
        if (nv == 8) return norm_go<IO, RT, VW, 8>(a, bwd, threads, s);
    if constexpr (VW == 1) return norm_go<IO, RT, VW, 32>(a, bwd, threads, s);
    return hipErrorInvalidValue;
}

static hipError_t launch_norm(const NormArgs &a, bool bwd, hipStream_t s) {
    if (a.bf16 && a.res_bf16)
        return norm_vec(a, 8) ? norm_vw<BF16, BF16, 8>(a, bwd, s) : norm_vw<BF16, BF16, 1>(a, bwd, s);
    if (a.bf16)
        return norm_vec(a, 8) ? norm_vw<BF16, F32, 8>(a, bwd, s) : norm_vw<BF16, F32, 1>(a, bwd, s);
    return norm_vec(a, 4) ? norm_vw<F32, F32, 4>(a, bwd, s) : norm_vw<F32, F32, 1>(a, bwd, s);
}
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s) { return launch_norm(a, false, s); }
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t s) { return launch_norm(a, true, s); }

}  // namespace ssm
