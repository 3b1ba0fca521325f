// layer_update.hip -- one token of the scan over heads:
//   dt = softplus(delta + bias);  h = exp(dt A) h + dt u (x) B;  y = h C + D u
// A pure stream over the state (8 bytes a state value, read and written once
// past the caches); everything else is small, so HBM bounds it: 253 us at 256 x
// 80 heads x 64 x 128, 1.35 GB at 5.3 TB/s, which is what a large copy reaches.
// One row of 80 heads takes 6 us, which is what a launch takes.
#include "layer_common.h"

namespace ssm {

typedef float f4v __attribute__((ext_vector_type(4)));

// A workgroup: kRows channels (rows of the state) of one head of one token, Q
// lanes a channel (the power of two that covers N with 4 states a lane).
// VEC: 16-byte accesses (N % 4 == 0, aligned state).
template <class IO, bool VEC, int R>
__global__ __launch_bounds__(256) void heads_update_kernel(HeadsArgs a, int log2q, int blocks) {
    using T = typename IO::T;
    const int Q = 1 << log2q, rows = 256 >> log2q;
    int64_t id = blockIdx.x;
    const int pb = static_cast<int>(id % blocks);
    id /= blocks;
    const int64_t h = id % a.H, b = id / a.H;
    const int64_t slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.n_slots) return;
    const int l = threadIdx.x & (Q - 1), n0 = 4 * l;
    const int64_t g = h / (a.H / a.G);
    const T *u = static_cast<const T *>(a.u) + b * a.u_b + h * a.P;
    const T *Bp = static_cast<const T *>(a.B) + b * a.B_b + g * a.N;
    const T *Cp = static_cast<const T *>(a.C) + b * a.C_b + g * a.N;
    float *st = a.state + (slot * a.H + h) * a.P * a.N;
    const int p0 = pb * rows * R + (threadIdx.x >> log2q);

    float s[R][4], uu[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int p = p0 + k * rows;
        uu[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k][i] = 0.0f;
        if (p < a.P && n0 < a.N) {
            uu[k] = IO::load(u, p);
            if constexpr (VEC) {
                const f4v v = __builtin_nontemporal_load(
                    reinterpret_cast<const f4v *>(st + static_cast<int64_t>(p) * a.N + n0));
                s[k][0] = v.x; s[k][1] = v.y; s[k][2] = v.z; s[k][3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < a.N) s[k][i] = st[static_cast<int64_t>(p) * a.N + n0 + i];
            }
        }
    }
    float dt = IO::load(static_cast<const T *>(a.delta) + b * a.dt_b, h);
    if (a.bias) dt += a.bias[h];
    if (a.softplus) dt = softplus_f32(dt);
    const float decay = exp2_hw(dt * (a.A[h] * kLog2e));
    const float Dh = a.D ? a.D[h] : 0.0f;
    float bv[4], cv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = n0 + i < a.N;
        bv[i] = in ? IO::load(Bp, n0 + i) : 0.0f;
        cv[i] = in ? IO::load(Cp, n0 + i) : 0.0f;
    }
    T *y = static_cast<T *>(a.y) + (b * a.H + h) * a.P;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int p = p0 + k * rows;
        const float w = dt * uu[k];
        float acc = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[k][i] = __builtin_fmaf(decay, s[k][i], w * bv[i]);
            acc = __builtin_fmaf(s[k][i], cv[i], acc);
        }
        if (p < a.P && n0 < a.N) {
            if constexpr (VEC) {
                const f4v v = {s[k][0], s[k][1], s[k][2], s[k][3]};
                __builtin_nontemporal_store(
                    v, reinterpret_cast<f4v *>(st + static_cast<int64_t>(p) * a.N + n0));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < a.N) st[static_cast<int64_t>(p) * a.N + n0 + i] = s[k][i];
            }
        }
        for (int o = Q >> 1; o > 0; o >>= 1) acc += __shfl_xor(acc, o, 64);
        if (l == 0 && p < a.P) IO::store(y, p, __builtin_fmaf(Dh, uu[k], acc));
    }
}

template <class IO>
static hipError_t update_io(const HeadsArgs &a, hipStream_t s) {
    int log2q = 0;
    while ((4 << log2q) < a.N) ++log2q;
    const int rows = 256 >> log2q;
    const bool vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
    // Four state pieces in flight a lane where that leaves two workgroups a
    // compute unit (four against one, 80 heads: 6.9 and 6.3 us at 1 row, 8.8 and
    // 10.3 at 4, 11.5 and 16.6 at 8, 261 and 413 at 256).
    const int64_t heads = a.batch * a.H;
    const bool big = heads * ((a.P + rows * 4 - 1) / (rows * 4)) >= 512;
    const int R = big ? 4 : 1;
    const int blocks = static_cast<int>((a.P + rows * R - 1) / (rows * R));
    const dim3 grid(static_cast<unsigned>(heads * blocks));
    if (vec && big) hipLaunchKernelGGL((heads_update_kernel<IO, true, 4>), grid, dim3(256), 0, s, a, log2q, blocks);
    else if (vec) hipLaunchKernelGGL((heads_update_kernel<IO, true, 1>), grid, dim3(256), 0, s, a, log2q, blocks);
    else if (big) hipLaunchKernelGGL((heads_update_kernel<IO, false, 4>), grid, dim3(256), 0, s, a, log2q, blocks);
    else hipLaunchKernelGGL((heads_update_kernel<IO, false, 1>), grid, dim3(256), 0, s, a, log2q, blocks);
    return hipGetLastError();
}

hipError_t launch_heads_update(const HeadsArgs &a, hipStream_t s) {
    return a.bf16 ? update_io<BF16>(a, s) : update_io<F32>(a, s);
}

}  // namespace ssm
