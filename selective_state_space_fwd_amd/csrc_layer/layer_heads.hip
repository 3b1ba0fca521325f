// layer_heads.hip -- the scan over heads: packed sequences, ranges joined, and
// the launch of the forward walks (layer_heads_fwd.h).
#include "layer_mat.h"

namespace ssm {

hipError_t heads_fwd_bf16(const HeadsArgs &a, hipStream_t s);
hipError_t heads_fwd_f32(const HeadsArgs &a, hipStream_t s);

// Joins the ranges: slot j of hend becomes the state that enters range j + 1
// (against time, blockIdx.z 1: j - 1).  Nothing enters a range from the last
// one's end.
__global__ __launch_bounds__(256) void heads_join_kernel(HeadsArgs a) {
    const int64_t per = a.P * a.N, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t h = blockIdx.y % a.H, b = blockIdx.y / a.H;
    if (i >= per) return;
    const bool reverse = blockIdx.z;
    float *hend = a.hend + (reverse ? a.batch * a.J * a.H * per : 0);
    const float *ldec = a.ldec + (reverse ? a.batch * a.J * a.H : 0);
    // eight ranges on their way at a time
    float v = 0.0f;
    for (int64_t x0 = 0; x0 < a.J - 1; x0 += 8) {
        float in[8], d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t x = x0 + e < a.J - 1 ? x0 + e : a.J - 2;
            const int64_t j = b * a.J + (reverse ? a.J - 1 - x : x);
            in[e] = hend[(j * a.H + h) * per + i];
            d[e] = ldec[j * a.H + h];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (x0 + e < a.J - 1) {
                const int64_t j = b * a.J + (reverse ? a.J - 1 - x0 - e : x0 + e);
                v = d[e] == -INFINITY ? in[e] : __builtin_fmaf(exp2_hw(d[e]), v, in[e]);
                hend[(j * a.H + h) * per + i] = v;
            }
    }
}

// Packed sequences: the chunks of each, behind one another; unused ones empty.
__device__ __forceinline__ void heads_table(const HeadsArgs &a, HeadsEntry *table) {
    __shared__ int64_t count[256];
    int64_t base = 0;
    for (int64_t r0 = 0; r0 < a.rows; r0 += 256) {
        const int64_t r = r0 + threadIdx.x;
        int64_t t0 = 0, t1 = 0;
        if (r < a.rows) {
            t0 = seq_at(a.cu, r, a.L);
            t1 = seq_at(a.cu, r + 1, a.L);
            if (t1 < t0) t1 = t0;
        }
        const int64_t n = (t1 - t0 + a.Q - 1) / a.Q;
        count[threadIdx.x] = n;
        __syncthreads();
        for (int o = 1; o < 256; o <<= 1) {     // inclusive sums
            const int64_t w = static_cast<int>(threadIdx.x) >= o ? count[threadIdx.x - o] : 0;
            __syncthreads();
            count[threadIdx.x] += w;
            __syncthreads();
        }
        int64_t at = base + count[threadIdx.x] - n;
        for (int64_t i = 0; i < n && at < a.nc; ++i, ++at) {
            const int64_t t = t0 + i * a.Q, left = t1 - t;
            table[at] = HeadsEntry{static_cast<int32_t>(t), static_cast<int32_t>(left < a.Q ? left : a.Q),
                                   static_cast<int32_t>(r),
                                   (i == 0 ? kFirst : 0) | (i == n - 1 ? kLast : 0)};
        }
        base += count[255];
        __syncthreads();
    }
    for (int64_t at = base + threadIdx.x; at < a.nc; at += 256) table[at] = HeadsEntry{0, 0, 0, 0};
}

// The first workgroup: the table of packed sequences.  The others: sequences
// without a token, whose last state is the one they start from (and the
// gradient of that the gradient of the last).  table, to: null, not wanted.
__global__ __launch_bounds__(256) void heads_rows_kernel(HeadsArgs a, HeadsEntry *table, const float *from,
                                                         float *to) {
    if (blockIdx.y == 0) {
        if (blockIdx.x == 0 && table) heads_table(a, table);
        return;
    }
    const int64_t per = a.H * a.P * a.N;
    for (int64_t r = blockIdx.y - 1; r < a.rows; r += gridDim.y - 1) {
        if (a.cu ? seq_at(a.cu, r, a.L) < seq_at(a.cu, r + 1, a.L) : a.L > 0) continue;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < per;
             i += static_cast<int64_t>(gridDim.x) * 256)
            to[r * per + i] = from ? from[r * per + i] : 0.0f;
    }
}

hipError_t launch_heads_join(const HeadsArgs &a, int walks, hipStream_t s) {
    hipLaunchKernelGGL(heads_join_kernel,
                       dim3(static_cast<unsigned>((a.P * a.N + 255) / 256),
                            static_cast<unsigned>(a.H * a.batch), static_cast<unsigned>(walks)),
                       dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_heads_rows(const HeadsArgs &a, const float *from, float *to, hipStream_t s) {
    HeadsEntry *table = a.cu && a.L > 0 && a.batch > 0 ? const_cast<HeadsEntry *>(a.table) : nullptr;
    const bool empty = to && a.rows > 0 && (a.cu || a.L == 0);
    if (!table && !empty) return hipSuccess;
    const unsigned rows = empty ? static_cast<unsigned>(a.rows < 65534 ? a.rows : 65534) : 0;
    hipLaunchKernelGGL(heads_rows_kernel, dim3(empty ? 16 : 1, rows + 1), dim3(256), 0, s, a, table, from, to);
    return hipGetLastError();
}

hipError_t launch_heads_fwd(const HeadsArgs &a, hipStream_t s) {
    const hipError_t e = launch_heads_rows(a, a.h0, a.last, s);
    if (e != hipSuccess || a.L == 0 || a.batch == 0) return e;
    return a.bf16 ? heads_fwd_bf16(a, s) : heads_fwd_f32(a, s);
}

}  // namespace ssm
