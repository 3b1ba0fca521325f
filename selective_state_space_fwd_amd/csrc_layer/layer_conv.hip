// layer_conv.hip -- the short causal depthwise convolution in front of the
// scan, token-major: v_t = bias + sum_k w_k x_{t-(W-1)+k}, y = silu(v).
//
// Forward, gradients and the single-token step are streams: each input is
// read and each output written once, and a few multiplications per value lie
// far below the vector rate, so HBM bounds them.  A lane owns four
// neighbouring channels and walks a run of tokens with the last W - 1 inputs
// in registers; the runs' W - 1 overlapping tokens come from the caches.
// Measured, 5376 channels of width 4 in bfloat16: 8 x 2048 tokens 353 MB in 76
// us (4.6 TB/s; a copy of as much takes 68), gradients of 4 x 2048 264 MB in 72
// us with the sums over the runs (3.7 TB/s; v is made again, and silu' takes an
// exponential and a reciprocal a value); a token of 256 rows in float32, 44 MB,
// in 12 us.
#include "layer_common.h"

namespace ssm {

// A lane's view of the sequence that a run of tokens is in.
struct SeqRun {
    int64_t row, begin, end;    // state row, first token, one past the last
};

__device__ __forceinline__ SeqRun seq_run(const ConvArgs &a, int64_t b, int64_t t) {
    if (!a.cu) return {b, 0, a.L};
    const int64_t r = seq_of(a.cu, a.rows, t, a.L);
    if (r < 0 || r >= a.rows) return {-1, t, t};
    return {r, seq_at(a.cu, r, a.L), seq_at(a.cu, r + 1, a.L)};
}

template <class IO, int VW, int W>
struct Taps {
    float w[W][VW], bias[VW];
    __device__ __forceinline__ void load(const ConvArgs &a, int64_t c) {
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = a.weight[(c + i) * W + k];
        }
    }
};

// The input at token t of the run's sequence; before its first token the
// sequence's state (or zero).
template <class IO, int VW, int W>
__device__ __forceinline__ void input_at(const ConvArgs &a, const SeqRun &q, int64_t b, int64_t t,
                                         int64_t c, float (&o)[VW]) {
    if (t >= q.begin) {
        load_vec<IO, VW>(static_cast<const typename IO::T *>(a.x) + b * a.x_batch +
                             t * a.x_token + c, o);
        return;
    }
    const int64_t k = W - 1 + t - q.begin;      // 0 .. W-2
#pragma unroll
    for (int i = 0; i < VW; ++i)
        o[i] = a.state && k >= 0 ? a.state[(q.row * a.C + c + i) * (W - 1) + k] : 0.0f;
}

// RUN: tokens a lane walks.
template <class IO, int VW, int W, int RUN>
__global__ __launch_bounds__(64) void conv_fwd_kernel(ConvArgs a) {
    using T = typename IO::T;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x) * VW;
    const int64_t nrun = (a.L + RUN - 1) / RUN;
    if (c >= a.C) return;
    Taps<IO, VW, W> k;
    k.load(a, c);
    for (int64_t id = blockIdx.y; id < a.batch * nrun; id += gridDim.y) {
        const int64_t b = id / nrun, t0 = (id % nrun) * RUN;
        const int64_t t1 = t0 + RUN < a.L ? t0 + RUN : a.L;
        int64_t t = t0;
        while (t < t1) {
            const SeqRun q = seq_run(a, b, t);
            const int64_t e = q.end < t1 ? q.end : t1;
            if (e <= t) break;                  // behind the last sequence
            float h[W][VW];                     // h[W-1]: the current input
#pragma unroll
            for (int j = 1; j < W; ++j) input_at<IO, VW, W>(a, q, b, t - W + j, c, h[j]);
            // the run's tokens all on their way before the first is used
            const T *x = static_cast<const T *>(a.x) + b * a.x_batch + t * a.x_token + c;
            Piece<IO, VW> in[RUN];
#pragma unroll
            for (int n = 0; n < RUN; ++n)
                if (t + n < e) in[n].load(x + n * a.x_token);
#pragma unroll
            for (int n = 0; n < RUN; ++n) {
                if (t + n < e) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                        for (int i = 0; i < VW; ++i) h[j][i] = h[j + 1][i];
                    in[n].get(h[W - 1]);
                    float o[VW];
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        float v = k.bias[i];
#pragma unroll
                        for (int j = 0; j < W; ++j) v = __builtin_fmaf(k.w[j][i], h[j][i], v);
                        o[i] = a.silu ? silu_f32(v) : v;
                    }
                    store_vec<IO, VW>(static_cast<T *>(a.y) + (b * a.L + t + n) * a.C + c, o);
                }
            }
            t = e;
            if (a.last && t == q.end) {
#pragma unroll
                for (int i = 0; i < VW; ++i)
#pragma unroll
                    for (int j = 1; j < W; ++j)
                        a.last[(q.row * a.C + c + i) * (W - 1) + j - 1] = h[j][i];
            }
        }
    }
}

// The last state (or, in the backward, the state's gradient) of sequences
// without a token: the state they started from, or zero.
__global__ void conv_empty_kernel(const int32_t *cu, int64_t L, int64_t rows, int64_t per_row,
                                  const float *from, float *to) {
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        if (cu ? seq_at(cu, r, L) < seq_at(cu, r + 1, L) : L > 0) continue;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < per_row;
             i += static_cast<int64_t>(gridDim.x) * 256)
            to[r * per_row + i] = from ? from[r * per_row + i] : 0.0f;
    }
}

// silu'(v) dy, or dy without the activation.
__device__ __forceinline__ float act_grad(int silu, float v, float dy) {
    if (!silu) return dy;
    const float s = sigmoid_f32(v);
    return dy * s * __builtin_fmaf(v, 1.0f - s, 1.0f);
}

constexpr int kBatch = 4;       // tokens that the backward fetches ahead

// Gradients.  With dv = silu'(v) dy: dx_t = sum_k w_k dv_{t+W-1-k},
// dweight_k = sum_t dv_t x_{t-W+1+k}, dbias = sum_t dv_t.  A run recomputes v
// of its own tokens and of the W - 1 behind it (whose dv reach into it); the
// sums over tokens leave as one partial row a run, added in a fixed order.
template <class IO, int VW, int W>
__global__ __launch_bounds__(64) void conv_bwd_kernel(ConvArgs a) {
    using T = typename IO::T;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x) * VW;
    const int64_t per = (a.L + a.run - 1) / a.run;
    if (c >= a.C) return;
    Taps<IO, VW, W> k;
    k.load(a, c);
    for (int64_t id = blockIdx.y; id < a.runs; id += gridDim.y) {
        const int64_t b = id / per, t0 = (id % per) * a.run;
        const int64_t t1 = t0 + a.run < a.L ? t0 + a.run : a.L;
        float dw[W][VW], db[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            db[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][i] = 0.0f;
        }
        int64_t t = t0;
        while (t < t1) {
            const SeqRun q = seq_run(a, b, t);
            if (q.end <= t) break;
            const int64_t own = q.end < t1 ? q.end : t1;       // tokens whose dx this run writes
            const int64_t e = own + W - 1 < q.end ? own + W - 1 : q.end;
            float h[W][VW], g[W][VW];           // inputs, and dv of the last W tokens
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < VW; ++i) { h[j][i] = 0.0f; g[j][i] = 0.0f; }
#pragma unroll
            for (int j = 1; j < W; ++j) input_at<IO, VW, W>(a, q, b, t - W + j, c, h[j]);
            const int64_t from = t;
            const T *x = static_cast<const T *>(a.x) + b * a.x_batch + t * a.x_token + c;
            const T *y = static_cast<const T *>(a.dy) + b * a.dy_batch + t * a.dy_token + c;
            // kBatch tokens at a time, the next ones on their way meanwhile
            Piece<IO, VW> xi[kBatch], yi[kBatch], xn[kBatch], yn[kBatch];
            auto fetch = [&](int64_t at) {
#pragma unroll
                for (int n = 0; n < kBatch; ++n)
                    if (from + at + n < e) {
                        xn[n].load(x + (at + n) * a.x_token);
                        yn[n].load(y + (at + n) * a.dy_token);
                    }
            };
            fetch(0);
            // past e the gradients are zero: the loop runs on to write the last dx
            while (t < own + W - 1) {
#pragma unroll
                for (int n = 0; n < kBatch; ++n) { xi[n] = xn[n]; yi[n] = yn[n]; }
                fetch(t - from + kBatch);
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    if (t >= own + W - 1) break;
                    float dy[VW];
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                        for (int i = 0; i < VW; ++i) { h[j][i] = h[j + 1][i]; g[j][i] = g[j + 1][i]; }
                    if (t < e) {
                        xi[n].get(h[W - 1]);
                        yi[n].get(dy);
                    }
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        float v = k.bias[i];
#pragma unroll
                        for (int j = 0; j < W; ++j) v = __builtin_fmaf(k.w[j][i], h[j][i], v);
                        g[W - 1][i] = t < e ? act_grad(a.silu, v, dy[i]) : 0.0f;
                        if (t < own) {
                            db[i] += g[W - 1][i];
#pragma unroll
                            for (int j = 0; j < W; ++j)
                                dw[j][i] = __builtin_fmaf(g[W - 1][i], h[j][i], dw[j][i]);
                        }
                    }
                    const int64_t p = t - (W - 1);  // the token whose last dv this was
                    if (p >= from) {
                        float o[VW];
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
                            float v = 0.0f;
#pragma unroll
                            for (int j = 0; j < W; ++j) v = __builtin_fmaf(k.w[W - 1 - j][i], g[j][i], v);
                            o[i] = v;
                        }
                        store_vec<IO, VW>(static_cast<T *>(a.dx) + (b * a.L + p) * a.C + c, o);
                    }
                    ++t;
                }
            }
            t = own;
        }
        float *part = a.part + id * (W + 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < W; ++j) store_vec<F32, VW>(part + j * a.C, dw[j]);
        store_vec<F32, VW>(part + W * a.C, db);
    }
}

// dstate: the same sum for the W - 1 inputs before each sequence.
template <class IO, int W>
__global__ __launch_bounds__(256) void conv_dstate_kernel(ConvArgs a) {
    using T = typename IO::T;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= a.C) return;
    Taps<IO, 1, W> k;
    k.load(a, c);
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const int64_t b = a.cu ? 0 : r;
        const int64_t begin = a.cu ? seq_at(a.cu, r, a.L) : 0;
        const int64_t end = a.cu ? seq_at(a.cu, r + 1, a.L) : a.L;
        const SeqRun q{r, begin, end};
        float g[W];
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) {
            const int64_t t = begin + j;
            g[j] = 0.0f;
            if (t >= end) continue;
            float v = k.bias[0], dy[1], x[1];
#pragma unroll
            for (int m = 0; m < W; ++m) {
                input_at<IO, 1, W>(a, q, b, t - W + 1 + m, c, x);
                v = __builtin_fmaf(k.w[m][0], x[0], v);
            }
            load_vec<IO, 1>(static_cast<const T *>(a.dy) + b * a.dy_batch + t * a.dy_token + c, dy);
            g[j] = act_grad(a.silu, v, dy[0]);
        }
        // state column i is the input at begin - (W-1) + i: it meets token
        // begin + j with tap i - j
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) {
            float v = 0.0f;
#pragma unroll
            for (int j = 0; j <= i; ++j) v = __builtin_fmaf(k.w[i - j][0], g[j], v);
            a.dstate[(r * a.C + c) * (W - 1) + i] = v;
        }
    }
}

// dweight and dbias: the runs' partial rows, added in a fixed order: 32 columns
// by 16 lanes, each every 16th run, then the 16 in a tree.
template <int W>
__global__ __launch_bounds__(512) void conv_reduce_kernel(ConvArgs a) {
    __shared__ float sum[16][33];
    const int64_t cols = (W + 1) * a.C;
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float v = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int64_t r = w; r < a.runs; r += 16) v += a.part[r * cols + col];
    }
    sum[w][x] = v;
    for (int n = 8; n > 0; n >>= 1) {
        __syncthreads();
        if (w < n) sum[w][x] += sum[w + n][x];
    }
    if (w || col >= cols) return;
    v = sum[0][x];
    const int64_t k = col / a.C, c = col % a.C;
    if (k < W) a.dweight[c * W + k] = v;
    else if (a.dbias) a.dbias[c] = v;
}

// One token of each row: taps from the row's slot, which moves on by one.
template <class IO, int VW, int W>
__global__ __launch_bounds__(256) void conv_update_kernel(ConvArgs a) {
    using T = typename IO::T;
    const int64_t per = a.C / VW;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.batch * per) return;
    const int64_t r = id / per, c = (id % per) * VW;
    const int64_t slot = a.slots ? a.slots[r] : r;
    if (slot < 0 || slot >= a.n_slots) return;
    constexpr int S = W - 1;
    float st[VW * S + 1], x[VW], o[VW];
    float *p = a.slot_state + (slot * a.C + c) * S;
    if constexpr (VW > 1 && S > 0) {
#pragma unroll
        for (int i = 0; i < VW * S; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            st[i] = v.x; st[i + 1] = v.y; st[i + 2] = v.z; st[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VW * S; ++i) st[i] = p[i];
    }
    load_vec<IO, VW>(static_cast<const T *>(a.x) + r * a.x_batch + c, x);
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        const float *w = a.weight + (c + i) * W;
        float v = a.bias ? a.bias[c + i] : 0.0f;
#pragma unroll
        for (int j = 0; j < S; ++j) v = __builtin_fmaf(w[j], st[i * S + j], v);
        v = __builtin_fmaf(w[S], x[i], v);
        o[i] = a.silu ? silu_f32(v) : v;
#pragma unroll
        for (int j = 0; j + 1 < S; ++j) st[i * S + j] = st[i * S + j + 1];
        if constexpr (S > 0) st[i * S + S - 1] = x[i];
    }
    store_vec<IO, VW>(static_cast<T *>(a.y) + r * a.C + c, o);
    if constexpr (VW > 1 && S > 0) {
#pragma unroll
        for (int i = 0; i < VW * S; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < VW * S; ++i) p[i] = st[i];
    }
}

// ------------------------------------------------------------------ launch
static bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
template <class IO>
static bool al4(const void *p) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(typename IO::T)) == 0; }
static unsigned grid_y(int64_t n) { return static_cast<unsigned>(n < 65535 ? n : 65535); }

// Four channels at a time need whole fours and aligned rows.
template <class IO>
static bool conv_vec(const ConvArgs &a, bool bwd) {
    constexpr int V = 4;
    bool ok = a.C % V == 0 && al4<IO>(a.x) && a.x_token % V == 0 && a.x_batch % V == 0;
    if (bwd) ok = ok && al4<IO>(a.dy) && a.dy_token % V == 0 && a.dy_batch % V == 0 && al4<IO>(a.dx) &&
                  al16(a.part);
    else ok = ok && al4<IO>(a.y);
    return ok && (!a.slot_state || al16(a.slot_state));
}

template <class IO, int VW, int W, int RUN>
static void conv_fwd_run(const ConvArgs &a, unsigned gx, hipStream_t s) {
    const int64_t runs = a.batch * ((a.L + RUN - 1) / RUN);
    if (runs > 0)
        hipLaunchKernelGGL((conv_fwd_kernel<IO, VW, W, RUN>), dim3(gx, grid_y(runs)), dim3(64), 0, s, a);
}

// Runs of 24 tokens where their 8-byte pieces fit the registers and leave eight
// wavefronts a SIMD to come; else of 16 (8 x 2048 x 5376 in bfloat16: 76 against
// 82 us, x 1024: 19.5 against 17.7; 4 x 2048 x 5376 in float32: 74 against 69).
template <class IO, int VW, int W>
static hipError_t conv_fwd_w(const ConvArgs &a, hipStream_t s) {
    const unsigned gx = static_cast<unsigned>((a.C + 64 * VW - 1) / (64 * VW));
    if (sizeof(typename IO::T) * VW == 8 && gx * a.batch * (a.L / 24) >= 8192)
        conv_fwd_run<IO, VW, W, sizeof(typename IO::T) * VW == 8 ? 24 : 16>(a, gx, s);
    else
        conv_fwd_run<IO, VW, W, 16>(a, gx, s);
    if (W > 1 && a.last && (a.cu || a.L == 0) && a.rows > 0)
        hipLaunchKernelGGL(conv_empty_kernel, dim3(4, grid_y(a.rows)), dim3(256), 0, s, a.cu, a.L,
                           a.rows, a.C * (W - 1), a.state, a.last);
    return hipGetLastError();
}

template <class IO, int VW, int W>
static hipError_t conv_bwd_w(const ConvArgs &a, hipStream_t s) {
    const unsigned gx = static_cast<unsigned>((a.C + 64 * VW - 1) / (64 * VW));
    if (a.runs > 0)
        hipLaunchKernelGGL((conv_bwd_kernel<IO, VW, W>), dim3(gx, grid_y(a.runs)), dim3(64), 0, s, a);
    hipLaunchKernelGGL((conv_reduce_kernel<W>),
                       dim3(static_cast<unsigned>(((W + 1) * a.C + 31) / 32)), dim3(512), 0, s, a);
    if (W > 1 && a.dstate && a.rows > 0)
        hipLaunchKernelGGL((conv_dstate_kernel<IO, W>),
                           dim3(static_cast<unsigned>((a.C + 255) / 256), grid_y(a.rows)),
                           dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class IO, int VW, int W>
static hipError_t conv_update_w(const ConvArgs &a, hipStream_t s) {
    const int64_t n = a.batch * (a.C / VW);
    hipLaunchKernelGGL((conv_update_kernel<IO, VW, W>), dim3(static_cast<unsigned>((n + 255) / 256)),
                       dim3(256), 0, s, a);
    return hipGetLastError();
}

// Bfloat16 goes by 8 bytes a lane: 16 would need twice the registers for taps,
// tokens on their way and sums, and give half the wavefronts (forward, 8 x
// 2048 x 5376: 80 against 90 us).
#define CONV_BY_WIDTH(NAME, BWD)                                                     \
    template <class IO, int VW>                                                      \
    static hipError_t NAME##_io(const ConvArgs &a, hipStream_t s) {                  \
        return a.W == 4 ? NAME##_w<IO, VW, 4>(a, s) : a.W == 3 ? NAME##_w<IO, VW, 3>(a, s) \
             : a.W == 2 ? NAME##_w<IO, VW, 2>(a, s) : NAME##_w<IO, VW, 1>(a, s);     \
    }                                                                                \
    hipError_t launch_##NAME(const ConvArgs &a, hipStream_t s) {                     \
        if (a.bf16)                                                                  \
            return conv_vec<BF16>(a, BWD) ? NAME##_io<BF16, 4>(a, s) : NAME##_io<BF16, 1>(a, s); \
        return conv_vec<F32>(a, BWD) ? NAME##_io<F32, 4>(a, s) : NAME##_io<F32, 1>(a, s); \
    }
CONV_BY_WIDTH(conv_fwd, false)
CONV_BY_WIDTH(conv_bwd, true)
CONV_BY_WIDTH(conv_update, false)
#undef CONV_BY_WIDTH

}  // namespace ssm
