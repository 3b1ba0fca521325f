// layer_heads.hip -- the scan over heads: one decay a head and token, B and C
// shared by the heads of a group, a state of head_dim x d_state a head:
//   h_t = exp(a_t) h_{t-1} + dt_t u_t (x) B_t,  a_t = dt_t A,  y_t = h_t C_t + D u_t
//
// In chunks of Q tokens, with s the running sum of a in the chunk:
//   y_t = exp(s_t) C_t h_in + sum_{s<=t} (C_t . B_s) exp(s_t - s_s) dt_s u_s + D u_t
//   h_out = exp(s_Q) h_in + sum_s exp(s_Q - s_s) dt_s u_s (x) B_s
// which are products for the matrix cores.  A workgroup of 4 wavefronts walks
// the chunks of one batch row (or a range of them); each wavefront keeps the
// state of its 16 PT channels in registers in float32, and the four share B, C
// and the products C_t . B_s in LDS.  So u is read and y written once and no
// state goes through memory.  Long rows with few heads are cut into ranges: a
// first launch computes each range's end state from zero, a second joins them.
#include "layer_mat.h"

namespace ssm {

// The wavefront's slice of channels: 16 PT of one head.  Slices of a group's
// heads lie behind one another; a workgroup takes four.
struct Slice {
    int64_t g, h;
    int p0, cols;       // first channel of the head, channels (0: none)
};

template <int PT>
__device__ __forceinline__ Slice slice_of(const HeadsArgs &a, int64_t wg, int w) {
    const int64_t hpg = a.H / a.G, sph = (a.P + 16 * PT - 1) / (16 * PT);
    const int64_t per = (hpg * sph + 3) / 4;
    const int64_t g = wg / per, i = (wg % per) * 4 + w;
    Slice s{g, 0, 0, 0};
    if (i < hpg * sph) {
        s.h = g * hpg + i / sph;
        s.p0 = static_cast<int>(i % sph) * 16 * PT;
        const int64_t left = a.P - s.p0;
        s.cols = static_cast<int>(left < 16 * PT ? left : 16 * PT);
    } else {
        s.h = g * hpg;      // an idle wavefront reads head values it does not use
    }
    return s;
}

template <class IO, int NP, int PT, int Q, bool FULL>
__global__ __launch_bounds__(256) void heads_fwd_kernel(HeadsArgs a, int vecs) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32;
    constexpr int LB = NP + M::kPad, UW = 64 * PT, LU = UW + M::kPad;
    constexpr int TRI = TT * (TT + 1) / 2;
    __shared__ __attribute__((aligned(16))) E Bs[Q * LB];
    __shared__ __attribute__((aligned(16))) E Cs[FULL ? Q * LB : 8];
    __shared__ __attribute__((aligned(16))) E Us[Q * LU];
    __shared__ f4 CB[FULL ? TRI * 64 : 1];
    // per wavefront and token: exp(s), dt exp(s_Q - s); exp(s - r), s - r and
    // dt with r the sum before the token's tile; dt exp(r_j - s) for tiles j
    __shared__ __attribute__((aligned(16))) float tok[4][(FULL ? 5 + TT - 1 : 2) * Q];

    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
    const int64_t hpg = a.H / a.G, sph = (a.P + 16 * PT - 1) / (16 * PT);
    const int64_t wgs = a.G * ((hpg * sph + 3) / 4);
    const int64_t wg = blockIdx.x % wgs, j = (blockIdx.x / wgs) % a.J, b = blockIdx.x / (wgs * a.J);
    const Slice sl = slice_of<PT>(a, wg, wv);
    const float A2 = a.A[sl.h] * kLog2e, Dh = FULL && a.D ? a.D[sl.h] : 0.0f;
    float *es = tok[wv], *ws = es + Q, *rt = es + 2 * Q, *sd = es + 3 * Q, *dts = es + 4 * Q,
          *cd = es + 5 * Q;

    const int64_t c0 = j * a.Kc, c1 = c0 + a.Kc < a.nc ? c0 + a.Kc : a.nc;
    f4 S[NT][PT];                               // state: rows n, columns p
    auto load_state = [&](const float *src, int64_t row) {   // (rows, H, P, N)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 16 * nt + 4 * g + i, p = 16 * pt + l;
                    S[nt][pt][i] = src && n < a.N && p < sl.cols
                                       ? src[((row * a.H + sl.h) * a.P + sl.p0 + p) * a.N + n] : 0.0f;
                }
    };
    auto store_state = [&](float *dst, int64_t row) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 16 * nt + 4 * g + i, p = 16 * pt + l;
                    if (n < a.N && p < sl.cols)
                        dst[((row * a.H + sl.h) * a.P + sl.p0 + p) * a.N + n] = S[nt][pt][i];
                }
    };
    // the state that enters the range (slot j - 1 holds it once joined)
    if (FULL && j > 0) load_state(a.hend, b * a.J + j - 1);
    else load_state(nullptr, 0);
    double ldec = 0.0;
    bool restarts = false;

    for (int64_t c = c0; c < c1; ++c) {
        const Chunk k = chunk_at(a, b, c);
        if (k.n <= 0) continue;
        if (k.first) {
            load_state(a.h0, k.row);
            restarts = true;
        }
        // ---- stage the chunk
        const E *Bg = static_cast<const E *>(a.B) + k.b * a.B_b + k.t * a.B_t + sl.g * a.N;
        stage_rows<IO, Q>(Bs, LB, Bg, a.B_t, k.n, static_cast<int>(a.N), NP, vecs & 1);
        if constexpr (FULL) {
            const E *Cg = static_cast<const E *>(a.C) + k.b * a.C_b + k.t * a.C_t + sl.g * a.N;
            stage_rows<IO, Q>(Cs, LB, Cg, a.C_t, k.n, static_cast<int>(a.N), NP, vecs & 2);
        }
        {   // each wavefront its own channels
            const E *Ug = static_cast<const E *>(a.u) + k.b * a.u_b + k.t * a.u_t + sl.h * a.P + sl.p0;
            E *Ud = Us + wv * 16 * PT;
            if (vecs & 4) {
                constexpr int V = Seg<IO>::VW, per = 16 * PT / V;
                using Vec = typename Seg<IO>::V;
                for (int i = lane; i < Q * per; i += 64) {
                    const int t = i / per, cc = (i % per) * V;
                    Vec v{};
                    if (t < k.n && cc < sl.cols) v = *reinterpret_cast<const Vec *>(Ug + t * a.u_t + cc);
                    *reinterpret_cast<Vec *>(Ud + t * LU + cc) = v;
                }
            } else {
                for (int i = lane; i < Q * 16 * PT; i += 64) {
                    const int t = i / (16 * PT), cc = i % (16 * PT);
                    Ud[t * LU + cc] = t < k.n && cc < sl.cols ? Ug[t * a.u_t + cc] : E(0);
                }
            }
        }
        // ---- step sizes and decays, a lane a token
        const float dt = lane < Q ? step_size<IO>(a, k, lane, sl.h) : 0.0f;
        const double s = lane_prefix(static_cast<double>(dt) * A2);
        const double sQ = __shfl(s, 63, 64);
        ldec += sQ;
        if (lane < Q) {
            ws[lane] = dt * exp2_d(sQ - s);
            if constexpr (FULL) es[lane] = exp2_d(s);
        }
        if constexpr (FULL) {
            double ref[TT];
            ref[0] = 0.0;
#pragma unroll
            for (int q = 1; q < TT; ++q) ref[q] = __shfl(s, 16 * q - 1, 64);
            double own = 0.0;
#pragma unroll
            for (int q = 1; q < TT; ++q) own = (lane >> 4) == q ? ref[q] : own;
            if (lane < Q) {
                rt[lane] = exp2_d(s - own);
                sd[lane] = static_cast<float>(s - own);
                dts[lane] = dt;
#pragma unroll
                for (int q = 1; q < TT; ++q)
                    cd[(q - 1) * Q + lane] = lane < 16 * q ? dt * exp2_d(ref[q] - s) : 0.0f;
            }
        }
        __syncthreads();
        if constexpr (FULL) {
            // ---- C_t . B_s, rows s, columns t, the tiles on and above the diagonal
            int id = 0;
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int r = 0; r <= q; ++r, ++id)
                    if ((id & 3) == wv) {
                        f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int m = 0; m < KN; ++m)
                            acc = M::mma(M::row(Bs + (16 * r + l) * LB + 32 * m, g),
                                         M::row(Cs + (16 * q + l) * LB + 32 * m, g), acc);
                        CB[id * 64 + lane] = acc;
                    }
            __syncthreads();
        }
        f4 Y[FULL ? TT : 1][PT];
        if constexpr (FULL) {
            // ---- what the state entering the chunk gives
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) Y[q][pt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < KN; ++m) {
                Frag hf[PT];
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) {
                    const f4 x = S[2 * m][pt], y = S[2 * m + 1][pt];
                    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                    hf[pt] = M::pack(v);
                }
#pragma unroll
                for (int q = 0; q < TT; ++q) {
                    const Frag cf = M::row_perm(Cs + (16 * q + l) * LB + 32 * m, g);
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt) Y[q][pt] = M::mma(cf, hf[pt], Y[q][pt]);
                }
            }
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                const f4 e = *reinterpret_cast<const f4 *>(es + 16 * q + 4 * g);
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) Y[q][pt] *= e;
            }
        }
        // ---- the chunk's own tokens, and the state behind it
        const float dec = exp2_d(sQ);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) S[nt][pt] *= dec;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            Frag uf[PT];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
                uf[pt] = M::col_perm(Us + 32 * m * LU + wv * 16 * PT + 16 * pt, LU, g, l);
            if constexpr (FULL) {
#pragma unroll
                for (int q = 2 * m; q < TT; ++q) {
                    // decayed products of token tiles 2m, 2m+1 with tile q
                    float v[8];
                    const float rq = rt[16 * q + l], sq = sd[16 * q + l];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 2 * m + e;
                        if (r > q) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[4 * e + i] = 0.0f;
                            continue;
                        }
                        const f4 cb = CB[(q * (q + 1) / 2 + r) * 64 + lane];
                        if (r < q) {
                            const f4 w = *reinterpret_cast<const f4 *>(cd + (q - 1) * Q + 16 * r + 4 * g);
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[4 * e + i] = cb[i] * w[i] * rq;
                        } else {
                            const f4 x = *reinterpret_cast<const f4 *>(sd + 16 * r + 4 * g);
                            const f4 d = *reinterpret_cast<const f4 *>(dts + 16 * r + 4 * g);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[4 * e + i] = 4 * g + i <= l ? cb[i] * (exp2_hw(sq - x[i]) * d[i]) : 0.0f;
                        }
                    }
                    // one rounding to the I/O type: an operand of the product, as u is
                    const Frag mf = M::pack(v);
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt) Y[q][pt] = M::mma(mf, uf[pt], Y[q][pt]);
                }
            }
            // the state's sums stay float32: the weighted u goes in as terms
            // that hold all its bits
            Frag wf[PT][M::kTerms];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
                float v[8];
                M::unpack(uf[pt], v);
                const f4 w0 = *reinterpret_cast<const f4 *>(ws + 32 * m + 4 * g);
                const f4 w1 = *reinterpret_cast<const f4 *>(ws + 32 * m + 16 + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) { v[i] *= w0[i]; v[4 + i] *= w1[i]; }
#pragma unroll
                for (int x = 0; x < M::kTerms; ++x) wf[pt][x] = M::take(v);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const Frag bf = M::col_perm(Bs + 32 * m * LB + 16 * nt, LB, g, l);
#pragma unroll
                for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                    for (int x = 0; x < M::kTerms; ++x) S[nt][pt] = M::mma(bf, wf[pt][x], S[nt][pt]);
            }
        }
        if constexpr (FULL) {
            // ---- y through the wavefront's own columns of Us
            E *Ud = Us + wv * 16 * PT;
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        E *x = Ud + (16 * q + 4 * g + i) * LU + 16 * pt + l;
                        IO::store(x, 0, __builtin_fmaf(Dh, IO::load(x, 0), Y[q][pt][i]));
                    }
            __builtin_amdgcn_wave_barrier();
            E *yg = static_cast<E *>(a.y) + ((k.b * a.L + k.t) * a.H + sl.h) * a.P + sl.p0;
            const int64_t ys = a.H * a.P;
            if (vecs & 8) {
                constexpr int V = Seg<IO>::VW, per = 16 * PT / V;
                using Vec = typename Seg<IO>::V;
                for (int i = lane; i < Q * per; i += 64) {
                    const int t = i / per, cc = (i % per) * V;
                    if (t < k.n && cc < sl.cols)
                        *reinterpret_cast<Vec *>(yg + t * ys + cc) =
                            *reinterpret_cast<const Vec *>(Ud + t * LU + cc);
                }
            } else {
                for (int i = lane; i < Q * 16 * PT; i += 64) {
                    const int t = i / (16 * PT), cc = i % (16 * PT);
                    if (t < k.n && cc < sl.cols) yg[t * ys + cc] = Ud[t * LU + cc];
                }
            }
            if (k.last && a.last) store_state(a.last, k.row);
        }
        __syncthreads();
    }
    if constexpr (!FULL) {
        store_state(a.hend, b * a.J + j);
        if (sl.cols > 0 && sl.p0 == 0 && lane == 0)
            a.ldec[(b * a.J + j) * a.H + sl.h] = restarts ? -INFINITY : static_cast<float>(ldec);
    }
}

// Joins the ranges: slot j of hend becomes the state that enters range j + 1.
__global__ __launch_bounds__(256) void heads_join_kernel(HeadsArgs a, float *hend, const float *ldec,
                                                         int reverse) {
    const int64_t per = a.P * a.N, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t h = blockIdx.y % a.H, b = blockIdx.y / a.H;
    if (i >= per) return;
    float v = 0.0f;
    for (int64_t x = 0; x < a.J; ++x) {
        const int64_t j = b * a.J + (reverse ? a.J - 1 - x : x);
        float *p = hend + (j * a.H + h) * per + i;
        const float d = ldec[j * a.H + h];
        v = d == -INFINITY ? *p : __builtin_fmaf(exp2_hw(d), v, *p);
        *p = v;
    }
}

// Packed sequences: the chunks of each, behind one another; unused ones empty.
__global__ __launch_bounds__(256) void heads_table_kernel(HeadsArgs a, HeadsEntry *table) {
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

// Sequences without a token: their last state is the one they start from (and
// the gradient of that the gradient of the last).
__global__ __launch_bounds__(256) void heads_empty_kernel(HeadsArgs a, const float *from, float *to) {
    const int64_t per = a.H * a.P * a.N;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        if (a.cu ? seq_at(a.cu, r, a.L) < seq_at(a.cu, r + 1, a.L) : a.L > 0) continue;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < per;
             i += static_cast<int64_t>(gridDim.x) * 256)
            to[r * per + i] = from ? from[r * per + i] : 0.0f;
    }
}

hipError_t launch_heads_table(const HeadsArgs &a, HeadsEntry *table, hipStream_t s) {
    hipLaunchKernelGGL(heads_table_kernel, dim3(1), dim3(256), 0, s, a, table);
    return hipGetLastError();
}

hipError_t launch_heads_join(const HeadsArgs &a, float *hend, const float *ldec, int reverse,
                             hipStream_t s) {
    hipLaunchKernelGGL(heads_join_kernel,
                       dim3(static_cast<unsigned>((a.P * a.N + 255) / 256),
                            static_cast<unsigned>(a.H * a.batch)),
                       dim3(256), 0, s, a, hend, ldec, reverse);
    return hipGetLastError();
}

hipError_t launch_heads_empty(const HeadsArgs &a, const float *from, float *to, hipStream_t s) {
    hipLaunchKernelGGL(heads_empty_kernel,
                       dim3(16, static_cast<unsigned>(a.rows < 65535 ? a.rows : 65535)), dim3(256), 0,
                       s, a, from, to);
    return hipGetLastError();
}

template <class IO, int NP, int PT, int Q>
static hipError_t fwd_go(const HeadsArgs &a, hipStream_t s) {
    const int64_t hpg = a.H / a.G, sph = (a.P + 16 * PT - 1) / (16 * PT);
    const int64_t wgs = a.G * ((hpg * sph + 3) / 4);
    const unsigned grid = static_cast<unsigned>(wgs * a.J * a.batch);
    const int vecs = (vec_rows<IO>(a.B, a.B_b, a.B_t, a.N) ? 1 : 0) |
                     (vec_rows<IO>(a.C, a.C_b, a.C_t, a.N) ? 2 : 0) |
                     (vec_rows<IO>(a.u, a.u_b, a.u_t, a.P) ? 4 : 0) |
                     (vec_rows<IO>(a.y, 0, a.H * a.P, a.P) ? 8 : 0);
    if (a.J > 1) {
        hipLaunchKernelGGL((heads_fwd_kernel<IO, NP, PT, Q, false>), dim3(grid), dim3(256), 0, s, a, vecs);
        const hipError_t e = launch_heads_join(a, a.hend, a.ldec, 0, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((heads_fwd_kernel<IO, NP, PT, Q, true>), dim3(grid), dim3(256), 0, s, a, vecs);
    return hipGetLastError();
}

template <class IO>
static hipError_t fwd_io(const HeadsArgs &a, hipStream_t s) {
    if (a.N <= 32) return fwd_go<IO, 32, 1, 64>(a, s);
    if (a.N <= 64) return fwd_go<IO, 64, 1, 64>(a, s);
    if (a.N <= 128) return fwd_go<IO, 128, 1, 64>(a, s);
    if constexpr (sizeof(typename IO::T) == 4) return fwd_go<IO, 256, 1, 32>(a, s);
    else return fwd_go<IO, 256, 1, 64>(a, s);
}

hipError_t launch_heads_fwd(const HeadsArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.last && a.rows > 0 && (a.cu || a.L == 0)) e = launch_heads_empty(a, a.h0, a.last, s);
    if (e != hipSuccess || a.L == 0 || a.batch == 0) return e;
    if (a.cu) {
        e = launch_heads_table(a, const_cast<HeadsEntry *>(a.table), s);
        if (e != hipSuccess) return e;
    }
    return a.bf16 ? fwd_io<BF16>(a, s) : fwd_io<F32>(a, s);
}

}  // namespace ssm
