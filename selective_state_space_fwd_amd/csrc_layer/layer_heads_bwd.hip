// layer_heads_bwd.hip -- gradients of the scan over heads.
//
// With gh the gradient of the state behind a chunk, s the running log decay
// in it, Lts = exp(s_t - s_s) for s <= t:
//   v_s  = sum_{t>=s} (C_t.B_s) Lts dy_t + exp(s_Q - s_s) gh B_s;  du_s = dt_s v_s + D dy_s
//   W_ts = Lts dt_s (dy_t.u_s)
//   dC_t = sum_heads( sum_{s<=t} W_ts B_s + exp(s_t) h_in^T dy_t )
//   dB_s = sum_heads( sum_{t>=s} W_ts C_t + dt_s exp(s_Q - s_s) gh^T u_s )
//   gh of the chunk before = exp(s_Q) gh + sum_t exp(s_t) dy_t (x) C_t
// The gradient E_k of a_k is the sum over all paths from a token s < k to a
// token t >= k.  With Z_ts = (C_t.B_s) W_ts, r_t = exp(s_t) dy_t.(h_in C_t),
// p_s = dt_s exp(s_Q - s_s) u_s.(gh B_s) and X = exp(s_Q) <gh, h_in>:
//   E_k = X + sum_{t>=k} r_t + sum_{s<k} p_s + sum_{t>=k} sum_{s<t} Z_ts - sum_{s>=k} sum_{t>s} Z_ts
//   ddt_s = u_s.v_s + A E_s
// and X needs no product of its own: a chunk's X plus its p is <gh, h> at its
// end, which is the next chunk's X plus that one's r.  The rounding errors of
// r and p gather along the way, and alike for all tokens behind, so they do
// not cancel in dA: every kAnchor-th chunk X is taken anew from float32 copies
// of the states.
//
// Two walks, one in each direction and both in one launch, keep the state (or
// gh) in registers and leave it at every chunk, with r and p, which go into
// dA in float32 and so are taken from the float32 state there.  Then every
// chunk is on its own: a workgroup takes a chunk of a group, loops over its
// heads, and sums dB and dC over them in registers, in a fixed order.
#include "layer_mat.h"

namespace ssm {

// Row in the permuted order out of a row kept in the natural one.
template <class IO>
__device__ __forceinline__ typename Mat<IO>::Frag row_nat(const typename IO::T *p, int g) {
    if constexpr (sizeof(typename IO::T) == 4) return Mat<IO>::row_perm(p, g);
    else return Mat<IO>::join(*reinterpret_cast<const uint2 *>(p + 4 * g),
                              *reinterpret_cast<const uint2 *>(p + 16 + 4 * g));
}

constexpr float kDirect = 0x1p-13f;

// ------------------------------------------------------------------ the walks
// DIR 0: state from u and B, dotted with C and dy.  DIR 1 (against time): gh
// from dy and C, dotted with B and u.  FULL false: only the end of a range.
template <class IO, int NP, int Q, bool FULL>
__global__ __launch_bounds__(256) void heads_walk_kernel(HeadsArgs a, int vecs) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32;
    constexpr int LB = NP + M::kPad, LU = 64 + M::kPad;
    __shared__ __attribute__((aligned(16))) E Ks[Q * LB];
    __shared__ __attribute__((aligned(16))) E Rs[FULL ? Q * LB : 8];
    __shared__ __attribute__((aligned(16))) E Xs[Q * LU];
    __shared__ __attribute__((aligned(16))) E Ys[FULL ? Q * LU : 8];
    __shared__ __attribute__((aligned(16))) float tok[4][2 * Q];

    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
    const int64_t hpg = a.H / a.G, sph = (a.P + 15) / 16, per = (hpg * sph + 3) / 4;
    const int64_t wgs = a.G * per, half = wgs * a.J * a.batch;
    const int dir = blockIdx.x >= half;
    const int64_t id = blockIdx.x - (dir ? half : 0);
    const int64_t wg = id % wgs, j = (id / wgs) % a.J, b = id / (wgs * a.J);
    const int64_t gr = wg / per, is = (wg % per) * 4 + wv;
    const bool idle = is >= hpg * sph;
    const int64_t h = gr * hpg + (idle ? 0 : is / sph);
    const int p0 = idle ? 0 : static_cast<int>(is % sph) * 16;
    const int cols = idle ? 0 : static_cast<int>(a.P - p0 < 16 ? a.P - p0 : 16);
    const float A2 = a.A[h] * kLog2e;
    float *es = tok[wv], *ws = es + Q;
    const int64_t Pr = sph * 16, slices = a.H * sph, slice = h * sph + p0 / 16;
    const int64_t chunks = a.batch * a.nc;

    f4 S[NT];
    auto load_state = [&](const float *src, int64_t row) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 16 * nt + 4 * g + i;
                S[nt][i] = src && n < a.N && l < cols
                               ? src[((row * a.H + h) * a.P + p0 + l) * a.N + n] : 0.0f;
            }
    };
    auto store_state = [&](float *dst, int64_t row) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 16 * nt + 4 * g + i;
                if (n < a.N && l < cols) dst[((row * a.H + h) * a.P + p0 + l) * a.N + n] = S[nt][i];
            }
    };
    float *hend = a.hend + (dir ? a.batch * a.J * a.H * a.P * a.N : 0);
    float *ldecs = a.ldec + (dir ? a.batch * a.J * a.H : 0);
    if (FULL && dir == 0 && j > 0) load_state(hend, b * a.J + j - 1);
    else if (FULL && dir == 1 && j + 1 < a.J) load_state(hend, b * a.J + j + 1);
    else load_state(nullptr, 0);
    double ldec = 0.0;
    bool restarts = false;

    const E *Xg = static_cast<const E *>(dir ? a.dy : a.u), *Yg = static_cast<const E *>(dir ? a.u : a.dy);
    const E *Kg = static_cast<const E *>(dir ? a.C : a.B), *Rg = static_cast<const E *>(dir ? a.B : a.C);
    const int64_t xb = dir ? a.dy_b : a.u_b, xt = dir ? a.dy_t : a.u_t;
    const int64_t yb = dir ? a.u_b : a.dy_b, yt = dir ? a.u_t : a.dy_t;
    const int64_t kb = dir ? a.C_b : a.B_b, kt = dir ? a.C_t : a.B_t;
    const int64_t rb = dir ? a.B_b : a.C_b, rt = dir ? a.B_t : a.C_t;
    // vecs: bits 0 B, 1 C, 2 u, 3 dy
    const bool vk = vecs & (dir ? 2 : 1), vr = vecs & (dir ? 1 : 2);
    const bool vx = vecs & (dir ? 8 : 4), vy = vecs & (dir ? 4 : 8);
    auto stage_own = [&](E *dst, const E *src, int64_t stride, int n, bool vec) {
        if (vec) {
            constexpr int V = Seg<IO>::VW, pieces = 16 / V;
            using Vec = typename Seg<IO>::V;
            for (int i = lane; i < Q * pieces; i += 64) {
                const int t = i / pieces, c = (i % pieces) * V;
                Vec v{};
                if (t < n && c < cols) v = *reinterpret_cast<const Vec *>(src + t * stride + c);
                *reinterpret_cast<Vec *>(dst + t * LU + c) = v;
            }
        } else {
            for (int i = lane; i < Q * 16; i += 64) {
                const int t = i >> 4, c = i & 15;
                dst[t * LU + c] = t < n && c < cols ? src[t * stride + c] : E(0);
            }
        }
    };

    const int64_t c0 = j * a.Kc, c1 = c0 + a.Kc < a.nc ? c0 + a.Kc : a.nc;
    for (int64_t x = c0; x < c1; ++x) {
        const int64_t c = dir ? c0 + c1 - 1 - x : x;
        const Chunk k = chunk_at(a, b, c);
        if (k.n <= 0) continue;
        if (dir ? k.last : k.first) {
            load_state(dir ? a.dlast : a.h0, k.row);
            restarts = true;
        }
        stage_rows<IO, Q>(Ks, LB, Kg + k.b * kb + k.t * kt + gr * a.N, kt, k.n,
                          static_cast<int>(a.N), NP, vk);
        stage_own(Xs + wv * 16, Xg + k.b * xb + k.t * xt + h * a.P + p0, xt, k.n, vx);
        if constexpr (FULL) {
            stage_rows<IO, Q>(Rs, LB, Rg + k.b * rb + k.t * rt + gr * a.N, rt, k.n,
                              static_cast<int>(a.N), NP, vr);
            stage_own(Ys + wv * 16, Yg + k.b * yb + k.t * yt + h * a.P + p0, yt, k.n, vy);
        }
        const float dt = lane < Q ? step_size<IO>(a, k, lane, h) : 0.0f;
        const double s = lane_prefix(static_cast<double>(dt) * A2);
        const double sQ = __shfl(s, 63, 64);
        const float dec = exp2_d(sQ);
        ldec += sQ;
        if (FULL && !idle && k.first) {
            // the product with the start state, where there is one
            if (sizeof(E) == 2 && dir == 1 && a.h0) {
                float v = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 16 * nt + 4 * g + i;
                        if (n < a.N && l < cols)
                            v = __builtin_fmaf(S[nt][i],
                                               a.h0[((k.row * a.H + h) * a.P + p0 + l) * a.N + n], v);
                    }
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
                if (lane == 0) a.hdot[k.row * slices + slice] = v;
            }
        } else if (FULL && sizeof(E) == 2 && !idle && c % kAnchor == 0 && dec >= kDirect) {
            f4 *to = reinterpret_cast<f4 *>(a.anchor) +
                     (((dir * a.batch + b) * a.na + c / kAnchor) * slices + slice) * NT * 64 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) to[nt * 64] = S[nt];
        }
        if (FULL && sizeof(E) == 2 && dir == 0 && !idle && p0 == 0 && lane == 0)
            a.through[(b * a.nc + c) * a.H + h] = dec;
        if (lane < Q) {
            const float up = exp2_d(s), down = exp2_d(sQ - s);
            // behind the chunk's end the staged rows are zero, whatever the weight
            ws[lane] = dir ? up : dt * down;
            es[lane] = dir ? down : up;
        }
        __syncthreads();
        if constexpr (FULL) {
            // ---- leave the state, and dot it with the other side's tokens
            E *to = static_cast<E *>(dir ? a.gout : a.hin) +
                    (((b * a.nc + c) * a.H + h) * Pr + p0 + l) * NP;
            if (!idle) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (sizeof(E) == 2)
                        *reinterpret_cast<uint2 *>(to + 16 * nt + 4 * g) =
                            make_uint2(Seg<BF16>::pk(S[nt].x, S[nt].y), Seg<BF16>::pk(S[nt].z, S[nt].w));
                    else
                        *reinterpret_cast<f4 *>(to + 16 * nt + 4 * g) = S[nt];
                }
            }
            f4 Y[TT];
#pragma unroll
            for (int q = 0; q < TT; ++q) Y[q] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < KN; ++m) {
                const f4 x0 = S[2 * m], x1 = S[2 * m + 1];
                float v[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                Frag hf[M::kTerms];
#pragma unroll
                for (int z = 0; z < M::kTerms; ++z) hf[z] = M::take(v);
#pragma unroll
                for (int q = 0; q < TT; ++q) {
                    const Frag rf = row_nat<IO>(Rs + (16 * q + l) * LB + 32 * m, g);
#pragma unroll
                    for (int z = 0; z < M::kTerms; ++z) Y[q] = M::mma(rf, hf[z], Y[q]);
                }
            }
            float total = 0.0f;
            float *rp = a.rp + ((dir * chunks + b * a.nc + c) * slices + slice) * Q;
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                const f4 e = *reinterpret_cast<const f4 *>(es + 16 * q + 4 * g);
                f4 d;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = Y[q][i] * IO::load(Ys, (16 * q + 4 * g + i) * LU + wv * 16 + l);
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o, 64);
                    d[i] = v * e[i];
                }
                if (l == 0 && !idle) *reinterpret_cast<f4 *>(rp + 16 * q + 4 * g) = d;
                if (dir == 0) total += (d.x + d.y) + (d.z + d.w);
                else {      // p_s has dt_s in it; the dot product is kept without
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        total += d[i] * __shfl(dt, 16 * q + 4 * g + i, 64);
                }
            }
            total += __shfl_xor(total, 16, 64);
            total += __shfl_xor(total, 32, 64);
            if (lane == 0 && !idle) a.rpsum[(dir * chunks + b * a.nc + c) * slices + slice] = total;
        }
        // ---- the chunk's tokens join
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= dec;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            float v[8];
            M::unpack(M::col_perm(Xs + 32 * m * LU + wv * 16, LU, g, l), v);
            const f4 w0 = *reinterpret_cast<const f4 *>(ws + 32 * m + 4 * g);
            const f4 w1 = *reinterpret_cast<const f4 *>(ws + 32 * m + 16 + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] *= w0[i]; v[4 + i] *= w1[i]; }
            Frag wf[M::kTerms];
#pragma unroll
            for (int z = 0; z < M::kTerms; ++z) wf[z] = M::take(v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const Frag kf = M::col_perm(Ks + 32 * m * LB + 16 * nt, LB, g, l);
#pragma unroll
                for (int z = 0; z < M::kTerms; ++z) S[nt] = M::mma(kf, wf[z], S[nt]);
            }
        }
        if (FULL && dir == 1 && k.first && a.dh0) store_state(a.dh0, k.row);
        __syncthreads();
    }
    if constexpr (!FULL) {
        store_state(hend, b * a.J + j);
        if (!idle && p0 == 0 && lane == 0)
            ldecs[(b * a.J + j) * a.H + h] = restarts ? -INFINITY : static_cast<float>(ldec);
    }
}

// <gh, h_in> of every kAnchor-th chunk that keeps kDirect, a wavefront a head;
// of no meaning, and not used, where a sequence begins.
__global__ __launch_bounds__(64) void heads_anchor_kernel(HeadsArgs a, int np) {
    const int64_t h = blockIdx.x % a.H, x = blockIdx.x / a.H;      // x: batch row and anchor
    const int64_t sph = (a.P + 15) / 16, per = sph * 4 * np;       // f4s of one head
    const int64_t all = a.batch * a.na * a.H * per;
    const int64_t c = x / a.na * a.nc + x % a.na * kAnchor;
    if (a.through[c * a.H + h] < kDirect) return;
    const f4 *p = reinterpret_cast<const f4 *>(a.anchor) + (x * a.H + h) * per;
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < per; i += 64) {
        const f4 q = p[i] * p[all + i];
        v += static_cast<double>((q.x + q.y) + (q.z + q.w));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if (threadIdx.x == 0) a.adot[x * a.H + h] = static_cast<float>(v);
}

// X of every chunk of one head of one batch row, a lane a chunk: itself where
// a sequence or an anchor gives <gh, h>, else from the chunk before.  Where the
// chunk keeps less than 2^-24 of its state X is below that share of <gh, h>,
// and taken as 0: the sum starts anew there.
__global__ __launch_bounds__(64) void heads_through_kernel(HeadsArgs a) {
    const int lane = threadIdx.x;
    const int64_t h = blockIdx.x, b = blockIdx.y;
    const int64_t sph = (a.P + 15) / 16, slices = a.H * sph, chunks = a.batch * a.nc;
    double before = 0.0;            // X + sum p of the chunk before the tile
    for (int64_t c0 = 0; c0 < a.nc; c0 += 64) {
        const int64_t c = c0 + lane;
        double r = 0.0, p = 0.0;
        bool stop = c >= a.nc;      // X does not come from the chunk before
        double start = 0.0;
        if (c < a.nc) {
            const Chunk k = chunk_at(a, b, c);
            if (k.n > 0) {
                const float *rs = a.rpsum + (b * a.nc + c) * slices + h * sph;
                for (int64_t i = 0; i < sph; ++i) {
                    r += rs[i];
                    p += rs[chunks * slices + i];
                }
                const double keep = a.through[(b * a.nc + c) * a.H + h];   // exp(s_Q)
                if (k.first) {
                    stop = true;
                    if (a.h0)
                        for (int64_t i = 0; i < sph; ++i) start += a.hdot[k.row * slices + h * sph + i];
                    start *= keep;
                } else if (c % kAnchor == 0 && keep >= kDirect) {
                    stop = true;
                    start = keep * a.adot[(b * a.na + c / kAnchor) * a.H + h];
                } else if (keep < 0x1p-24) {
                    stop = true;
                }
            } else {
                stop = true;
            }
        }
        // X_c = stop ? start : X_{c-1} + p_{c-1} - r_c
        double prev = __shfl_up(p, 1, 64);
        double v = stop ? start : (lane ? prev : before) - r;
        bool reset = stop;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double w = __shfl_up(v, o, 64);
            const int f = __shfl_up(static_cast<int>(reset), o, 64);
            if (lane >= o && !reset) { v += w; reset = f; }
        }
        if (c < a.nc) a.through[(b * a.nc + c) * a.H + h] = static_cast<float>(v);
        before = __shfl(v + p, 63, 64);
    }
}

// -------------------------------------------------------------- a chunk alone
template <class IO, int NP, int Q, int PS>
__global__ __launch_bounds__(256) void heads_chunk_bwd_kernel(HeadsArgs a, int vecs) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32, KP = PS / 32;
    constexpr int LB = NP + M::kPad, LU = PS + M::kPad, LW = Q + M::kPad;
    constexpr int TRI = TT * (TT + 1) / 2, OWN = (TRI + 3) / 4, NW = (NT + 3) / 4;
    constexpr int SB = Q * LB, SU = Q * LU, SH = PS * LB;
    extern __shared__ __attribute__((aligned(16))) unsigned char mem[];
    E *Bs = reinterpret_cast<E *>(mem), *Cs = Bs + SB, *Us = Cs + SB, *Ys = Us + SU,
      *Hs = Ys + SU, *Gs = Hs + SH, *Mf = Gs + SH;      // Mf: TRI x 64 lanes x 4
    f4 *CB = reinterpret_cast<f4 *>(Mf + TRI * 256);    // rows t, columns s
    float *tok = reinterpret_cast<float *>(CB + TRI * 64);
    float *es = tok, *we = tok + Q, *rt = tok + 2 * Q, *sd = tok + 3 * Q, *dts = tok + 4 * Q,
          *cx = tok + 5 * Q;                            // cx: TT - 1 rows
    float *colv = tok + (4 + TT) * Q;                   // TRI x 16 each
    float *rowz = colv + TRI * 16, *diag = rowz + TRI * 16, *diagz = diag + Q;   // Q each
    float *through = diagz + Q;                         // one a wavefront
    E *Ws = Hs;                                         // at the end: Q x LW

    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
    const int64_t chunks = a.batch * a.nc, hpg = a.H / a.G;
    const int64_t ci = blockIdx.x % chunks, rest = blockIdx.x / chunks;
    const int64_t gr = rest % a.G, hs = rest / a.G;
    const Chunk k = chunk_at(a, ci / a.nc, ci % a.nc);
    const int64_t h0 = gr * hpg + hs * a.hblk;
    const int64_t h1 = (hs + 1) * a.hblk < hpg ? h0 + a.hblk : (gr + 1) * hpg;
    if (k.n <= 0) {         // an unused chunk of a packed batch: nothing to add
        if (static_cast<int64_t>(threadIdx.x) < h1 - h0)
            for (int64_t h = h0 + threadIdx.x; h < h1; h += 256)
                for (int i = 0; i < 3; ++i) a.part[(i * chunks + ci) * a.H + h] = 0.0f;
        return;
    }
    const int64_t sph = (a.P + 15) / 16, Pr = sph * 16, slices = a.H * sph;

    stage_rows<IO, Q>(Bs, LB, static_cast<const E *>(a.B) + k.b * a.B_b + k.t * a.B_t + gr * a.N,
                      a.B_t, k.n, static_cast<int>(a.N), NP, vecs & 1);
    stage_rows<IO, Q>(Cs, LB, static_cast<const E *>(a.C) + k.b * a.C_b + k.t * a.C_t + gr * a.N,
                      a.C_t, k.n, static_cast<int>(a.N), NP, vecs & 2);
    __syncthreads();
    {   // C_t . B_s once for all heads
        int id = 0;
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
            for (int r = 0; r <= q; ++r, ++id)
                if ((id & 3) == wv) {
                    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int m = 0; m < KN; ++m)
                        acc = M::mma(M::row(Cs + (16 * q + l) * LB + 32 * m, g),
                                     M::row(Bs + (16 * r + l) * LB + 32 * m, g), acc);
                    CB[id * 64 + lane] = acc;
                }
    }
    f4 dB[TT][NW], dC[TT][NW], W[OWN];
#pragma unroll
    for (int q = 0; q < TT; ++q)
#pragma unroll
        for (int n = 0; n < NW; ++n) dB[q][n] = dC[q][n] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int o = 0; o < OWN; ++o) W[o] = f4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int64_t h = h0; h < h1; ++h) {
        const float A2 = a.A[h] * kLog2e, Dh = a.D ? a.D[h] : 0.0f;
        const float dt = lane < Q ? step_size<IO>(a, k, lane, h) : 0.0f;
        const double s = lane_prefix(static_cast<double>(dt) * A2);
        const double sQ = __shfl(s, 63, 64);
        __syncthreads();    // the head before is done with tok and Mf
        if (wv == 0) {
            double ref[TT];
            ref[0] = 0.0;
#pragma unroll
            for (int q = 1; q < TT; ++q) ref[q] = __shfl(s, 16 * q - 1, 64);
            double own = 0.0;
#pragma unroll
            for (int q = 1; q < TT; ++q) own = (lane >> 4) == q ? ref[q] : own;
            if (lane < Q) {
                es[lane] = exp2_d(s);
                we[lane] = exp2_d(sQ - s);
                rt[lane] = exp2_d(s - own);
                sd[lane] = static_cast<float>(s - own);
                dts[lane] = dt;
#pragma unroll
                for (int q = 1; q < TT; ++q)
                    cx[(q - 1) * Q + lane] = lane < 16 * q ? exp2_d(ref[q] - s) : 0.0f;
            }
        }
        // X from the staged states themselves: exact in float32; in bfloat16 its
        // error, 2^-9 of X, is the smaller one where the chunk keeps little
        const bool direct = sizeof(E) == 4 || exp2_d(sQ) < kDirect;
        float xdot = 0.0f;
        f4 DX[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o) DX[o] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        __syncthreads();
        // decay of tile (q, r) in this lane: rows t = 4g + i, column s = l
        auto decay = [&](int q, int r) {
            f4 v;
            if (r < q) {
                const float c = cx[(q - 1) * Q + 16 * r + l];
                v = *reinterpret_cast<const f4 *>(rt + 16 * q + 4 * g) * c;
            } else {
                const float x = sd[16 * r + l];
                const f4 y = *reinterpret_cast<const f4 *>(sd + 16 * q + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = l <= 4 * g + i ? exp2_hw(y[i] - x) : 0.0f;
            }
            return v;
        };
        {   // decayed products for v, as operands with k = t
            int id = 0;
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int r = 0; r <= q; ++r, ++id)
                    if ((id & 3) == wv) {
                        const f4 m = CB[id * 64 + lane] * decay(q, r);
                        if constexpr (sizeof(E) == 2)
                            *reinterpret_cast<uint2 *>(Mf + (id * 64 + lane) * 4) =
                                make_uint2(Seg<BF16>::pk(m.x, m.y), Seg<BF16>::pk(m.z, m.w));
                        else
                            *reinterpret_cast<f4 *>(Mf + (id * 64 + lane) * 4) = m;
                    }
        }
        for (int p0 = 0; p0 < a.P; p0 += PS) {
            const int pc = static_cast<int>(a.P - p0 < PS ? a.P - p0 : PS);
            if (p0) __syncthreads();
            stage_rows<IO, Q>(Us, LU, static_cast<const E *>(a.u) + k.b * a.u_b + k.t * a.u_t + h * a.P + p0,
                              a.u_t, k.n, pc, PS, vecs & 4);
            stage_rows<IO, Q>(Ys, LU, static_cast<const E *>(a.dy) + k.b * a.dy_b + k.t * a.dy_t + h * a.P + p0,
                              a.dy_t, k.n, pc, PS, vecs & 8);
            const int64_t so = ((ci * a.H + h) * Pr + p0) * NP;
            const int prow = static_cast<int>(Pr - p0 < PS ? Pr - p0 : PS);
            stage_rows<IO, PS>(Hs, LB, static_cast<const E *>(a.hin) + so, NP, prow, NP, NP, true);
            stage_rows<IO, PS>(Gs, LB, static_cast<const E *>(a.gout) + so, NP, prow, NP, NP, true);
            __syncthreads();
            if (direct) {
                constexpr int V = Seg<IO>::VW;
                for (int i = threadIdx.x; i < PS * NP / V; i += 256) {
                    const int at = i / (NP / V) * LB + i % (NP / V) * V;
                    float x[V], y[V];
                    load_vec<IO, V>(Hs + at, x);
                    load_vec<IO, V>(Gs + at, y);
#pragma unroll
                    for (int e = 0; e < V; ++e) xdot = __builtin_fmaf(x[e], y[e], xdot);
                }
            }
            {   // dy_t . u_s
                int id = 0;
#pragma unroll
                for (int q = 0; q < TT; ++q)
#pragma unroll
                    for (int r = 0; r <= q; ++r, ++id)
                        if ((id & 3) == wv) {
#pragma unroll
                            for (int m = 0; m < KP; ++m)
                                DX[id >> 2] = M::mma(M::row(Ys + (16 * q + l) * LU + 32 * m, g),
                                                     M::row(Us + (16 * r + l) * LU + 32 * m, g),
                                                     DX[id >> 2]);
                        }
            }
            f4 V[TT];
            if (16 * wv < PS) {     // du of 16 channels a wavefront
                f4 I[TT];
#pragma unroll
                for (int r = 0; r < TT; ++r) V[r] = I[r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int m = 0; m < KN; ++m) {
                    const Frag gf = M::row(Gs + (16 * wv + l) * LB + 32 * m, g);
#pragma unroll
                    for (int r = 0; r < TT; ++r)
                        I[r] = M::mma(M::row(Bs + (16 * r + l) * LB + 32 * m, g), gf, I[r]);
                }
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    const Frag yf = M::col_perm(Ys + 32 * m * LU + 16 * wv, LU, g, l);
#pragma unroll
                    for (int r = 0; r < 2 * m + 2; ++r) {
                        float v[8];
                        Frag mf;
                        const int i1 = (2 * m + 1) * (2 * m + 2) / 2 + r, i0 = 2 * m * (2 * m + 1) / 2 + r;
                        if constexpr (sizeof(E) == 2) {
                            typename Mat<BF16>::Bits bits;
                            bits.d[0] = r <= 2 * m ? *reinterpret_cast<const uint2 *>(Mf + (i0 * 64 + lane) * 4)
                                                   : make_uint2(0, 0);
                            bits.d[1] = *reinterpret_cast<const uint2 *>(Mf + (i1 * 64 + lane) * 4);
                            mf = bits.f;
                        } else {
                            const f4 hi = *reinterpret_cast<const f4 *>(Mf + (i1 * 64 + lane) * 4);
                            f4 lo = {0.0f, 0.0f, 0.0f, 0.0f};
                            if (r <= 2 * m) lo = *reinterpret_cast<const f4 *>(Mf + (i0 * 64 + lane) * 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) { v[i] = lo[i]; v[4 + i] = hi[i]; }
                            mf = M::pack(v);
                        }
                        V[r] = M::mma(mf, yf, V[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < TT; ++r) {
                    const f4 w = *reinterpret_cast<const f4 *>(we + 16 * r + 4 * g);
                    const f4 d = *reinterpret_cast<const f4 *>(dts + 16 * r + 4 * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        V[r][i] = d[i] * __builtin_fmaf(w[i], I[r][i], V[r][i]) +
                                  Dh * IO::load(Ys, (16 * r + 4 * g + i) * LU + 16 * wv + l);
                }
            }
            // what the states give dC and dB: a quarter of the columns n a wavefront
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const int nt = wv * NW + n;
                if (nt >= NT) break;
                Frag hf[KP], gf[KP];
#pragma unroll
                for (int m = 0; m < KP; ++m) {
                    hf[m] = M::col_perm(Hs + 32 * m * LB + 16 * nt, LB, g, l);
                    gf[m] = M::col_perm(Gs + 32 * m * LB + 16 * nt, LB, g, l);
                }
#pragma unroll
                for (int q = 0; q < TT; ++q) {
                    f4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
                    for (int m = 0; m < KP; ++m) {
                        x = M::mma(row_nat<IO>(Ys + (16 * q + l) * LU + 32 * m, g), hf[m], x);
                        y = M::mma(row_nat<IO>(Us + (16 * q + l) * LU + 32 * m, g), gf[m], y);
                    }
                    const f4 e = *reinterpret_cast<const f4 *>(es + 16 * q + 4 * g);
                    const f4 w = *reinterpret_cast<const f4 *>(we + 16 * q + 4 * g) *
                                 *reinterpret_cast<const f4 *>(dts + 16 * q + 4 * g);
                    dC[q][n] += e * x;
                    dB[q][n] += w * y;
                }
            }
            __syncthreads();        // u is no longer read: du goes out through its place
            if (16 * wv < PS) {
#pragma unroll
                for (int r = 0; r < TT; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        IO::store(Us, (16 * r + 4 * g + i) * LU + 16 * wv + l, V[r][i]);
            }
            __syncthreads();
            E *dug = static_cast<E *>(a.du) + ((k.b * a.L + k.t) * a.H + h) * a.P + p0;
            const int64_t ds = a.H * a.P;
            if (vecs & 16) {
                constexpr int Vw = Seg<IO>::VW, per = PS / Vw;
                using Vec = typename Seg<IO>::V;
                for (int i = threadIdx.x; i < Q * per; i += 256) {
                    const int t = i / per, c = (i % per) * Vw;
                    if (t < k.n && c < pc)
                        *reinterpret_cast<Vec *>(dug + t * ds + c) = *reinterpret_cast<const Vec *>(Us + t * LU + c);
                }
            } else {
                for (int i = threadIdx.x; i < Q * PS; i += 256) {
                    const int t = i / PS, c = i % PS;
                    if (t < k.n && c < pc) dug[t * ds + c] = Us[t * LU + c];
                }
            }
        }
        {   // sums of the decayed products over rows and columns, and W
            int id = 0;
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int r = 0; r <= q; ++r, ++id)
                    if ((id & 3) == wv) {
                        const f4 x = DX[id >> 2] * decay(q, r), z = x * CB[id * 64 + lane];
                        const float ds = dts[16 * r + l];
                        W[id >> 2] += x * ds;
                        float col = (z.x + z.y) + (z.z + z.w);
                        col += __shfl_xor(col, 16, 64);
                        col += __shfl_xor(col, 32, 64);
                        if (g == 0) colv[id * 16 + l] = col;
                        f4 row;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // the diagonal crosses no decay
                            float v = r < q || l < 4 * g + i ? z[i] * ds : 0.0f;
#pragma unroll
                            for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o, 64);
                            row[i] = v;
                            if (r == q && l == 4 * g + i) {
                                diag[16 * q + l] = DX[id >> 2][i];          // dy_t . u_t
                                diagz[16 * q + l] = z[i];                   // its share of colv
                            }
                        }
                        if (l == 0) *reinterpret_cast<f4 *>(rowz + id * 16 + 4 * g) = row;
                    }
        }
        if (direct) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) xdot += __shfl_xor(xdot, o, 64);
            if (lane == 0) through[wv] = xdot;
        }
        __syncthreads();
        if (wv == 0) {      // a lane a token
            // E without differences of long sums: of the tiles (q, r) of Z, those
            // with r < own < q count whole, those of the own row from the token
            // on, those of the own column up to it; only the tile on the
            // diagonal is a difference
            float cv = 0.0f, dd = 0.0f, r = 0.0f, p = 0.0f;
            double rows = 0.0, cols_ = 0.0, whole = 0.0;
            if (lane < Q) {
                const int own = lane >> 4, dg = own * (own + 1) / 2 + own;
                for (int q = own + 1; q < TT; ++q) {
                    const int at = q * (q + 1) / 2;
                    cv += colv[(at + own) * 16 + l];
                    for (int x = 0; x < own; ++x)
                        for (int i = 0; i < 16; i += 4) {
                            const f4 w = *reinterpret_cast<const f4 *>(rowz + (at + x) * 16 + i);
                            whole += (w.x + w.y) + (w.z + w.w);
                        }
                }
                cols_ = static_cast<double>(cv) * dt;
                for (int x = 0; x < own; ++x) rows += rowz[(own * (own + 1) / 2 + x) * 16 + l];
                rows += static_cast<double>(rowz[dg * 16 + l]) -
                        static_cast<double>(colv[dg * 16 + l] - diagz[lane]) * dt;
                cv += colv[dg * 16 + l];
                dd = diag[lane];
                const float *rp = a.rp + (ci * slices + h * sph) * Q + lane;
                for (int64_t i = 0; i < sph; ++i) {
                    r += rp[i * Q];
                    p += rp[chunks * slices * Q + i * Q];
                }
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {      // rows: from the token on; columns: up to it
                const double x = __shfl_down(rows, o, 16), y = __shfl_up(cols_, o, 16);
                if (l + o < 16) rows += x;
                if (l >= o) cols_ += y;
            }
            const double before = __shfl_up(cols_, 1, 16);
            const double pd = static_cast<double>(p) * dt;
            const double rs = lane_prefix(static_cast<double>(r)), ps = lane_prefix(pd);
            const float X = direct ? exp2_d(sQ) * ((through[0] + through[1]) + (through[2] + through[3]))
                                   : a.through[ci * a.H + h];
            const double E_ = X + (__shfl(rs, 63, 64) - rs + r) + (ps - pd) + whole + rows +
                              (l ? before : 0.0);
            const float ddt = cv + p + a.A[h] * static_cast<float>(E_);
            float dd_ = 0.0f;
            if (lane < k.n) {
                float raw = IO::load(static_cast<const E *>(a.delta) + k.b * a.dt_b + (k.t + lane) * a.dt_t, h);
                if (a.bias) raw += a.bias[h];
                dd_ = a.softplus ? ddt / (1.0f + expf(-raw)) : ddt;
                IO::store(static_cast<E *>(a.ddelta) + (k.b * a.L + k.t + lane) * a.H, h, dd_);
            }
            double sA = lane < k.n ? E_ * dt : 0.0, sD = lane < k.n ? dd : 0.0f, sb = dd_;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                sA += __shfl_xor(sA, o, 64);
                sD += __shfl_xor(sD, o, 64);
                sb += __shfl_xor(sb, o, 64);
            }
            if (lane == 0) {
                a.part[ci * a.H + h] = static_cast<float>(sA);
                a.part[(chunks + ci) * a.H + h] = static_cast<float>(sD);
                a.part[(2 * chunks + ci) * a.H + h] = static_cast<float>(sb);
            }
        }
    }
    // ---- W over all heads, as rows t by columns s; nothing above the diagonal
    __syncthreads();
    for (int i = threadIdx.x; i < Q * LW; i += 256) Ws[i] = E(0);
    __syncthreads();
    {
        int id = 0;
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
            for (int r = 0; r <= q; ++r, ++id)
                if ((id & 3) == wv) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        IO::store(Ws, (16 * q + 4 * g + i) * LW + 16 * r + l, W[id >> 2][i]);
                }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const int nt = wv * NW + n;
        if (nt >= NT) break;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            const Frag bf = M::col_perm(Bs + 32 * m * LB + 16 * nt, LB, g, l);
            const Frag cf = M::col_perm(Cs + 32 * m * LB + 16 * nt, LB, g, l);
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                dC[q][n] = M::mma(row_nat<IO>(Ws + (16 * q + l) * LW + 32 * m, g), bf, dC[q][n]);
                dB[q][n] = M::mma(M::col_perm(Ws + 32 * m * LW + 16 * q, LW, g, l), cf, dB[q][n]);
            }
        }
        const int col = 16 * nt + l;
        if (col >= a.N) continue;
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * q + 4 * g + i;
                if (t >= k.n) continue;
                const int64_t o = ((k.b * a.L + k.t + t) * a.G + gr) * a.N + col;
                if (a.hsplit > 1) {
                    const int64_t all = a.batch * a.L * a.G * a.N;
                    a.dBp[hs * all + o] = dB[q][n][i];
                    a.dCp[hs * all + o] = dC[q][n][i];
                } else {
                    IO::store(static_cast<E *>(a.dB), o, dB[q][n][i]);
                    IO::store(static_cast<E *>(a.dC), o, dC[q][n][i]);
                }
            }
    }
}

// dA, dD and ddelta_bias: the chunks' shares, added in a fixed order.
__global__ __launch_bounds__(64) void heads_sums_kernel(HeadsArgs a) {
    const int64_t h = blockIdx.x, chunks = a.batch * a.nc;
    float *out = blockIdx.y == 0 ? a.dA : blockIdx.y == 1 ? a.dD : a.dbias;
    if (!out) return;
    double v = 0.0;
    for (int64_t c = threadIdx.x; c < chunks; c += 64)
        v += a.part[(blockIdx.y * chunks + c) * a.H + h];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if (threadIdx.x == 0) out[h] = static_cast<float>(v);
}

// dB and dC: the blocks of heads, added in order.
template <class IO>
__global__ __launch_bounds__(256) void heads_blocks_kernel(HeadsArgs a) {
    using E = typename IO::T;
    const int64_t n = a.batch * a.L * a.G * a.N;
    const float *p = blockIdx.y ? a.dCp : a.dBp;
    E *out = static_cast<E *>(blockIdx.y ? a.dC : a.dB);
    int64_t end = n;
    if (a.cu) end = seq_at(a.cu, a.rows, a.L) * a.G * a.N;      // tokens behind the last sequence
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < end;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        float v = 0.0f;
        for (int64_t x = 0; x < a.hsplit; ++x) v += p[x * n + i];
        IO::store(out, i, v);
    }
}

// ------------------------------------------------------------------ launch
template <class IO, int NP, int Q, int PS>
static hipError_t bwd_go(const HeadsArgs &a, hipStream_t s) {
    using M = Mat<IO>;
    using E = typename M::E;
    constexpr int TT = Q / 16, TRI = TT * (TT + 1) / 2;
    constexpr int LB = NP + M::kPad, LU = PS + M::kPad;
    constexpr size_t lds = sizeof(E) * (2 * Q * LB + 2 * Q * LU + 2 * PS * LB + TRI * 256) +
                           16 * TRI * 64 + 4 * ((4 + TT) * Q + 2 * TRI * 16 + 2 * Q + 4);
    static_assert(lds <= 160 * 1024, "LDS of a compute unit");
    static_assert(Q * (Q + M::kPad) <= 2 * PS * LB, "W takes the states' place");
    const int64_t hpg = a.H / a.G, sph = (a.P + 15) / 16;
    const int64_t wgs = a.G * ((hpg * sph + 3) / 4), chunks = a.batch * a.nc;
    const int vecs = (vec_rows<IO>(a.B, a.B_b, a.B_t, a.N) ? 1 : 0) |
                     (vec_rows<IO>(a.C, a.C_b, a.C_t, a.N) ? 2 : 0) |
                     (vec_rows<IO>(a.u, a.u_b, a.u_t, a.P) ? 4 : 0) |
                     (vec_rows<IO>(a.dy, a.dy_b, a.dy_t, a.P) ? 8 : 0) |
                     (vec_rows<IO>(a.du, 0, a.H * a.P, a.P) ? 16 : 0);
    const unsigned walks = static_cast<unsigned>(2 * wgs * a.J * a.batch);
    if (a.J > 1) {
        hipLaunchKernelGGL((heads_walk_kernel<IO, NP, Q, false>), dim3(walks), dim3(256), 0, s, a, vecs);
        hipError_t e = launch_heads_join(a, a.hend, a.ldec, 0, s);
        if (e == hipSuccess)
            e = launch_heads_join(a, a.hend + a.batch * a.J * a.H * a.P * a.N,
                                  a.ldec + a.batch * a.J * a.H, 1, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((heads_walk_kernel<IO, NP, Q, true>), dim3(walks), dim3(256), 0, s, a, vecs);
    if constexpr (sizeof(E) == 2) {
        hipLaunchKernelGGL(heads_anchor_kernel, dim3(static_cast<unsigned>(a.batch * a.na * a.H)),
                           dim3(64), 0, s, a, NP);
        hipLaunchKernelGGL(heads_through_kernel,
                           dim3(static_cast<unsigned>(a.H), static_cast<unsigned>(a.batch)), dim3(64), 0,
                           s, a);
    }
    hipLaunchKernelGGL((heads_chunk_bwd_kernel<IO, NP, Q, PS>),
                       dim3(static_cast<unsigned>(chunks * a.G * a.hsplit)), dim3(256), lds, s, a, vecs);
    return hipGetLastError();
}

template <class IO>
static hipError_t bwd_io(const HeadsArgs &a, hipStream_t s) {
    constexpr bool f32 = sizeof(typename IO::T) == 4;
    constexpr int Q = f32 ? 32 : 64;
    hipError_t e = a.N <= 32 ? bwd_go<IO, 32, Q, 64>(a, s) : a.N <= 64 ? bwd_go<IO, 64, Q, 64>(a, s)
                   : a.N <= 128 ? bwd_go<IO, 128, Q, 64>(a, s) : bwd_go<IO, 256, 32, f32 ? 32 : 64>(a, s);
    if (e != hipSuccess) return e;
    if (a.hsplit > 1)
        hipLaunchKernelGGL((heads_blocks_kernel<IO>), dim3(1024, 2), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_heads_bwd(const HeadsArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.dh0 && a.rows > 0 && (a.cu || a.L == 0)) e = launch_heads_empty(a, a.dlast, a.dh0, s);
    if (e != hipSuccess) return e;
    if (a.L > 0 && a.batch > 0) {
        if (a.cu) {
            e = launch_heads_table(a, const_cast<HeadsEntry *>(a.table), s);
            if (e != hipSuccess) return e;
        }
        e = a.bf16 ? bwd_io<BF16>(a, s) : bwd_io<F32>(a, s);
        if (e != hipSuccess) return e;
    }
    // without a token the sums are zero
    hipLaunchKernelGGL(heads_sums_kernel, dim3(static_cast<unsigned>(a.H), 3), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace ssm
