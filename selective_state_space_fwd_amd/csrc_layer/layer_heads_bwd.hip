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
// not cancel in dA: every kAnchor-th chunk X is taken anew from its states, which
// have the rest of their float32 bits beside them there.
//
// Two walks, one in each direction and both in one launch, keep the state (or
// gh) in registers and leave it at every chunk, with r and p, which go into
// dA in float32 and so are taken from the float32 state there.  Then every
// chunk is on its own: a workgroup takes a chunk of a group, loops over its
// heads, and sums dB and dC over them in registers, in a fixed order.
//
// 4 x 2048 x 80 heads x 64, 128 states, bfloat16: 526 us (walks 315, products of
// the states 51, chunks 197, decays 21, the rest 14 by a profiler's clock), against
// 50 for 263 MB at a copy's rate.  What bounds it: the states go through memory,
// 0.5 GB written by the walks and 0.67 read by the two launches behind them, about
// 220 us; that is the price of chunks that do not wait for each other, without which
// 640 walks of everything would be all the parallel work there is.  The rest is
// the steps of a chunk behind one another, as in the forward walk.  Float32 at
// the same sizes: 1280 us.
#include <type_traits>

#include "layer_mat.h"

namespace ssm {

// Sum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ float row_sum(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xf, 0xf, false));  // row_ror:1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xf, 0xf, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, false));
    return v;
}

// A bfloat16 chunk that keeps less than this of its state takes X from the
// states as they are: off by 2^-9 of X, which is 2^-22 of what came in.
constexpr float kDirect = 0x1p-13f;

// ------------------------------------------------------------------ the walks
template <class IO, int NP, int Q, bool FULL>
struct WalkMem {
    using M = Mat<IO>;
    using E = typename M::E;
    static constexpr int LB = NP + M::kPad, LU = 64 + M::kPad;
    __attribute__((aligned(16))) E K[Q * LB];               // read down its columns
    __attribute__((aligned(16))) E R[FULL ? Q * LB : 8];    // rows in the permuted order
    __attribute__((aligned(16))) E X[Q * LU];
    __attribute__((aligned(16))) E Y[FULL ? Q * LU : 8];
    __attribute__((aligned(16))) float tok[4][Q];
};

// Wavefronts a SIMD to hold the registers to, as in the forward walk (128
// states in bfloat16: 162 registers, three workgroups a compute unit).
template <class IO, int NP, int Q, bool FULL>
constexpr int walk_waves() {
    return NP > 128 || 2 * sizeof(WalkMem<IO, NP, Q, FULL>) > 160 * 1024 ? 1 : 2;
}

// DIR 0: state from u and B, dotted with C and dy.  DIR 1 (against time): gh
// from dy and C, dotted with B and u.  FULL false: only the end of a range.
// WIDE: as in the forward walk.
template <class IO, int NP, int Q, bool FULL, bool WIDE>
__global__ __launch_bounds__(256, (walk_waves<IO, NP, Q, FULL>())) void heads_walk_kernel(HeadsArgs a) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    using Mem = WalkMem<IO, NP, Q, FULL>;
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    constexpr int V = Seg<IO>::VW, ES = sizeof(E);
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32;
    constexpr int LB = Mem::LB, LU = Mem::LU;
    constexpr int PB = NP / V, NB = Q * PB / 256, PU = 64 / V, NU = Q * PU / 256;
    static_assert(Q * PB % 256 == 0 && Q * PU % 256 == 0, "whole rounds of the workgroup");
    __shared__ Mem mem;

    int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, g = lane >> 4, l = lane & 15;
    const int N = static_cast<int>(a.N), P = static_cast<int>(a.P), H = static_cast<int>(a.H);
    const int hpg = static_cast<int>(a.H / a.G), sph = (P + 15) / 16, per = (hpg * sph + 3) / 4;
    const int wgs = static_cast<int>(a.G) * per, J = static_cast<int>(a.J);
    const int ranges = FULL ? J : J - 1;    // nobody needs the end of a walk's last
    const int half = wgs * ranges * static_cast<int>(a.batch);
    const int all = static_cast<int>(by_xcd(blockIdx.x, gridDim.x));
    const int dir = all >= half, id = all - (dir ? half : 0);
    const int wg = id % wgs, j = id / wgs % ranges + (!FULL && dir), b = id / (wgs * ranges);
    const int gr = wg / per, is0 = wg % per * 4, is = is0 + wv;
    const bool idle = is >= hpg * sph;
    const int h = gr * hpg + (idle ? 0 : is / sph), p0 = idle ? 0 : is % sph * 16;
    const int cols = idle ? 0 : min(P - p0, 16);
    const double A2 = static_cast<double>(a.A[h]) * 1.4426950408889634;
    const float bias = a.bias ? a.bias[h] : 0.0f;
    float *ws = mem.tok[wv];
    const int64_t slices = a.H * sph, slice = static_cast<int64_t>(h) * sph + p0 / 16;
    // of the wavefront, in the walk's first chunk (of the row)
    const int64_t slot0 = (dir * a.batch + b) * a.nc * slices + slice;
    E *left = static_cast<E *>(dir ? a.gout : a.hin) + (b * a.nc * slices + slice) * NT * 256;
    float *rp0 = a.rp + slot0 * Q, *rpsum0 = a.rpsum + slot0;
    uint16_t *rest0 = a.rest + ((dir * a.batch + b) * a.na * slices + slice) * NT * 256;

    f4 S[NT];
    auto state_at = [&](int N_, int nt, int i) -> uint32_t {
        const int n = 16 * nt + 4 * g + i;
        return n < N_ && l < cols ? static_cast<uint32_t>((p0 + l) * N_ + n) * 4 : kDrop;
    };
    auto state_view = [&](const float *p, int64_t row) {
        return view(p + (row * H + h) * P * N, 0x7fffffff);
    };
    auto load_state = [&](f4 (&to)[NT], const float *src, int64_t row) {
        const Rsrc r = state_view(src, row);
        int N_ = N;
        asm volatile("" : "+s"(N_));            // the offsets are made here, not kept over the walk
        if ((N_ & 3) == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                to[nt] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, state_at(N_, nt, 0), 0, 0));
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    to[nt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, state_at(N_, nt, i), 0, 0));
        }
    };
    auto store_state = [&](float *dst, int64_t row) {
        const Rsrc r = state_view(dst, row);
        int N_ = N;
        asm volatile("" : "+s"(N_));
        if ((N_ & 3) == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, S[nt]), r, state_at(N_, nt, 0), 0, 0);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[nt][i]), r, state_at(N_, nt, i), 0, 0);
        }
    };
    auto clear_state = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    float *hend = a.hend + (dir ? a.batch * a.J * a.H * a.P * a.N : 0);
    float *ldecs = a.ldec + (dir ? a.batch * a.J * a.H : 0);
    clear_state();
    if (FULL && dir == 0 && j > 0) load_state(S, hend, static_cast<int64_t>(b) * J + j - 1);
    if (FULL && dir == 1 && j + 1 < J) load_state(S, hend, static_cast<int64_t>(b) * J + j + 1);
    double ldec = 0.0;
    bool restarts = false;

    // WIDE: the strides are small enough for 32 bits
    using Stride = typename std::conditional<WIDE, int, int64_t>::type;
    const Stride xt = static_cast<Stride>(dir ? a.dy_t : a.u_t), yt = static_cast<Stride>(dir ? a.u_t : a.dy_t);
    const Stride kt = static_cast<Stride>(dir ? a.C_t : a.B_t), rt = static_cast<Stride>(dir ? a.B_t : a.C_t);
    const E *Xp = static_cast<const E *>(dir ? a.dy : a.u) + b * (dir ? a.dy_b : a.u_b) + gr * hpg * P;
    const E *Yp = static_cast<const E *>(dir ? a.u : a.dy) + b * (dir ? a.u_b : a.dy_b) + gr * hpg * P;
    const E *Kp = static_cast<const E *>(dir ? a.C : a.B) + b * (dir ? a.C_b : a.B_b) + gr * N;
    const E *Rp = static_cast<const E *>(dir ? a.B : a.C) + b * (dir ? a.B_b : a.C_b) + gr * N;
    const E *Tp = static_cast<const E *>(a.delta) + b * a.dt_b + h;

    // the chunk on its way in registers, as in the forward walk.  Channels of
    // a slice past the group's: past every range
    u4 Kr[NB], Rr[FULL ? NB : 1], Xr[NU], Yr[FULL ? NU : 1];
    uint32_t ko = 0, ro = 0, xo = 0, yo = 0;
    float dtr = 0.0f;
    auto channel = [&](int c) {                 // of the group; column c of 64; -1: none
        const int i = is0 + (c >> 4), p = i % sph * 16 + (c & 15);
        return i < hpg * sph && p < P ? i / sph * P + p : -1;
    };
    if constexpr (WIDE) {
        const int t = tid / PB, c = tid % PB * V, tu = tid / PU, ch = channel(tid % PU * V);
        ko = c < N ? static_cast<uint32_t>(t * static_cast<int>(kt) + c) * ES : kDrop;
        ro = c < N ? static_cast<uint32_t>(t * static_cast<int>(rt) + c) * ES : kDrop;
        xo = ch >= 0 ? static_cast<uint32_t>(tu * static_cast<int>(xt) + ch) * ES : kDrop;
        yo = ch >= 0 ? static_cast<uint32_t>(tu * static_cast<int>(yt) + ch) * ES : kDrop;
    }
    auto rows = [&](u4 *r, int n, int each, const E *from, int nt, uint32_t off, int t, int64_t stride) {
        const Rsrc v = view(from, 0x7fffffff);
#pragma unroll
        for (int i = 0; i < n; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(v, t + i * each < nt ? off : kDrop,
                                                         i * each * static_cast<int>(stride) * ES, 0);
    };
    auto fetch_ry = [&](const Chunk &k) {
        if constexpr (FULL) {
            rows(Rr, NB, 256 / PB, Rp + k.t * rt, k.n, ro, tid / PB, rt);
            rows(Yr, NU, 256 / PU, Yp + k.t * yt, k.n, yo, tid / PU, yt);
        }
    };
    auto fetch_kx = [&](const Chunk &k) {
        rows(Kr, NB, 256 / PB, Kp + k.t * kt, k.n, ko, tid / PB, kt);
        rows(Xr, NU, 256 / PU, Xp + k.t * xt, k.n, xo, tid / PU, xt);
        dtr = 0.0f;
        if (lane < k.n) {
            const float v = IO::load(Tp + (k.t + lane) * a.dt_t, 0) + bias;
            dtr = a.softplus ? softplus_exact(v) : v;
        }
    };
    auto put_ry = [&]() {
        if constexpr (FULL) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                M::put_perm(mem.R + (tid / PB + i * (256 / PB)) * LB, tid % PB * V, Rr[i]);
#pragma unroll
            for (int i = 0; i < NU; ++i)
                *reinterpret_cast<u4 *>(mem.Y + (tid / PU + i * (256 / PU)) * LU + tid % PU * V) = Yr[i];
        }
    };
    auto plain = [&](E *to, int ld, const E *from, int64_t stride, int n, bool perm) {
        for (int i = tid; i < Q * NP; i += 256) {
            const int t = i / NP, c = i % NP;
            to[t * ld + (perm ? M::pos(c) : c)] = t < n && c < N ? from[t * stride + c] : E(0);
        }
    };
    auto plain_ch = [&](E *to, const E *from, int64_t stride, int n) {
        for (int i = tid; i < Q * 64; i += 256) {
            const int t = i >> 6, c = i & 63, ch = channel(c);
            to[t * LU + c] = t < n && ch >= 0 ? from[t * stride + ch] : E(0);
        }
    };

    const int c0 = j * static_cast<int>(a.Kc), c1 = min(c0 + static_cast<int>(a.Kc), static_cast<int>(a.nc));
    auto chunk = [&](int x) {                   // the x-th of the walk, none past its end
        Chunk k = chunk_at(a, b, dir ? c0 + c1 - 1 - x : x);
        return k;
    };
    Chunk next = chunk(c0);
    if constexpr (WIDE) {
        fetch_ry(next);
        fetch_kx(next);
        put_ry();
    }
    for (int x = c0; x < c1; ++x) {
        // addresses are made here, not kept (and spilled) over the walk
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane), "+v"(tid));
        const Chunk k = next;
        const int c = dir ? c0 + c1 - 1 - x : x;            // of the row
        if (x + 1 < c1) next = chunk(x + 1); else next.n = 0;
        if (k.n > 0 && (dir ? k.last : k.first)) {
            const ArgsAgain q = args_again();
            const float *from = dir ? q->dlast : q->h0;
            if (from) load_state(S, from, k.row); else clear_state();
            restarts = true;
        }
        float dt;
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                *reinterpret_cast<u4 *>(mem.K + (tid / PB + i * (256 / PB)) * LB + tid % PB * V) = Kr[i];
#pragma unroll
            for (int i = 0; i < NU; ++i)
                *reinterpret_cast<u4 *>(mem.X + (tid / PU + i * (256 / PU)) * LU + tid % PU * V) = Xr[i];
            dt = dtr;
            fetch_ry(next);
        } else {
            plain(mem.K, LB, Kp + k.t * kt, kt, k.n, false);
            plain_ch(mem.X, Xp + k.t * xt, xt, k.n);
            if constexpr (FULL) {
                plain(mem.R, LB, Rp + k.t * rt, rt, k.n, true);
                plain_ch(mem.Y, Yp + k.t * yt, yt, k.n);
            }
            dt = 0.0f;
            if (lane < k.n) {
                const float v = IO::load(Tp + (k.t + lane) * a.dt_t, 0) + bias;
                dt = a.softplus ? softplus_exact(v) : v;
            }
        }
        const double s = lane_prefix(dt * A2);
        const double sQ = lane_value(s, 63);
        const float dec = exp2_d(sQ);
        ldec += sQ;
        // behind the chunk's end the staged rows are zero, whatever the weight
        const float up = exp2_d(s), down = exp2_d(sQ - s);
        if (lane < Q) ws[lane] = dir ? up : dt * down;
        const float ts = dir ? dt * down : up;  // a token's share in r, p
        __syncthreads();
        if (FULL && k.n > 0) {
            // ---- leave the state: a lane's values side by side
            const Rsrc to = view(left + c * slices * (NT * 256), idle ? 0 : NT * 256 * ES);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) M::store(M::half(S[nt]), to, lane * 4 * ES, nt * 256 * ES);
            if constexpr (sizeof(E) == 2) {
                if (!idle && k.first) {
                    // X of a first chunk needs the product with the start state
                    const ArgsAgain again = args_again();
                    if (dir == 1 && again->h0) {
                        f4 h0[NT];
                        load_state(h0, again->h0, k.row);
                        float v = 0.0f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const f4 q = S[nt] * h0[nt];
                            v += (q.x + q.y) + (q.z + q.w);
                        }
#pragma unroll
                        for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
                        if (lane == 0) again->hdot[k.row * slices + slice] = v;
                    }
                } else if (!idle && c % kAnchor == 0 && dec >= kDirect) {
                    const Rsrc an = view(rest0 + c / kAnchor * slices * (NT * 256), NT * 256 * 2);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        M::store(M::rest(S[nt], M::half(S[nt])), an, lane * 8, nt * 512);
                }
                if (dir == 0 && p0 == 0 && lane == 0 && !idle)
                    a.through[(static_cast<int64_t>(b) * a.nc + c) * H + h] = dec;
            }
            // ---- and dot it with the other side's tokens: channels by tokens
            f4 Y[TT];
#pragma unroll
            for (int q = 0; q < TT; ++q) Y[q] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < KN; ++m) {
                const f4 x0 = S[2 * m], x1 = S[2 * m + 1];
                float v[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                Frag hf[M::kTerms], rf[TT];
#pragma unroll
                for (int q = 0; q < TT; ++q) rf[q] = M::row_perm(mem.R + (16 * q + l) * LB + 32 * m, g);
#pragma unroll
                for (int z = 0; z < M::kTerms; ++z) hf[z] = M::take(v);
#pragma unroll
                for (int z = 0; z < M::kTerms; ++z)
#pragma unroll
                    for (int q = 0; q < TT; ++q) Y[q] = M::mma(hf[z], rf[q], Y[q]);
            }
            float sum[TT];
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                const f4 y = M::fours(mem.Y + (16 * q + l) * LU + 16 * wv + 4 * g);
                sum[q] = __builtin_fmaf(Y[q].x, y.x, Y[q].y * y.y) + __builtin_fmaf(Y[q].z, y.z, Y[q].w * y.w);
            }
            // a lane its token's; kept without the decay (and dt) to the chunk's end
            const float own = group_sums<TT>(sum);
            if (lane < Q && !idle) rp0[c * slices * Q + lane] = own;
            if constexpr (sizeof(E) == 2) {
                float total = row_sum(lane < Q ? own * ts : 0.0f);
                total = swap16_add(total, total);
                total = swap32_add(total, total);
                if (lane == 0 && !idle) rpsum0[c * slices] = total;
            }
        }
        if constexpr (FULL && WIDE) {
            __syncthreads();
            put_ry();
        }
        if constexpr (WIDE) fetch_kx(next);
        // ---- the chunk's tokens join
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= dec;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            float v[8];
            M::unpack(M::col_perm(mem.X + 32 * m * LU + wv * 16, LU, g, l), v);
            const f4 w0 = *reinterpret_cast<const f4 *>(ws + 32 * m + 4 * g);
            const f4 w1 = *reinterpret_cast<const f4 *>(ws + 32 * m + 16 + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] *= w0[i]; v[4 + i] *= w1[i]; }
            Frag wf[M::kTerms];
#pragma unroll
            for (int z = 0; z < M::kTerms; ++z) wf[z] = M::take(v);
            constexpr int STEP = NT < 4 ? NT : 4;
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += STEP) {
                Frag kf[STEP];
#pragma unroll
                for (int i = 0; i < STEP; ++i)
                    kf[i] = M::col_perm(mem.K + 32 * m * LB + 16 * (n0 + i), LB, g, l);
#pragma unroll
                for (int z = 0; z < M::kTerms; ++z)
#pragma unroll
                    for (int i = 0; i < STEP; ++i) S[n0 + i] = M::mma(kf[i], wf[z], S[n0 + i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (FULL && dir == 1 && k.n > 0 && k.first) {
            float *dh0 = args_again()->dh0;
            if (dh0) store_state(dh0, k.row);
        }
        __syncthreads();
    }
    if constexpr (!FULL) {
        store_state(hend, static_cast<int64_t>(b) * J + j);
        if (!idle && p0 == 0 && lane == 0)
            ldecs[(static_cast<int64_t>(b) * J + j) * H + h] = restarts ? -INFINITY : static_cast<float>(ldec);
    }
}

// <gh, h_in> of every kAnchor-th chunk that keeps kDirect, a workgroup a head;
// of no meaning, and not used, where a sequence begins.  A stream: 336 MB in 51
// us (6.6 TB/s) at 4 x 2048 x 80 heads.
__global__ __launch_bounds__(256) void heads_anchor_kernel(HeadsArgs a, int np) {
    const int64_t h = blockIdx.x % a.H, x = blockIdx.x / a.H;      // x: batch row and anchor
    const int64_t sph = (a.P + 15) / 16, per = sph * 2 * np;       // 8 values of one head each
    const int64_t all = a.batch * a.na * a.H * per;
    const int64_t c = x / a.na * a.nc + x % a.na * kAnchor;
    if (a.through[c * a.H + h] < kDirect) return;
    const uint4 *s0 = static_cast<const uint4 *>(a.hin) + (c * a.H + h) * per;
    const uint4 *s1 = static_cast<const uint4 *>(a.gout) + (c * a.H + h) * per;
    const uint4 *r0 = reinterpret_cast<const uint4 *>(a.rest) + (x * a.H + h) * per;
    __shared__ double sum[4];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < per; i += 256) {
        const uint4 p = s0[i], q = s1[i], pr = r0[i], qr = r0[all + i];
        const uint32_t ps[4] = {p.x, p.y, p.z, p.w}, qs[4] = {q.x, q.y, q.z, q.w};
        const uint32_t pt[4] = {pr.x, pr.y, pr.z, pr.w}, qt[4] = {qr.x, qr.y, qr.z, qr.w};
        float w = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float p0, p1, q0, q1;
            Mat<BF16>::whole(ps[e], pt[e], p0, p1);
            Mat<BF16>::whole(qs[e], qt[e], q0, q1);
            w += __builtin_fmaf(p0, q0, p1 * q1);
        }
        v += static_cast<double>(w);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
// Eight wavefronts of up to 128 registers and 78 KB of LDS at 128 states in
// bfloat16, so that two workgroups share a compute unit and there are four
// wavefronts a SIMD to wait for LDS and memory in turn.  (Four wavefronts of 256
// registers, each with twice the sums: 285 against 211 us at 4 x 2048 x 80
// heads, most of the time waiting; the next head's data fetched ahead: 219.)
// C is needed before the heads and after them: h has its place meanwhile.  All
// rows are kept in the permuted order.
template <class IO, int NP, int Q, int PS>
struct ChunkMem {
    using M = Mat<IO>;
    using E = typename M::E;
    static constexpr int LB = NP + (sizeof(E) == 2 ? 16 : M::kPad), LU = PS + M::kPad;
    static constexpr int LW = Q + M::kPad, TT = Q / 16, TRI = TT * (TT + 1) / 2;
    static constexpr int kC = (Q > PS ? Q : PS) * LB;
    __attribute__((aligned(16))) E B[Q * LB];
    __attribute__((aligned(16))) E HC[kC];                      // h_in; C
    static constexpr int WT = sizeof(E) == 2 ? 2 : 1;           // values that hold one of W
    __attribute__((aligned(16))) E G[PS * LB > WT * Q * LW ? PS * LB : WT * Q * LW];   // gh; at last W
    __attribute__((aligned(16))) E U[Q * LU];
    __attribute__((aligned(16))) E Y[Q * LU];
    __attribute__((aligned(16))) typename M::Half Mh[TRI * 64];
    // a head's tokens: exp(s), exp(s_Q - s), exp(s - r), s - r (in two floats) and
    // dt with r the sum before the token's tile; exp(r_q - s) for the tiles q
    // behind it
    __attribute__((aligned(16))) float tok[6 * Q + TT * (TT - 1) / 2 * 16];
};

// What a chunk and head leave for heads_grad_kernel: row and column sums of Z
// by tiles (the columns' without dt), dy_t.u_t and Z_tt, and <gh, h_in>.
template <int Q>
struct GradRec {
    static constexpr int TT = Q / 16, TRI = TT * (TT + 1) / 2;
    float rowz[TRI * 16], colv[TRI * 16], diag[Q], diagz[Q], xdot[8];
};

// The row and column of tile i of a triangle's, in order of rows.
__device__ __forceinline__ int tile_q(int i) { return (i >= 1) + (i >= 3) + (i >= 6); }
__device__ __forceinline__ int tile_r(int i) { return i - tile_q(i) * (tile_q(i) + 1) / 2; }

template <class IO, int NP, int Q, int PS, bool WIDE>
__global__ __launch_bounds__(512, (sizeof(ChunkMem<IO, NP, Q, PS>) <= 80 * 1024 ? 4 : 2)) void
heads_chunk_bwd_kernel(HeadsArgs a, GradRec<Q> *rec) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    using Half = typename M::Half;
    using Mem = ChunkMem<IO, NP, Q, PS>;
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    constexpr int V = Seg<IO>::VW, ES = sizeof(E);
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32, KP = PS / 32;
    constexpr int LB = Mem::LB, LU = Mem::LU, LW = Mem::LW;
    constexpr int TRI = Mem::TRI, OWN = (TRI + 7) / 8, FOUR = M::pos(4);
    // dB and dC: NW column tiles and QR row tiles a wavefront
    constexpr int NW = NT > 8 ? NT / 8 : 1, QS = NT < 8 ? 8 / NT : 1, QR = TT > QS ? TT / QS : 1;
    // du: 16 channels and RR row tiles a wavefront
    constexpr int PT = PS / 16, RR = TT * PT > 8 ? TT * PT / 8 : 1;
    static_assert(RR <= 2, "of one operand");
    constexpr int PU = PS / V, TU = Q * PU, NU = (TU + 511) / 512;      // pieces of u (dy)
    constexpr int TS = PS * NP / V, NS = (TS + 511) / 512;              // pieces of h (gh)
    extern __shared__ __attribute__((aligned(16))) unsigned char raw[];
    Mem &mem = *reinterpret_cast<Mem *>(raw);

    int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, g = lane >> 4, l = lane & 15;
    const int N = static_cast<int>(a.N), P = static_cast<int>(a.P), H = static_cast<int>(a.H);
    const int G = static_cast<int>(a.G), hpg = H / G, sph = (P + 15) / 16;
    const int id = static_cast<int>(by_xcd(blockIdx.x, gridDim.x));
    const int hs = id % static_cast<int>(a.hsplit), gr = id / static_cast<int>(a.hsplit) % G;
    const int ci = id / static_cast<int>(a.hsplit * G);
    const Chunk k = chunk_at(a, ci / a.nc, ci % a.nc);
    if (k.n <= 0) return;           // an unused chunk of a packed batch
    const int h0 = gr * hpg + hs * static_cast<int>(a.hblk);
    const int h1 = min(h0 + static_cast<int>(a.hblk), (gr + 1) * hpg);
    const int slices = H * sph;

    const E *Bp = static_cast<const E *>(a.B) + k.b * a.B_b + k.t * a.B_t + gr * N;
    const E *Up = static_cast<const E *>(a.u) + k.b * a.u_b + k.t * a.u_t;
    const E *Yp = static_cast<const E *>(a.dy) + k.b * a.dy_b + k.t * a.dy_t;
    const E *Tp = static_cast<const E *>(a.delta) + k.b * a.dt_b + k.t * a.dt_t;
    E *Dp = static_cast<E *>(a.du) + (k.b * a.L + k.t) * a.H * a.P;

    auto put_bc = [&](E *to, const E *from, int64_t stride) {
        if constexpr (WIDE) {
            for (int i = tid; i < Q * NP / V; i += 512) {
                const int t = i / (NP / V), c = i % (NP / V) * V;
                u4 v = {0, 0, 0, 0};
                if (t < k.n && c < N) v = *reinterpret_cast<const u4 *>(from + t * stride + c);
                M::put_perm(to + t * LB, c, v);
            }
        } else {
            for (int i = tid; i < Q * NP; i += 512) {
                const int t = i / NP, c = i % NP;
                to[t * LB + M::pos(c)] = t < k.n && c < N ? from[t * stride + c] : E(0);
            }
        }
    };

    // ---- a head's tokens and states on their way in registers
    u4 Ur[NU], Yr[NU], Hr[NS], Gr[NS];
    uint32_t uo = 0, yo = 0;
    float dtr = 0.0f;
    if constexpr (WIDE) {
        const int t = tid / PU, c = tid % PU * V;
        uo = static_cast<uint32_t>(t * static_cast<int>(a.u_t) + c) * ES;
        yo = static_cast<uint32_t>(t * static_cast<int>(a.dy_t) + c) * ES;
    }
    auto fetch = [&](int h, int p0) {
        if constexpr (WIDE) {
            const Rsrc ru = view(Up + h * P + p0, 0x7fffffff), ry = view(Yp + h * P + p0, 0x7fffffff);
            const bool in = p0 + tid % PU * V < P;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const bool ok = in && tid / PU + i * (512 / PU) < k.n;
                Ur[i] = __builtin_amdgcn_raw_buffer_load_b128(ru, ok ? uo : kDrop,
                                                              i * (512 / PU) * static_cast<int>(a.u_t) * ES, 0);
                Yr[i] = __builtin_amdgcn_raw_buffer_load_b128(ry, ok ? yo : kDrop,
                                                              i * (512 / PU) * static_cast<int>(a.dy_t) * ES, 0);
            }
        }
        dtr = 0.0f;
        if (lane < k.n) {
            const float v = IO::load(Tp + lane * a.dt_t, h) + (a.bias ? a.bias[h] : 0.0f);
            dtr = a.softplus ? softplus_exact(v) : v;
        }
    };
    auto fetch_states = [&](int h, int p0) {
        // states: 16 channels behind one another, nothing past the head's last
        const int64_t at = (static_cast<int64_t>(ci) * slices + h * sph + p0 / 16) * NT * 256;
        const uint32_t bytes = static_cast<uint32_t>(min(PS / 16, sph - p0 / 16)) * NT * 256 * ES;
        const Rsrc rh = view(static_cast<const E *>(a.hin) + at, bytes);
        const Rsrc rg = view(static_cast<const E *>(a.gout) + at, bytes);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            Hr[i] = __builtin_amdgcn_raw_buffer_load_b128(rh, (tid + 512 * i) * 16, 0, 0);
            Gr[i] = __builtin_amdgcn_raw_buffer_load_b128(rg, (tid + 512 * i) * 16, 0, 0);
        }
    };
    // a piece of a state, as the walks' lanes left it, into rows of channels
    auto put_state = [&](E *to, int x, const u4 &v) {
        constexpr int LN = V / 4;               // lanes a piece
        const int sl = x / (NT * 64 / LN), nt = x / (64 / LN) % NT, ln = x % (64 / LN) * LN;
        E *at = to + (16 * sl + (ln & 15)) * LB + M::pos(16 * nt + 4 * (ln >> 4));
        Half hv[LN];
        __builtin_memcpy(hv, &v, 16);
#pragma unroll
        for (int i = 0; i < LN; ++i) *reinterpret_cast<Half *>(at + i * LB) = hv[i];
    };

    put_bc(mem.B, Bp, a.B_t);
    put_bc(mem.HC, static_cast<const E *>(a.C) + k.b * a.C_b + k.t * a.C_t + gr * N, a.C_t);
    __syncthreads();
    f4 CB[OWN], W[OWN], DX[OWN], dB[QR][NW], dC[QR][NW];
    const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int o = 0; o < OWN; ++o) W[o] = CB[o] = DX[o] = zero;
#pragma unroll
    for (int o = 0; o < OWN; ++o) {             // C_t . B_s: rows t, columns s
        const int idx = wv + 8 * o, q = tile_q(idx), r = tile_r(idx);
        if (idx >= TRI) continue;
#pragma unroll
        for (int m = 0; m < KN; ++m)
            CB[o] = M::mma(M::row_perm(mem.HC + (16 * q + l) * LB + 32 * m, g),
                           M::row_perm(mem.B + (16 * r + l) * LB + 32 * m, g), CB[o]);
    }
#pragma unroll
    for (int q = 0; q < QR; ++q)
#pragma unroll
        for (int n = 0; n < NW; ++n) dB[q][n] = dC[q][n] = zero;
    __syncthreads();                            // C gives its place to h

    float *es = mem.tok, *we = es + Q, *rt = es + 2 * Q, *sd = es + 3 * Q, *dts = es + 5 * Q, *cx = es + 6 * Q;
    const int nt0 = NT > 8 ? NW * wv : wv % NT, q0 = NT < 8 ? wv / NT * QR : 0;
    const int pc = 16 * (wv % PT), r0 = wv / PT * RR;
    float xdot = 0.0f;
    int h = h0, p0 = 0;
    while (h < h1) {
        // addresses are made here, not kept (and spilled) over the loop
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane), "+v"(tid));
        const double A2 = static_cast<double>(a.A[h]) * 1.4426950408889634;
        const float Dh = a.D ? a.D[h] : 0.0f;
        // ---- stage
        fetch(h, p0);
        fetch_states(h, p0);
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (TU % 512 != 0 && tid + 512 * i >= TU) continue;
                M::put_perm(mem.U + (tid / PU + i * (512 / PU)) * LU, tid % PU * V, Ur[i]);
                M::put_perm(mem.Y + (tid / PU + i * (512 / PU)) * LU, tid % PU * V, Yr[i]);
            }
        } else {
            for (int i = tid; i < Q * PS; i += 512) {
                const int t = i / PS, c = i % PS;
                const bool in = t < k.n && p0 + c < P;
                mem.U[t * LU + M::pos(c)] = in ? Up[t * a.u_t + h * P + p0 + c] : E(0);
                mem.Y[t * LU + M::pos(c)] = in ? Yp[t * a.dy_t + h * P + p0 + c] : E(0);
            }
        }
        const float dt = dtr;
        const double s = lane_prefix(dt * A2);
        const double sQ = lane_value(s, 63);
        // X from the staged states themselves: exact in float32; in bfloat16 its
        // error, 2^-9 of X, is the smaller one where the chunk keeps little
        const bool direct = ES == 4 || exp2_d(sQ) < kDirect;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (TS % 512 != 0 && tid + 512 * i >= TS) continue;
            put_state(mem.HC, tid + 512 * i, Hr[i]);
            put_state(mem.G, tid + 512 * i, Gr[i]);
            if (direct) {
                float x[V], y[V];
                typename Seg<IO>::V hv, gv;
                __builtin_memcpy(&hv, &Hr[i], 16);
                __builtin_memcpy(&gv, &Gr[i], 16);
                Seg<IO>::unpack(hv, x);
                Seg<IO>::unpack(gv, y);
#pragma unroll
                for (int e = 0; e < V; ++e) xdot = __builtin_fmaf(x[e], y[e], xdot);
            }
        }
        const int hn = p0 + PS < P ? h : h + 1, pn = p0 + PS < P ? p0 + PS : 0;
        const bool last = hn != h;
        if (p0 == 0 && lane < Q) {
            double ref[TT];
            ref[0] = 0.0;
#pragma unroll
            for (int q = 1; q < TT; ++q) ref[q] = lane_value(s, 16 * q - 1);
            if (wv == 0) es[lane] = exp2_d(s);
            if (wv == 1) { we[lane] = exp2_d(sQ - s); dts[lane] = dt; }
            if (wv == 2) {
                double own = 0.0;
#pragma unroll
                for (int q = 1; q < TT; ++q) own = g == q ? ref[q] : own;
                rt[lane] = exp2_d(s - own);
                sd[lane] = static_cast<float>(s - own);
                sd[Q + lane] = static_cast<float>(s - own - sd[lane]);
            }
            if (wv == 3) {
#pragma unroll
                for (int q = 1; q < TT; ++q)
                    if (g < q) cx[q * (q - 1) / 2 * 16 + lane] = exp2_d(ref[q] - s);
            }
        }
        __syncthreads();
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane));
        // ---- the wavefront's tiles: decayed products for v (k = t), dy_t . u_s
        GradRec<Q> *rc = rec + static_cast<int64_t>(ci) * H + h;
        if (p0 == 0) {
#pragma unroll
            for (int o = 0; o < OWN; ++o) DX[o] = zero;
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const int idx = wv + 8 * o, q = tile_q(idx), r = tile_r(idx);
            if (idx >= TRI) continue;
#pragma unroll
            for (int m = 0; m < KP; ++m)
                DX[o] = M::mma(M::row_perm(mem.Y + (16 * q + l) * LU + 32 * m, g),
                               M::row_perm(mem.U + (16 * r + l) * LU + 32 * m, g), DX[o]);
            if (p0 != 0 && !last) continue;
            // decay from s (column l) to t (rows 4g + i)
            f4 d;
            if (r < q) {
                d = *reinterpret_cast<const f4 *>(rt + 16 * q + 4 * g) * cx[q * (q - 1) / 2 * 16 + 16 * r + l];
            } else {
                const float x = sd[16 * r + l], xl = sd[Q + 16 * r + l];
                const f4 y = *reinterpret_cast<const f4 *>(sd + 16 * q + 4 * g);
                const f4 yl = *reinterpret_cast<const f4 *>(sd + Q + 16 * q + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d[i] = l <= 4 * g + i ? exp2_hw((y[i] - x) + (yl[i] - xl)) : 0.0f;
            }
            if (p0 == 0) mem.Mh[idx * 64 + lane] = M::half(CB[o] * d);
            if (last) {
                const f4 x = DX[o] * d, z = x * CB[o];
                const float ds = dts[16 * r + l];
                W[o] += x * ds;
                float col = (z.x + z.y) + (z.z + z.w);
                col += __shfl_xor(col, 16, 64);
                col += __shfl_xor(col, 32, 64);
                if (g == 0) rc->colv[idx * 16 + l] = col;
                f4 row;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the diagonal crosses no decay
                    row[i] = row_sum(r < q || l < 4 * g + i ? z[i] * ds : 0.0f);
                    if (r == q && l == 4 * g + i) {
                        rc->diag[16 * q + l] = DX[o][i];
                        rc->diagz[16 * q + l] = z[i];
                    }
                }
                if (l == 0) *reinterpret_cast<f4 *>(rc->rowz + idx * 16 + 4 * g) = row;
            }
        }
        if (last && direct) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) xdot += __shfl_xor(xdot, o, 64);
            if (lane == 0) rc->xdot[wv] = xdot;
        }
        if (last) xdot = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane));
        // ---- what the states give dC and dB
        if (q0 < TT) {
            Frag hf[NW][KP], gf[NW][KP];
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int m = 0; m < KP; ++m) {
                    const int at = 32 * m * LB + M::pos(16 * (nt0 + n));
                    hf[n][m] = M::template col_perm<FOUR>(mem.HC + at, LB, g, l);
                    gf[n][m] = M::template col_perm<FOUR>(mem.G + at, LB, g, l);
                }
#pragma unroll
            for (int q = 0; q < QR; ++q) {
                f4 x[NW], y[NW];
#pragma unroll
                for (int n = 0; n < NW; ++n) x[n] = y[n] = zero;
#pragma unroll
                for (int m = 0; m < KP; ++m) {
                    const Frag yr = M::row_perm(mem.Y + (16 * (q0 + q) + l) * LU + 32 * m, g);
                    const Frag ur = M::row_perm(mem.U + (16 * (q0 + q) + l) * LU + 32 * m, g);
#pragma unroll
                    for (int n = 0; n < NW; ++n) {
                        x[n] = M::mma(yr, hf[n][m], x[n]);
                        y[n] = M::mma(ur, gf[n][m], y[n]);
                    }
                }
                const f4 e = *reinterpret_cast<const f4 *>(es + 16 * (q0 + q) + 4 * g);
                const f4 w = *reinterpret_cast<const f4 *>(we + 16 * (q0 + q) + 4 * g) *
                             *reinterpret_cast<const f4 *>(dts + 16 * (q0 + q) + 4 * g);
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    dC[q][n] += e * x[n];
                    dB[q][n] += w * y[n];
                    // added here, not where the loop ends, x and y kept until then
                    asm volatile("" : "+v"(dC[q][n]), "+v"(dB[q][n]));
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane));
        // ---- du: first what gh gives
        f4 X[RR];
        if (r0 < TT) {
#pragma unroll
            for (int r = 0; r < RR; ++r) X[r] = zero;
#pragma unroll
            for (int m = 0; m < KN; ++m) {
                const Frag gf = M::row_perm(mem.G + (pc + l) * LB + 32 * m, g);
#pragma unroll
                for (int r = 0; r < RR; ++r)
                    X[r] = M::mma(M::row_perm(mem.B + (16 * (r0 + r) + l) * LB + 32 * m, g), gf, X[r]);
            }
#pragma unroll
            for (int r = 0; r < RR; ++r) X[r] *= *reinterpret_cast<const f4 *>(we + 16 * (r0 + r) + 4 * g);
        }
        __syncthreads();                        // Mh is there; nobody reads u any more
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane));
        if (r0 < TT) {
            E *Ud = mem.U + M::pos(pc) + (l >> 2) * FOUR + (l & 3);     // du in u's place
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                const Frag yf = M::template col_perm<FOUR>(mem.Y + 32 * m * LU + M::pos(pc), LU, g, l);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    const int i1 = (2 * m + 1) * (2 * m + 2) / 2 + r0 + r, i0 = 2 * m * (2 * m + 1) / 2 + r0 + r;
                    if (r0 + r > 2 * m + 1) continue;
                    Half first = M::none();
                    if (r0 + r <= 2 * m) first = mem.Mh[i0 * 64 + lane];
                    X[r] = M::mma(M::join(first, mem.Mh[i1 * 64 + lane]), yf, X[r]);
                }
            }
            // the operand's values are dy where X's rows and columns are: RR row
            // tiles are of one operand
            float y[8];
            M::unpack(M::template col_perm<FOUR>(mem.Y + 32 * (r0 / 2) * LU + M::pos(pc), LU, g, l), y);
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const f4 dq = *reinterpret_cast<const f4 *>(dts + 16 * (r0 + r) + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = y[i], y1 = y[4 + i];
                    IO::store(Ud, (16 * (r0 + r) + 4 * g + i) * LU,
                              __builtin_fmaf(dq[i], X[r][i], Dh * ((r0 + r) & 1 ? y1 : y0)));
                }
            }
            __builtin_amdgcn_wave_barrier();
            E *dug = Dp + h * P + p0 + pc;
            const int ds = H * P, left = P - p0 - pc;
            if constexpr (WIDE) {
                constexpr int pieces = 16 / V;
                const Rsrc rd = view(dug, 0x7fffffff);
                const int c = lane % pieces * V;
#pragma unroll
                for (int i = 0; i < (16 * RR * pieces + 63) / 64; ++i) {
                    const int tr = lane / pieces + i * (64 / pieces), t = 16 * r0 + tr;
                    if (16 * RR * pieces % 64 == 0 || tr < 16 * RR)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            M::template get_perm<u4>(mem.U + t * LU, pc + c), rd,
                            t < k.n && c < left ? static_cast<uint32_t>(t * ds + c) * ES : kDrop, 0, 0);
                }
            } else {
                for (int i = lane; i < 16 * RR * 16; i += 64) {
                    const int t = 16 * r0 + (i >> 4), c = i & 15;
                    if (t < k.n && c < left)
                        dug[static_cast<int64_t>(t) * ds + c] = mem.U[t * LU + M::pos(pc + c)];
                }
            }
        }
        __syncthreads();
        h = hn;
        p0 = pn;
    }
    // ---- W over all heads, rows t by columns s, nothing above the diagonal
    const ArgsAgain z = args_again();
    E *Ws = mem.G;
    for (int i = tid; i < Mem::WT * Q * LW; i += 512) Ws[i] = E(0);
    put_bc(mem.HC, static_cast<const E *>(z->C) + k.b * z->C_b + k.t * z->C_t + gr * N, z->C_t);
    __syncthreads();
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int idx = wv + 8 * o, q = tile_q(idx), r = tile_r(idx);
        if (idx >= TRI) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // in two values of 16 bits: a sum over all heads, rounded to one it
            // would add as much again to the error of dB and dC
            const int at = (16 * q + 4 * g + i) * LW + M::pos(16 * r + l);
            IO::store(Ws, at, W[o][i]);
            if constexpr (Mem::WT == 2) IO::store(Ws, Q * LW + at, W[o][i] - IO::load(Ws, at));
        }
    }
    __syncthreads();
    if (q0 >= TT) return;
#pragma unroll
    for (int n = 0; n < NW; ++n) {
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            const int at = 32 * m * LB + M::pos(16 * (nt0 + n));
            const Frag bf = M::template col_perm<FOUR>(mem.B + at, LB, g, l);
            const Frag cf = M::template col_perm<FOUR>(mem.HC + at, LB, g, l);
#pragma unroll
            for (int q = 0; q < QR; ++q)
#pragma unroll
                for (int t = 0; t < Mem::WT; ++t) {
                    const E *w = Ws + t * Q * LW;
                    dC[q][n] = M::mma(M::row_perm(w + (16 * (q0 + q) + l) * LW + 32 * m, g), bf, dC[q][n]);
                    dB[q][n] = M::mma(M::template col_perm<FOUR>(w + 32 * m * LW + M::pos(16 * (q0 + q)), LW, g, l),
                                      cf, dB[q][n]);
                }
        }
        const int col = 16 * (nt0 + n) + l;
        if (col >= N) continue;
#pragma unroll
        for (int q = 0; q < QR; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * (q0 + q) + 4 * g + i;
                if (t >= k.n) continue;
                const int64_t o = ((k.b * z->L + k.t + t) * G + gr) * N + col;
                if (z->hsplit > 1) {
                    const int64_t all = z->batch * z->L * G * N;
                    z->dBp[hs * all + o] = dB[q][n][i];
                    z->dCp[hs * all + o] = dC[q][n][i];
                } else {
                    IO::store(static_cast<E *>(z->dB), o, dB[q][n][i]);
                    IO::store(static_cast<E *>(z->dC), o, dC[q][n][i]);
                }
            }
    }
}

// E, and with it ddelta and the chunk's shares of dA, dD and ddelta_bias: a
// wavefront a head, a lane a token.  E comes without differences of long sums:
// of the tiles (q, r) of Z those with r < own < q count whole, those of the own
// row from the token on, those of the own column up to it; only the tile on
// the diagonal is a difference.  21 us at 4 x 2048 x 80 heads (28 with the loads
// one behind another): 1.8 KB a chunk and head, and single values of delta.
template <class IO, int Q>
__global__ __launch_bounds__(256) void heads_grad_kernel(HeadsArgs a, const GradRec<Q> *rec) {
    using E = typename IO::T;
    constexpr int TT = Q / 16;
    const int lane = threadIdx.x & 63, l = lane & 15, own = lane >> 4;
    const int64_t chunks = a.batch * a.nc, id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (id >= chunks * a.H) return;
    const int64_t ci = id / a.H, h = id % a.H;
    const int64_t sph = (a.P + 15) / 16, slices = a.H * sph;
    const Chunk k = chunk_at(a, ci / a.nc, ci % a.nc);
    if (k.n <= 0) {
        if (lane < 3) a.part[(lane * chunks + ci) * a.H + h] = 0.0f;
        return;
    }
    float raw = 0.0f, dt = 0.0f;
    if (lane < k.n) {
        raw = IO::load(static_cast<const E *>(a.delta) + k.b * a.dt_b + (k.t + lane) * a.dt_t, h);
        if (a.bias) raw += a.bias[h];
        dt = a.softplus ? softplus_exact(raw) : raw;
    }
    const double s = lane_prefix(static_cast<double>(dt) * a.A[h] * 1.4426950408889634);
    const double sQ = lane_value(s, 63);
    const float dec = exp2_d(sQ);
    const bool direct = sizeof(E) == 4 || dec < kDirect;
    const GradRec<Q> &rc = rec[id];
    float cv = 0.0f, dd = 0.0f, r = 0.0f, p = 0.0f;
    double rows = 0.0, cols = 0.0, whole = 0.0;
    // all loads without a branch between them; a lane's own row and column of tiles
    const bool in = lane < Q;
    float rz[TT], cz[TT], tz[TT][TT];
#pragma unroll
    for (int x = 0; x < TT; ++x) {
        rz[x] = in && x <= own ? rc.rowz[(own * (own + 1) / 2 + x) * 16 + l] : 0.0f;
        cz[x] = in && x >= own ? rc.colv[(x * (x + 1) / 2 + own) * 16 + l] : 0.0f;
#pragma unroll
        for (int y = 0; y + 1 < x; ++y) tz[x][y] = rc.rowz[(x * (x + 1) / 2 + y) * 16 + l];
    }
    const float diagz = in ? rc.diagz[lane] : 0.0f;
    if (in) {
        dd = rc.diag[lane];
        const float *rp = a.rp + (ci * slices + h * sph) * Q + lane;
#pragma unroll 4
        for (int64_t i = 0; i < sph; ++i) {
            r += rp[i * Q];
            p += rp[chunks * slices * Q + i * Q];
        }
        r *= exp2_d(s);
        p *= exp2_d(sQ - s);
    }
    float dr_ = 0.0f, dc_ = 0.0f;               // of the tile on the diagonal
#pragma unroll
    for (int x = 0; x < TT; ++x) {
        if (x < own) rows += rz[x];
        if (x > own) cv += cz[x];
        if (x == own) { dr_ = rz[x]; dc_ = cz[x]; }
#pragma unroll
        for (int y = 0; y + 1 < x; ++y) {
            const float all = row_sum(tz[x][y]);
            if (in && y < own && own < x) whole += all;
        }
    }
    cols = static_cast<double>(cv) * dt;
    rows += static_cast<double>(dr_) - static_cast<double>(dc_ - diagz) * dt;
    cv += dc_;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {      // rows: from the token on; columns: up to it
        const double x = __shfl_down(rows, o, 16), y = __shfl_up(cols, o, 16);
        if (l + o < 16) rows += x;
        if (l >= o) cols += y;
    }
    const double before = __shfl_up(cols, 1, 16);
    const double pd = static_cast<double>(p) * dt;
    const double rs = lane_prefix(static_cast<double>(r)), ps = lane_prefix(pd);
    float xdot = 0.0f;
    if (direct)
#pragma unroll
        for (int w = 0; w < 8; ++w) xdot += rc.xdot[w];
    const double X = direct ? static_cast<double>(dec) * xdot
                            : a.through[ci * a.H + h];
    const double grad = X + (lane_value(rs, 63) - rs + r) + (ps - pd) + whole + rows + (l ? before : 0.0);
    const float ddt = cv + p + a.A[h] * static_cast<float>(grad);
    float dr = 0.0f;
    if (lane < k.n) {
        dr = a.softplus ? ddt / (1.0f + expf(-raw)) : ddt;
        IO::store(static_cast<E *>(a.ddelta) + (k.b * a.L + k.t + lane) * a.H, h, dr);
    }
    double sA = lane < k.n ? grad * dt : 0.0, sD = lane < k.n ? dd : 0.0f, sb = dr;
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

// dA, dD and ddelta_bias (which 0, 1, 2): the chunks' shares, added in a fixed
// order, a wavefront a head.
__device__ __forceinline__ void sum_chunks(const HeadsArgs &a, int which, int64_t h) {
    const int64_t chunks = a.batch * a.nc;
    float *out = which == 0 ? a.dA : which == 1 ? a.dD : a.dbias;
    if (!out || h >= a.H) return;
    double v = 0.0;
    for (int64_t c = threadIdx.x & 63; c < chunks; c += 64) v += a.part[(which * chunks + c) * a.H + h];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) out[h] = static_cast<float>(v);
}

// The sums over chunks (blockIdx.y 0 .. 2), and dB and dC (3, 4): the blocks of
// heads, added in order.
template <class IO>
__global__ __launch_bounds__(256) void heads_sums_kernel(HeadsArgs a) {
    using E = typename IO::T;
    const int64_t n = a.batch * a.L * a.G * a.N;
    if (blockIdx.y < 3)
        return sum_chunks(a, blockIdx.y, static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6));
    const float *p = blockIdx.y == 4 ? a.dCp : a.dBp;
    E *out = static_cast<E *>(blockIdx.y == 4 ? a.dC : a.dB);
    int64_t end = n;
    if (a.cu) end = seq_at(a.cu, a.rows, a.L) * a.G * a.N;      // tokens behind the last sequence
    // four at a time (whole: n and end are multiples of N) where N allows it
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    if (a.N % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 8 == 0) {
        for (int64_t i = first * 4; i < end; i += step * 4) {
            f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int64_t x = 0; x < a.hsplit; ++x) v += *reinterpret_cast<const f4 *>(p + x * n + i);
            if constexpr (sizeof(E) == 2)
                *reinterpret_cast<uint2 *>(out + i) =
                    make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
            else
#pragma unroll
                for (int e = 0; e < 4; ++e) out[i + e] = v[e];
        }
        return;
    }
    for (int64_t i = first; i < end; i += step) {
        float v = 0.0f;
        for (int64_t x = 0; x < a.hsplit; ++x) v += p[x * n + i];
        IO::store(out, i, v);
    }
}

// ------------------------------------------------------------------ launch
template <class IO, int NP, int Q, int PS, bool WIDE>
static hipError_t bwd_go(const HeadsArgs &a, hipStream_t s) {
    using E = typename IO::T;
    constexpr size_t lds = sizeof(ChunkMem<IO, NP, Q, PS>);
    static_assert(lds <= 160 * 1024, "LDS of a compute unit");
    static_assert(sizeof(GradRec<Q>) <= kGradRec, "workspace of a chunk and head");
    const int64_t hpg = a.H / a.G, sph = (a.P + 15) / 16;
    const int64_t wgs = a.G * ((hpg * sph + 3) / 4), chunks = a.batch * a.nc;
    const unsigned walks = static_cast<unsigned>(2 * wgs * a.batch);     // of one range
    GradRec<Q> *rec = reinterpret_cast<GradRec<Q> *>(a.rec);
    if (a.J > 1) {
        hipLaunchKernelGGL((heads_walk_kernel<IO, NP, Q, false, WIDE>),
                           dim3(walks * static_cast<unsigned>(a.J - 1)), dim3(256), 0, s, a);
        const hipError_t e = launch_heads_join(a, 2, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((heads_walk_kernel<IO, NP, Q, true, WIDE>),
                       dim3(walks * static_cast<unsigned>(a.J)), dim3(256), 0, s, a);
    if constexpr (sizeof(E) == 2) {
        hipLaunchKernelGGL(heads_anchor_kernel, dim3(static_cast<unsigned>(a.batch * a.na * a.H)),
                           dim3(256), 0, s, a, NP);
        hipLaunchKernelGGL(heads_through_kernel,
                           dim3(static_cast<unsigned>(a.H), static_cast<unsigned>(a.batch)), dim3(64), 0,
                           s, a);
    }
    hipLaunchKernelGGL((heads_chunk_bwd_kernel<IO, NP, Q, PS, WIDE>),
                       dim3(static_cast<unsigned>(chunks * a.G * a.hsplit)), dim3(512), lds, s, a, rec);
    hipLaunchKernelGGL((heads_grad_kernel<IO, Q>), dim3(static_cast<unsigned>((chunks * a.H + 3) / 4)),
                       dim3(256), 0, s, a, rec);
    return hipGetLastError();
}

template <class IO, int NP, int Q, int PS>
static hipError_t bwd_wide(const HeadsArgs &a, hipStream_t s) {
    const int64_t far = (1LL << 31) / static_cast<int64_t>(sizeof(typename IO::T)) / 64 - 65536;
    const bool wide = vec_rows<IO>(a.B, a.B_b, a.B_t, a.N) && vec_rows<IO>(a.C, a.C_b, a.C_t, a.N) &&
                      vec_rows<IO>(a.u, a.u_b, a.u_t, a.P) && vec_rows<IO>(a.dy, a.dy_b, a.dy_t, a.P) &&
                      vec_rows<IO>(a.du, 0, a.H * a.P, a.P) && a.B_t < far && a.C_t < far &&
                      a.u_t < far && a.dy_t < far && a.H * a.P < far;
    return wide ? bwd_go<IO, NP, Q, PS, true>(a, s) : bwd_go<IO, NP, Q, PS, false>(a, s);
}

template <class IO>
static hipError_t bwd_io(const HeadsArgs &a, hipStream_t s) {
    constexpr bool f32 = sizeof(typename IO::T) == 4;
    constexpr int Q = f32 ? 32 : 64;
    return a.N <= 32 ? bwd_wide<IO, 32, Q, 64>(a, s) : a.N <= 64 ? bwd_wide<IO, 64, Q, 64>(a, s)
           : a.N <= 128 ? bwd_wide<IO, 128, Q, 64>(a, s) : bwd_wide<IO, 256, 32, f32 ? 32 : 64>(a, s);
}

template <class IO>
static hipError_t sums_io(const HeadsArgs &a, hipStream_t s) {
    const bool blocks = a.hsplit > 1 && a.L > 0 && a.batch > 0;
    const unsigned heads = static_cast<unsigned>((a.H + 3) / 4);
    hipLaunchKernelGGL((heads_sums_kernel<IO>), dim3(blocks && heads < 1024 ? 1024 : heads, blocks ? 5 : 3),
                       dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_heads_bwd(const HeadsArgs &a, hipStream_t s) {
    hipError_t e = launch_heads_rows(a, a.dlast, a.dh0, s);
    if (e != hipSuccess) return e;
    if (a.L > 0 && a.batch > 0) {
        e = a.bf16 ? bwd_io<BF16>(a, s) : bwd_io<F32>(a, s);
        if (e != hipSuccess) return e;
    }
    // without a token the sums are zero
    return a.bf16 ? sums_io<BF16>(a, s) : sums_io<F32>(a, s);
}

}  // namespace ssm
