// layer_heads_fwd.h -- the scan over heads, forward: one decay a head and token, B and C
// shared by the heads of a group, a state of head_dim x d_state a head:
//   h_t = exp(a_t) h_{t-1} + dt_t u_t (x) B_t,  a_t = dt_t A,  y_t = h_t C_t + D u_t
//
// In chunks of Q tokens, with s the running sum of a in the chunk:
//   y_t = exp(s_t) C_t h_in + sum_{s<=t} (C_t . B_s) exp(s_t - s_s) dt_s u_s + D u_t
//   h_out = exp(s_Q) h_in + sum_s exp(s_Q - s_s) dt_s u_s (x) B_s
// which are products for the matrix cores.  A workgroup of 4 wavefronts walks
// the chunks of one batch row (or a range of them); each wavefront keeps the
// state of its 16 channels in registers in float32, and the four share B, C
// and the decayed products C_t . B_s in LDS.  The next chunk is on its way in
// registers meanwhile.  So u is read and y written once and no
// state goes through memory.  Long rows with few heads are cut into ranges: a
// first launch computes each range's end state from zero, a second joins them.
//
// What bounds it: not memory (8 x 2048 x 80 heads x 64, 128 states, bfloat16:
// 368 MB in 198 us, 1.9 TB/s; 71 us at a copy's rate) and not the matrix cores
// (a quarter of the time), but the steps of a chunk behind one another: rows
// into LDS, step sizes, C . B, decays, y, state.  At 128 states three
// workgroups share a compute unit; its vector units and LDS are each busy about
// half of the time.  1 x 65536 x 32 heads, 24 ranges: pre-pass 156, join 15, walk
// 260 us.
// In float32 the products run at a sixteenth of the rate: 8 x 2048 x 80 heads,
// 963 us.
#pragma once

#include "layer_mat.h"

namespace ssm {

// Workgroups of a group of heads, and the heads of one: HW = 1, four slices of
// 16 channels of one head; HW = 4 (head_dim <= 32), the slices of the heads
// behind one another, four to a workgroup.
template <int HW>
inline int heads_wgs(const HeadsArgs &a) {
    const int64_t hpg = a.H / a.G, sph = (a.P + 15) / 16;
    return static_cast<int>(HW == 1 ? hpg * ((sph + 3) / 4) : (hpg * sph + 3) / 4);
}

// What the kernel reads of the arguments, in few scalar registers.
struct FwdK {
    const void *u, *delta, *B, *C;
    const float *A, *D, *bias, *h0;
    void *y;
    float *last, *hend, *ldec;
    const HeadsEntry *table;    // null: dense rows
    int64_t u_b, u_t, dt_b, dt_t, B_b, B_t, C_b, C_t;
    int L, H, P, N, hpg, wgs, per, sph, nc, Kc, J, softplus, wide;
};

// LDS of a chunk: about 50 KB at 128 states in bfloat16, so that three
// workgroups share a compute unit.
template <class IO, int NP, int HW, int Q, bool FULL>
struct FwdMem {
    using M = Mat<IO>;
    using E = typename M::E;
    // B and C with their columns in the permuted order; B's rows, read down
    // their columns too, 16 elements apart (45 cycles for 4 KB, against 67 at 8)
    static constexpr int LC = NP + M::kPad, LU = 64 + M::kPad;
    static constexpr int LB = NP + (sizeof(E) == 2 ? 16 : M::kPad);
    static constexpr int TT = Q / 16, TRI = TT * (TT + 1) / 2;
    static constexpr int kTok = FULL ? 6 * Q + TT * (TT - 1) / 2 * 16 : Q;
    __attribute__((aligned(16))) E B[Q * LB];
    __attribute__((aligned(16))) E C[FULL ? Q * LC : 8];
    __attribute__((aligned(16))) E U[Q * LU];
    __attribute__((aligned(16))) typename M::Half Mh[FULL ? HW * TRI * 64 : 1];
    // a head's tokens: dt exp(s_Q - s); exp(s); exp(s - r), s - r (in two floats:
    // differences of it count) and dt with r the sum before the token's tile;
    // dt exp(r_j - s) for the tiles j behind it
    __attribute__((aligned(16))) float tok[HW][kTok];
};

// Which tiles (q, r) of C_t . B_s wavefront w computes, o = 0, 1, ...; r < 0:
// none.  Four rows of tiles: the last row's first three, the third row, the
// second row, the first and the last.  Two rows: one each.
template <int TT>
__device__ __forceinline__ constexpr int deal_q(int w, int o) {
    if constexpr (TT == 2) return w == 0 ? 0 : 1;
    return w == 3 ? (o == 0 ? 0 : 3) : 3 - w;
}
template <int TT>
__device__ __forceinline__ constexpr int deal_r(int w, int o) {
    if constexpr (TT == 2) return o == 0 && w < 3 ? (w == 2 ? 1 : 0) : -1;
    return w == 3 ? (o == 0 ? 0 : o == 1 ? 3 : -1) : o <= (w == 2 ? 1 : 2) ? o : -1;
}

// Wavefronts a SIMD to hold the registers to: two (one where the LDS has no
// room for more, or above 128 states).  At 128 states in bfloat16 the kernel
// then takes 163 registers, and three workgroups fit; held to three it takes
// 135 and was slower (8 x 2048 x 80 heads: 243 against 234 us).
template <class IO, int NP, int HW, int Q, bool FULL>
constexpr int fwd_waves() {
    return NP > 128 || 2 * sizeof(FwdMem<IO, NP, HW, Q, FULL>) > 160 * 1024 ? 1 : 2;
}

// WIDE: rows of B, C, u and y in 16-byte pieces, a chunk's within 2^31 bytes,
// and the next chunk in registers; otherwise elements, staged when needed.
template <class IO, int NP, int HW, int Q, bool FULL, bool WIDE>
__global__ __launch_bounds__(256, (fwd_waves<IO, NP, HW, Q, FULL>())) void heads_fwd_kernel(FwdK a) {
    using M = Mat<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    using Mem = FwdMem<IO, NP, HW, Q, FULL>;
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    constexpr int V = Seg<IO>::VW, ES = sizeof(E);
    constexpr int NT = NP / 16, KN = NP / 32, TT = Q / 16, KS = Q / 32, OWN = TT == 2 ? 1 : 3;
    constexpr int LB = Mem::LB, LC = Mem::LC, LU = Mem::LU;
    constexpr int PB = NP / V, NB = Q * PB / 256, PU = 64 / V, NU = Q * PU / 256;
    static_assert(Q * PB % 256 == 0 && Q * PU % 256 == 0, "whole rounds of the workgroup");
    __shared__ Mem mem;

    int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, g = lane >> 4, l = lane & 15;
    const int id = static_cast<int>(by_xcd(blockIdx.x, gridDim.x));
    const int ranges = FULL ? a.J : a.J - 1;    // nobody needs the end of the last
    const int wg = id % a.wgs, j = id / a.wgs % ranges, b = id / (a.wgs * ranges);
    const int gr = wg / a.per, in = wg % a.per;
    // the slice of channels of column block w: its head (of this workgroup's,
    // hs) and first channel; a head past the group's: none
    const int sph = a.sph, pbs = (sph + 3) / 4;
    const int h0 = gr * a.hpg + (HW == 1 ? in / pbs : in * 4 / sph), hend = (gr + 1) * a.hpg;
    auto head_slot = [&](int w) { return HW == 1 ? 0 : (in * 4 + w) / sph - in * 4 / sph; };
    auto first_chan = [&](int w) { return HW == 1 ? in % pbs * 64 + 16 * w : (in * 4 + w) % sph * 16; };
    const int hs = head_slot(wv), p0 = first_chan(wv);
    const bool out = h0 + hs >= hend || p0 >= a.P;
    const int h = out ? h0 : h0 + hs, cols = out ? 0 : min(a.P - p0, 16);
    // the wavefronts of a head share its arrays
    const int mates = HW == 1 ? 4 : min(sph, 4), rank = HW == 1 ? wv : (in * 4 + wv) % sph;
    const int nh = HW == 1 ? 1 : head_slot(3) + 1;
    const double A2 = static_cast<double>(a.A[h]) * 1.4426950408889634;
    const float Dh = FULL && a.D ? a.D[h] : 0.0f, bias = a.bias ? a.bias[h] : 0.0f;
    float *ws = mem.tok[hs], *es = ws + Q, *rt = ws + 2 * Q, *sd = ws + 3 * Q, *dts = ws + 5 * Q,
          *cd = ws + 6 * Q;

    f4 S[NT];                                   // state: rows n, columns p
    // a head's state of (rows, H, P, N), through a view: 16 bytes at a time
    // where N is a multiple of 4, past the range where there is no state
    auto state_at = [&](int N, int nt, int i) -> uint32_t {
        const int n = 16 * nt + 4 * g + i;
        return n < N && l < cols ? static_cast<uint32_t>((p0 + l) * N + n) * 4 : kDrop;
    };
    auto load_state = [&](const float *src, int64_t row) {
        const Rsrc r = view(src + (row * a.H + h) * a.P * a.N, 0x7fffffff);
        int N = a.N;
        asm volatile("" : "+s"(N));             // the offsets are made here, not kept over the walk
        if ((N & 3) == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, state_at(N, nt, 0), 0, 0));
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    S[nt][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, state_at(N, nt, i), 0, 0));
        }
    };
    auto store_state = [&](float *dst, int64_t row) {
        const Rsrc r = view(dst + (row * a.H + h) * a.P * a.N, 0x7fffffff);
        int N = a.N;
        asm volatile("" : "+s"(N));             // the offsets are made here, not kept over the walk
        if ((N & 3) == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, S[nt]), r, state_at(N, nt, 0), 0, 0);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[nt][i]), r, state_at(N, nt, i), 0, 0);
        }
    };
    auto clear_state = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear_state();
    // the state that enters the range (slot j - 1 holds it once joined)
    if (FULL && j > 0) load_state(a.hend, static_cast<int64_t>(b) * a.J + j - 1);
    double ldec = 0.0;
    bool restarts = false;

    const E *Bp = static_cast<const E *>(a.B) + b * a.B_b + gr * a.N;
    const E *Cp = static_cast<const E *>(a.C) + b * a.C_b + gr * a.N;
    const E *Up = static_cast<const E *>(a.u) + b * a.u_b;
    const E *Tp = static_cast<const E *>(a.delta) + b * a.dt_b + h;
    E *Yp = static_cast<E *>(a.y) + static_cast<int64_t>(b) * a.L * a.H * a.P + h * a.P + p0;

    // ---- the next chunk on its way in registers: byte offsets of a lane's
    // first pieces in the chunk, past every range where there is no column
    u4 Br[NB], Cr[FULL ? NB : 1], Ur[NU];
    uint32_t bo = 0, co = 0, uo = 0;
    float dtr = 0.0f;
    if constexpr (WIDE) {
        const int t = tid / PB, c = tid % PB * V;
        bo = c < a.N ? static_cast<uint32_t>(t * static_cast<int>(a.B_t) + c) * ES : kDrop;
        if constexpr (FULL)
            co = c < a.N ? static_cast<uint32_t>(t * static_cast<int>(a.C_t) + c) * ES : kDrop;
        const int tu = tid / PU, cu = tid % PU * V, w = cu >> 4;
        const int hh = h0 + head_slot(w), p = first_chan(w) + (cu & 15);
        uo = hh < hend && p < a.P
                 ? static_cast<uint32_t>(tu * static_cast<int>(a.u_t) + hh * a.P + p) * ES : kDrop;
    }
    auto step = [&](const Chunk &k) {           // a lane's step size
        if (lane >= k.n) return 0.0f;
        const float v = IO::load(Tp + (k.t + lane) * a.dt_t, 0) + bias;
        return a.softplus ? softplus_exact(v) : v;
    };
    auto rows = [&](u4 *r, int n, int each, const E *from, int nt, uint32_t off, int t, int stride) {
        const Rsrc v = view(from, 0x7fffffff);
#pragma unroll
        for (int i = 0; i < n; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(v, t + i * each < nt ? off : kDrop,
                                                         i * each * stride * ES, 0);
    };
    auto fetch_c = [&](const Chunk &k) {
        if constexpr (FULL)
            rows(Cr, NB, 256 / PB, Cp + k.t * a.C_t, k.n, co, tid / PB, static_cast<int>(a.C_t));
    };
    auto fetch_bu = [&](const Chunk &k) {
        rows(Br, NB, 256 / PB, Bp + k.t * a.B_t, k.n, bo, tid / PB, static_cast<int>(a.B_t));
        rows(Ur, NU, 256 / PU, Up + k.t * a.u_t, k.n, uo, tid / PU, static_cast<int>(a.u_t));
        dtr = step(k);
    };
    auto put_c = [&]() {
        if constexpr (FULL)
#pragma unroll
            for (int i = 0; i < NB; ++i)
                M::put_perm(mem.C + (tid / PB + i * (256 / PB)) * LC, tid % PB * V, Cr[i]);
    };
    auto chunk = [&](int c) {
        Chunk k;
        if (a.table) {
            const HeadsEntry e = a.table[c];
            k.t = e.t; k.n = e.n; k.row = e.row;
            k.first = e.flags & kFirst; k.last = e.flags & kLast;
        } else {
            k.t = static_cast<int64_t>(c) * Q;
            k.n = min(a.L - static_cast<int>(k.t), Q);
            k.row = b;
            k.first = c == 0;
            k.last = c == a.nc - 1;
        }
        return k;
    };

    const int c0 = j * a.Kc, c1 = min(c0 + a.Kc, a.nc);
    Chunk next = chunk(c0);
    if constexpr (WIDE) {
        fetch_c(next);
        fetch_bu(next);
        put_c();
    }
    for (int c = c0; c < c1; ++c) {
        // addresses are made here, not kept (and spilled) over the walk
        asm volatile("" : "+v"(l), "+v"(g), "+v"(lane), "+v"(tid));
        const Chunk k = next;
        if (k.n <= 0) break;                    // unused chunks lie behind the used ones
        if (k.first) {
            if (a.h0) load_state(a.h0, k.row); else clear_state();
            restarts = true;
        }
        if (c + 1 < c1) next = chunk(c + 1); else next.n = 0;
        // ---- stage the chunk: C is in LDS since the last one's products
        float dt;
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                M::put_perm(mem.B + (tid / PB + i * (256 / PB)) * LB, tid % PB * V, Br[i]);
#pragma unroll
            for (int i = 0; i < NU; ++i)
                *reinterpret_cast<u4 *>(mem.U + (tid / PU + i * (256 / PU)) * LU + tid % PU * V) = Ur[i];
            dt = dtr;
            fetch_c(next);
        } else {
            for (int i = tid; i < Q * NP; i += 256) {
                const int t = i / NP, cc = i % NP;
                const bool in_ = t < k.n && cc < a.N;
                mem.B[t * LB + M::pos(cc)] = in_ ? Bp[(k.t + t) * a.B_t + cc] : E(0);
                if constexpr (FULL) mem.C[t * LC + M::pos(cc)] = in_ ? Cp[(k.t + t) * a.C_t + cc] : E(0);
            }
            for (int i = tid; i < Q * 64; i += 256) {
                const int t = i >> 6, w = (i & 63) >> 4, hh = h0 + head_slot(w);
                const int p = first_chan(w) + (i & 15);
                mem.U[t * LU + (i & 63)] = t < k.n && hh < hend && p < a.P
                                               ? Up[(k.t + t) * a.u_t + hh * a.P + p] : E(0);
            }
            dt = step(k);
        }
        // ---- step sizes and decays, a lane a token
        const double s = lane_prefix(dt * A2);
        const double sQ = lane_value(s, 63);
        if constexpr (!FULL) ldec += sQ;
        if (lane < Q) {
            if (rank == 0) ws[lane] = dt * exp2_d(sQ - s);
            if constexpr (FULL) {
                double ref[TT];
                ref[0] = 0.0;
#pragma unroll
                for (int q = 1; q < TT; ++q) ref[q] = lane_value(s, 16 * q - 1);
                if (rank == (1 < mates ? 1 : 0)) es[lane] = exp2_d(s);
                if (rank == (2 < mates ? 2 : 0)) {
                    double own = 0.0;
#pragma unroll
                    for (int q = 1; q < TT; ++q) own = g == q ? ref[q] : own;
                    rt[lane] = exp2_d(s - own);
                    sd[lane] = static_cast<float>(s - own);
                    sd[Q + lane] = static_cast<float>(s - own - sd[lane]);
                    dts[lane] = dt;
                }
                if (rank == mates - 1) {
#pragma unroll
                    for (int q = 1; q < TT; ++q)
                        if (g < q) cd[q * (q - 1) / 2 * 16 + lane] = dt * exp2_d(ref[q] - s);
                }
            }
        }
        __syncthreads();
        f4 Y[FULL ? TT : 1];
        if constexpr (FULL) {
            // ---- what the state entering the chunk gives, and C_t . B_s (rows s,
            // columns t) of the tiles on and above the diagonal, which are dealt
            // out to the wavefronts by rows of C, read once for both
            f4 T[OWN];
#pragma unroll
            for (int q = 0; q < TT; ++q) Y[q] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int o = 0; o < OWN; ++o) T[o] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            // one version a wavefront: which tiles are its own is known, and a
            // step's operands are read while the step before is multiplied
            auto products = [&](auto w) {
                constexpr int W = decltype(w)::value;
                Frag cf[2][TT], bf[2][OWN];
                auto read = [&](int m) {
#pragma unroll
                    for (int q = 0; q < TT; ++q)
                        cf[m & 1][q] = M::row_perm(mem.C + (16 * q + l) * LC + 32 * m, g);
#pragma unroll
                    for (int o = 0; o < OWN; ++o)
                        if (deal_r<TT>(W, o) >= 0)
                            bf[m & 1][o] = M::row_perm(mem.B + (16 * deal_r<TT>(W, o) + l) * LB + 32 * m, g);
                };
                read(0);
#pragma unroll
                for (int m = 0; m < KN; ++m) {
                    if (m + 1 < KN) read(m + 1);
                    const Frag hf = M::join(M::half(S[2 * m]), M::half(S[2 * m + 1]));
#pragma unroll
                    for (int q = 0; q < TT; ++q) Y[q] = M::mma(cf[m & 1][q], hf, Y[q]);
#pragma unroll
                    for (int o = 0; o < OWN; ++o)
                        if (deal_r<TT>(W, o) >= 0)
                            T[o] = M::mma(bf[m & 1][o], cf[m & 1][deal_q<TT>(W, o)], T[o]);
                }
            };
            if (wv == 0) products(Int<0>());
            else if (wv == 1) products(Int<1>());
            else if (wv == 2) products(Int<2>());
            else products(Int<3>());
            // ---- the products decayed, for each head of the workgroup.  One
            // rounding to the I/O type: operands of a product, as u is.
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int r = deal_r<TT>(wv, o), q = deal_q<TT>(wv, o);
                if (r < 0) continue;
#pragma unroll 1
                for (int x = 0; x < nh; ++x) {
                    const float *tk = mem.tok[HW == 1 ? 0 : x];
                    f4 v;
                    if (r < q) {
                        v = T[o] * *reinterpret_cast<const f4 *>(
                                       tk + 6 * Q + q * (q - 1) / 2 * 16 + 16 * r + 4 * g);
                        v *= tk[2 * Q + 16 * q + l];
                    } else {
                        const float y = tk[3 * Q + 16 * q + l], yl = tk[4 * Q + 16 * q + l];
                        const f4 z = *reinterpret_cast<const f4 *>(tk + 3 * Q + 16 * r + 4 * g);
                        const f4 zl = *reinterpret_cast<const f4 *>(tk + 4 * Q + 16 * r + 4 * g);
                        const f4 d = *reinterpret_cast<const f4 *>(tk + 5 * Q + 16 * r + 4 * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = 4 * g + i <= l ? T[o][i] * (exp2_hw((y - z[i]) + (yl - zl[i])) * d[i]) : 0.0f;
                    }
                    mem.Mh[((HW == 1 ? 0 : x) * Mem::TRI + q * (q + 1) / 2 + r) * 64 + lane] = M::half(v);
                }
            }
#pragma unroll
            for (int q = 0; q < TT; ++q) Y[q] *= *reinterpret_cast<const f4 *>(es + 16 * q + 4 * g);
            __syncthreads();
        }
        // ---- the chunk's own tokens, and the state behind it.  First what the
        // next chunk needs: C into its place, which nobody reads any more, and
        // B and u on their way.
        if constexpr (WIDE) {
            put_c();
            fetch_bu(next);
        }
        Frag uf[KS];
#pragma unroll
        for (int m = 0; m < KS; ++m) uf[m] = M::col_perm(mem.U + 32 * m * LU + 16 * wv, LU, g, l);
        if constexpr (FULL) {
#pragma unroll
            for (int q = 0; q < TT; ++q) {
#pragma unroll
                for (int m = 0; 2 * m <= q; ++m) {
                    const typename M::Half *mh = mem.Mh + (hs * Mem::TRI + q * (q + 1) / 2 + 2 * m) * 64 + lane;
                    Y[q] = M::mma(M::join(mh[0], 2 * m + 1 <= q ? mh[64] : M::none()), uf[m], Y[q]);
                }
            }
            // the operand's values are u where Y's rows and columns are; y goes
            // into the wavefront's own columns of U
            E *Ud = mem.U + wv * 16;
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                float v[8];
                M::unpack(uf[m], v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    IO::store(Ud, (32 * m + 16 * (e >> 2) + 4 * g + (e & 3)) * LU + l,
                              __builtin_fmaf(Dh, v[e], Y[2 * m + (e >> 2)][e & 3]));
            }
            __builtin_amdgcn_sched_barrier(0);  // Y's registers are free from here
        }
        const float dec = exp2_d(sQ);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= dec;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            // the state's sums stay float32: the weighted u goes in as terms
            // that hold all its bits
            float v[8];
            M::unpack(uf[m], v);
            const f4 w0 = *reinterpret_cast<const f4 *>(ws + 32 * m + 4 * g);
            const f4 w1 = *reinterpret_cast<const f4 *>(ws + 32 * m + 16 + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] *= w0[i]; v[4 + i] *= w1[i]; }
            Frag wf[M::kTerms];
#pragma unroll
            for (int x = 0; x < M::kTerms; ++x) wf[x] = M::take(v);
            constexpr int STEP = NT < 4 ? NT : 4;
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += STEP) {
                Frag bf[STEP];
#pragma unroll
                for (int i = 0; i < STEP; ++i)
                    bf[i] = M::template col_perm<8>(mem.B + 32 * m * LB + M::pos(16 * (n0 + i)), LB, g, l);
                // term by term: no product waits for the one before it
#pragma unroll
                for (int y = 0; y < M::kTerms; ++y)
#pragma unroll
                    for (int i = 0; i < STEP; ++i) S[n0 + i] = M::mma(bf[i], wf[y], S[n0 + i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (FULL) {
            // ---- y out
            const E *Ud = mem.U + wv * 16;
            const int ys = a.H * a.P;
            E *yg = Yp + k.t * ys;
            if constexpr (WIDE) {
                constexpr int pieces = 16 / V;
                const Rsrc ry = view(yg, 0x7fffffff);
                const int cc = lane % pieces * V;
#pragma unroll
                for (int i = 0; i < Q * pieces / 64; ++i) {
                    const int t = lane / pieces + i * (64 / pieces);
                    __builtin_amdgcn_raw_buffer_store_b128(
                        *reinterpret_cast<const u4 *>(Ud + t * LU + cc), ry,
                        t < k.n && cc < cols ? static_cast<uint32_t>(t * ys + cc) * ES : kDrop, 0, 0);
                }
            } else {
                for (int i = lane; i < Q * 16; i += 64) {
                    const int t = i >> 4, cc = i & 15;
                    if (t < k.n && cc < cols) yg[static_cast<int64_t>(t) * ys + cc] = Ud[t * LU + cc];
                }
            }
            if (k.last && a.last) store_state(a.last, k.row);
        }
        __syncthreads();
    }
    if constexpr (!FULL) {
        store_state(a.hend, static_cast<int64_t>(b) * a.J + j);
        if (!out && p0 == 0 && lane == 0)
            a.ldec[(static_cast<int64_t>(b) * a.J + j) * a.H + h] =
                restarts ? -INFINITY : static_cast<float>(ldec);
    }
}

// ------------------------------------------------------------------ launch
template <class IO, int NP, int HW, int Q, bool WIDE>
hipError_t heads_fwd_go(const HeadsArgs &a, FwdK k, hipStream_t s) {
    k.per = heads_wgs<HW>(a);
    k.wgs = static_cast<int>(a.G * k.per);
    const unsigned grid = static_cast<unsigned>(k.wgs * a.batch);     // of one range
    if (a.J > 1) {
        hipLaunchKernelGGL((heads_fwd_kernel<IO, NP, HW, Q, false, WIDE>),
                           dim3(grid * static_cast<unsigned>(a.J - 1)), dim3(256), 0, s, k);
        const hipError_t e = launch_heads_join(a, 1, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((heads_fwd_kernel<IO, NP, HW, Q, true, WIDE>),
                       dim3(grid * static_cast<unsigned>(a.J)), dim3(256), 0, s, k);
    return hipGetLastError();
}

template <class IO, int NP, int HW, int Q>
hipError_t heads_fwd_wide(const HeadsArgs &a, const FwdK &k, hipStream_t s) {
    return k.wide ? heads_fwd_go<IO, NP, HW, Q, true>(a, k, s) : heads_fwd_go<IO, NP, HW, Q, false>(a, k, s);
}

template <class IO, int HW>
hipError_t heads_fwd_np(const HeadsArgs &a, const FwdK &k, hipStream_t s) {
    if (a.N <= 32) return heads_fwd_wide<IO, 32, HW, 64>(a, k, s);
    if (a.N <= 64) return heads_fwd_wide<IO, 64, HW, 64>(a, k, s);
    if (a.N <= 128) return heads_fwd_wide<IO, 128, HW, 64>(a, k, s);
    return heads_fwd_wide<IO, 256, HW, sizeof(typename IO::T) == 4 ? 32 : 64>(a, k, s);
}

template <class IO>
hipError_t heads_fwd_io(const HeadsArgs &a, hipStream_t s) {
    FwdK k{};
    k.u = a.u; k.delta = a.delta; k.B = a.B; k.C = a.C; k.A = a.A; k.D = a.D; k.bias = a.bias;
    k.h0 = a.h0; k.y = a.y; k.last = a.last; k.hend = a.hend; k.ldec = a.ldec;
    k.table = a.cu ? a.table : nullptr;
    k.u_b = a.u_b; k.u_t = a.u_t; k.dt_b = a.dt_b; k.dt_t = a.dt_t;
    k.B_b = a.B_b; k.B_t = a.B_t; k.C_b = a.C_b; k.C_t = a.C_t;
    k.L = static_cast<int>(a.L); k.H = static_cast<int>(a.H); k.P = static_cast<int>(a.P);
    k.N = static_cast<int>(a.N); k.hpg = static_cast<int>(a.H / a.G);
    k.sph = static_cast<int>((a.P + 15) / 16); k.nc = static_cast<int>(a.nc);
    k.Kc = static_cast<int>(a.Kc); k.J = static_cast<int>(a.J); k.softplus = a.softplus;
    const int64_t far = (1LL << 31) / static_cast<int64_t>(sizeof(typename IO::T)) / 64 - 65536;
    k.wide = vec_rows<IO>(a.B, a.B_b, a.B_t, a.N) && vec_rows<IO>(a.C, a.C_b, a.C_t, a.N) &&
             vec_rows<IO>(a.u, a.u_b, a.u_t, a.P) && vec_rows<IO>(a.y, 0, a.H * a.P, a.P) &&
             a.B_t < far && a.C_t < far && a.u_t < far && a.H * a.P < far;
    // Up to 32 channels a head fill no workgroup: several heads share one (8 x
    // 2048 x 80 heads, 64 states, bfloat16: 104 against 180 us at 16 channels, 142
    // against 151 at 32); from there on a head's own arrays are the better use of
    // LDS (171 against 242 us at 64).
    return a.P > 32 ? heads_fwd_np<IO, 1>(a, k, s) : heads_fwd_np<IO, 4>(a, k, s);
}

}  // namespace ssm
