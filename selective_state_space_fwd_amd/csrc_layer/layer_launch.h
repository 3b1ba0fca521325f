// layer_launch.h -- argument blocks and launchers of the layer operators: the
// scan over heads, the short convolution and the root-mean-square norm.
// Built and validated by layer_api.hip; strides are in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

struct ConvArgs {
    int64_t batch, L, C;        // tokens per batch row, channels
    int W;                      // taps, 1..4
    int bf16, silu;
    const void *x, *dy;
    int64_t x_batch, x_token;   // strides of x
    int64_t dy_batch, dy_token; // strides of dy
    const float *weight;        // (C, W), column W-1 on the current token
    const float *bias;          // (C) or null
    const float *state;         // (rows, C, W-1) inputs before each sequence, or null
    const int32_t *cu;          // packed: n_seqs + 1 offsets (batch == 1), or null
    int64_t rows;               // batch, or n_seqs when packed
    void *y;                    // (batch, L, C)
    float *last;                // (rows, C, W-1) or null
    // backward
    void *dx;                   // (batch, L, C) io type
    float *dweight, *dbias;     // (C, W), (C)
    float *dstate;              // (rows, C, W-1) or null
    float *part;                // workspace: (runs, W + 1, C)
    int64_t runs, run;          // a batch row's run of `run` tokens leaves one partial row
    // single token
    float *slot_state;          // (n_slots, C, W-1)
    const int32_t *slots;       // (batch) or null: row i is slot i
    int64_t n_slots;
};
hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_update(const ConvArgs &a, hipStream_t s);

struct NormArgs {
    int64_t rows, d, group;     // group divides d
    int bf16;                   // x, z, y, dy, dz
    int res_bf16;               // residual, residual_out; backward: x, dresidual, dx
    float eps;
    const void *x, *z, *residual, *dy, *dresidual;
    int64_t x_row, z_row, res_row, dy_row;   // row strides
    const float *weight;        // (d)
    void *y;                    // (rows, d): io type, or 8-bit e4m3 when block > 0
    void *residual_out;         // (rows, d)
    int64_t block;              // 8-bit output: values that share a scale, 0: none
    float *scale;               // (rows, blocks of a row)
    // backward
    void *dx, *dz;
    float *dweight, *part;      // part: (nblk, d)
    int64_t nblk;
};
constexpr int64_t kNormMaxGroup = 16384;
int64_t norm_bwd_blocks(int64_t rows, int64_t d, int64_t group);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t s);

// Every kAnchor-th chunk of the backward has its states in all 32 bits (bfloat16).
// At 4 x 2048 x 80 heads dA is off by 3e-7 of its norm with 2; with 4 by 1.4e-6
// for 50 us of 570 less, and a sharper head's up to 3e-6 with 8.
constexpr int kAnchor = 2;
// Bytes that a chunk's products leave for the gradient of its decays.
constexpr int kGradRec = 1824;

// One chunk of the scan over heads: tokens t .. t + n - 1 of sequence `row`.
struct HeadsEntry {
    int32_t t, n, row, flags;   // flags: kFirst, kLast chunk of its sequence
};
constexpr int kFirst = 1, kLast = 2;

struct HeadsArgs {
    int64_t batch, L, H, P, G, N;
    int bf16, softplus;
    const void *u, *delta, *B, *C, *dy;
    int64_t u_b, u_t, dt_b, dt_t, B_b, B_t, C_b, C_t, dy_b, dy_t;   // strides
    const float *A, *D, *bias, *h0, *dlast;
    const int32_t *cu;
    int64_t rows;               // batch, or n_seqs when packed
    void *y;                    // (batch, L, H, P)
    float *last;                // (rows, H, P, N) or null
    // backward outputs
    void *du, *ddelta, *dB, *dC;    // (batch, L, ...) io type, dense
    float *dA, *dD, *dbias, *dh0;
    // plan: chunks of Q tokens, nc of them per batch row (packed: at most nc in
    // all), walked in ranges of Kc by J workgroups one behind the other
    int Q;
    int64_t nc, Kc, J;
    // workspace views
    const HeadsEntry *table;    // packed: nc chunks, unused ones with n = 0
    float *hend;                // (2, batch, J, H, P, N) state that enters a range; second: its gradient
    float *ldec;                // (2, batch, J, H) log2 decay of a range, kReset: the range restarts
    void *hin, *gout;           // (batch nc, H, Pr, Np) io type, P and N padded, in the order of
                                // the walks' lanes: states that enter
                                // the chunks, gradients of those that leave them
    float *rp;                  // (2, batch nc, H slices, Q) dot products across chunks, see layer_heads_bwd.hip
    float *rpsum;               // (2, batch nc, H slices) their sums over a chunk's tokens
    float *hdot;                // (rows, H slices) <gradient leaving a first chunk, start state>
    uint16_t *rest;             // (2, batch, na, H slices, 16 Np) low halves of every kAnchor-th
                                // chunk's states (bfloat16 I/O; hin and gout hold the high ones)
    float *adot;                // (batch, na, H) their products
    int64_t na;
    float *through;             // (batch nc, H) exp(s_Q) <gout, hin>
    void *rec;                  // (batch nc, H) sums over the products of a chunk, kGradRec bytes each
    float *part;                // (3, batch nc, H) dA, dD, ddelta_bias of a chunk
    int64_t hsplit, hblk;       // backward: blocks of hblk heads of a group
    float *dBp, *dCp;           // (hsplit, batch, L, G, N) float32 when hsplit > 1
    // single token
    float *state;               // (n_slots, H, P, N)
    const int32_t *slots;
    int64_t n_slots;
};
// Tokens of a chunk in the backward, padded states, and the workspace's sizes.
constexpr int heads_np(int64_t N) { return N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256; }
constexpr int heads_fwd_chunk(int bf16, int64_t N) { return !bf16 && N > 128 ? 32 : 64; }
constexpr int heads_bwd_chunk(int bf16, int64_t N) { return !bf16 || N > 128 ? 32 : 64; }
hipError_t launch_heads_join(const HeadsArgs &a, int walks, hipStream_t s);
hipError_t launch_heads_rows(const HeadsArgs &a, const float *from, float *to, hipStream_t s);
hipError_t launch_heads_fwd(const HeadsArgs &a, hipStream_t s);
hipError_t launch_heads_bwd(const HeadsArgs &a, hipStream_t s);
hipError_t launch_heads_update(const HeadsArgs &a, hipStream_t s);

}  // namespace ssm
