// layer_api.hip -- the C entry points of the layer operators: validation,
// plans, workspace layout and launch.  Declarations and contracts are in
// include/ssm.h.
#include "ssm.h"

#include "layer_launch.h"

namespace {

constexpr int64_t kMaxGrid = 2147483647;
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether a product of dimensions stays within what the kernels index with.
bool fits(double a, double b, double c = 1.0, double d = 1.0) { return a * b * c * d < 9.0e18; }

ssm_status status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

bool io_ok(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
size_t io_size(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

// ------------------------------------------------------------- scan over heads
ssm_status check_heads(const ssm_heads_desc *d, bool update) {
    if (!d) return SSM_ERR_NULL_ARG;
    if (d->batch < 0 || d->heads < 1 || d->head_dim < 1 || d->groups < 1) return SSM_ERR_BAD_SHAPE;
    if (d->heads % d->groups != 0) return SSM_ERR_BAD_SHAPE;
    if (d->d_state < 1 || d->d_state > SSM_MAX_D_STATE) return SSM_ERR_UNSUPPORTED;
    if (d->head_dim > SSM_MAX_HEAD_DIM || d->heads > SSM_MAX_HEADS) return SSM_ERR_UNSUPPORTED;
    if (!io_ok(d->io_dtype) || d->flags != 0 || d->reserved != 0) return SSM_ERR_UNSUPPORTED;
    const int64_t st[] = {d->u_batch_stride, d->u_token_stride, d->delta_batch_stride,
                          d->delta_token_stride, d->B_batch_stride, d->B_token_stride,
                          d->C_batch_stride, d->C_token_stride, d->dy_batch_stride,
                          d->dy_token_stride};
    for (int64_t s : st)
        if (s < 0) return SSM_ERR_BAD_SHAPE;
    if (!fits(d->batch, d->heads, d->head_dim, 4.0 * d->d_state)) return SSM_ERR_BAD_SHAPE;
    if (update) return SSM_OK;
    if (d->seqlen < 0 || d->n_seqs < 0) return SSM_ERR_BAD_SHAPE;
    if (d->seqlen > SSM_MAX_SEQLEN) return SSM_ERR_UNSUPPORTED;
    if (d->n_seqs > 0 && d->batch != 1) return SSM_ERR_BAD_SHAPE;
    if (!fits(d->batch, d->seqlen, d->heads, 4.0 * d->head_dim)) return SSM_ERR_BAD_SHAPE;
    return SSM_OK;
}

struct HeadsPlan {
    int Q = 64;
    int64_t nc = 0, Kc = 1, J = 1, wgs = 0, sph = 0, rows = 0;
    int64_t hsplit = 1, hblk = 1, na = 0;
    size_t table = 0, hend = 0, ldec = 0, hin = 0, gout = 0, rp = 0, rpsum = 0, hdot = 0, through = 0,
           rest = 0, adot = 0, rec = 0, part = 0, dBp = 0, dCp = 0, bytes = 0;
};

// A walk is serial over its chunks, and a compute unit holds three of its
// workgroups (at 128 states).  Below one workgroup a compute unit the rows are
// cut into ranges of at least 4 chunks, for about three a compute unit; the
// launch that finds the ranges' states costs half a walk more.  (1 x 65536 x 32
// heads: pre-pass, join and walk 503 us aimed at 768 workgroups, 553 at 512,
// 562 at 1024.)
ssm_status plan_heads(const ssm_heads_desc *d, bool bwd, HeadsPlan *p) {
    const int bf16 = d->io_dtype == SSM_BF16;
    const int64_t hpg = d->heads / d->groups;
    p->rows = d->n_seqs > 0 ? d->n_seqs : d->batch;
    p->Q = bwd ? ssm::heads_bwd_chunk(bf16, d->d_state) : ssm::heads_fwd_chunk(bf16, d->d_state);
    p->nc = ceil_div(d->seqlen, p->Q);
    if (d->n_seqs > 0) {
        p->nc += d->n_seqs;
        if (p->nc > d->seqlen) p->nc = d->seqlen;
    }
    p->sph = ceil_div(d->head_dim, 16);
    p->wgs = d->groups * ceil_div(hpg * p->sph, 4);
    const int64_t base = d->batch * p->wgs * (bwd ? 2 : 1);
    // the most that a walk of one head a workgroup takes, should it be more
    const int64_t most = d->batch * d->heads * ceil_div(p->sph, 4) * (bwd ? 2 : 1);
    p->Kc = p->nc > 0 ? p->nc : 1;
    if (base > 0 && base < 256 && p->nc >= 8) {
        int64_t J = ceil_div(768, base);
        if (J > p->nc / 4) J = p->nc / 4;
        p->Kc = ceil_div(p->nc, J);
    }
    p->J = p->nc > 0 ? ceil_div(p->nc, p->Kc) : 1;
    const int64_t chunks = d->batch * p->nc;
    if (static_cast<double>(base > most ? base : most) * p->J > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    size_t at = 0;
    auto take = [&](double n, double esz) {
        const size_t o = at;
        at = align_up(at + static_cast<size_t>(n * esz));
        return o;
    };
    const double state = static_cast<double>(d->heads) * d->head_dim * d->d_state;
    if (d->n_seqs > 0) p->table = take(p->nc, sizeof(ssm::HeadsEntry));
    if (p->J > 1) {
        p->hend = take(state * d->batch * p->J * (bwd ? 2 : 1), 4);
        p->ldec = take(static_cast<double>(d->batch) * p->J * d->heads * (bwd ? 2 : 1), 4);
    }
    if (bwd) {
        if (d->batch > 65535) return SSM_ERR_UNSUPPORTED;
        // Blocks of a group's heads, each a workgroup a chunk, for two workgroups
        // a compute unit, which is what one holds; the blocks' dB and dC are then
        // added.  More blocks add more, fewer leave units empty: 1 x 2048, 2 x
        // 2048 and 4 x 2048 x 80 heads 224, 326 and 566 us; aimed at 1024
        // workgroups 250, 346 and 579, at 256 224, 351 and 623.
        p->hsplit = 1;
        if (chunks > 0 && chunks * d->groups < 512) p->hsplit = ceil_div(512, chunks * d->groups);
        if (p->hsplit > hpg) p->hsplit = hpg;
        p->hblk = ceil_div(hpg, p->hsplit);
        p->hsplit = ceil_div(hpg, p->hblk);
        if (static_cast<double>(chunks) * d->groups * p->hsplit > kMaxGrid ||
            static_cast<double>(chunks) * d->heads > kMaxGrid)
            return SSM_ERR_UNSUPPORTED;
        const double slices = static_cast<double>(d->heads) * p->sph;
        const double st = static_cast<double>(chunks) * slices * 16 * ssm::heads_np(d->d_state);
        p->hin = take(st, io_size(d->io_dtype));
        p->gout = take(st, io_size(d->io_dtype));
        p->rp = take(2.0 * chunks * slices * p->Q, 4);
        p->rpsum = take(2.0 * chunks * slices, 4);
        p->hdot = take(p->rows * slices, 4);
        p->na = ceil_div(p->nc, ssm::kAnchor);
        if (bf16) p->rest = take(2.0 * d->batch * p->na * slices * 16 * ssm::heads_np(d->d_state), 2);
        p->adot = take(static_cast<double>(d->batch) * p->na * d->heads, 4);
        p->through = take(static_cast<double>(chunks) * d->heads, 4);
        p->rec = take(static_cast<double>(chunks) * d->heads, ssm::kGradRec);
        p->part = take(3.0 * chunks * d->heads, 4);
        if (p->hsplit > 1) {
            const double n = static_cast<double>(p->hsplit) * d->batch * d->seqlen * d->groups * d->d_state;
            p->dBp = take(n, 4);
            p->dCp = take(n, 4);
        }
    }
    p->bytes = at;
    return SSM_OK;
}

void heads_args(const ssm_heads_desc *d, const HeadsPlan &p, bool bwd, ssm::HeadsArgs *a) {
    a->batch = d->batch; a->L = d->seqlen; a->H = d->heads; a->P = d->head_dim; a->G = d->groups;
    a->N = d->d_state;
    a->bf16 = d->io_dtype == SSM_BF16;
    a->softplus = d->softplus != 0;
    a->u_b = d->u_batch_stride; a->u_t = d->u_token_stride;
    a->dt_b = d->delta_batch_stride; a->dt_t = d->delta_token_stride;
    a->B_b = d->B_batch_stride; a->B_t = d->B_token_stride;
    a->C_b = d->C_batch_stride; a->C_t = d->C_token_stride;
    a->dy_b = d->dy_batch_stride; a->dy_t = d->dy_token_stride;
    a->rows = p.rows;
    a->Q = p.Q; a->nc = p.nc; a->Kc = p.Kc; a->J = p.J;
    a->hsplit = p.hsplit; a->hblk = p.hblk;
    char *w = static_cast<char *>(d->workspace);
    auto f = [&](size_t o) { return reinterpret_cast<float *>(w + o); };
    a->table = reinterpret_cast<ssm::HeadsEntry *>(w + p.table);
    a->hend = f(p.hend); a->ldec = f(p.ldec);
    if (!bwd) return;
    a->hin = w + p.hin; a->gout = w + p.gout;
    a->rp = f(p.rp); a->rpsum = f(p.rpsum); a->hdot = f(p.hdot); a->through = f(p.through);
    a->rest = reinterpret_cast<uint16_t *>(f(p.rest)); a->adot = f(p.adot); a->na = p.na;
    a->rec = w + p.rec; a->part = f(p.part); a->dBp = f(p.dBp); a->dCp = f(p.dCp);
}

ssm_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SSM_OK;
    if (!ws || have < need) return SSM_ERR_WORKSPACE;
    return aligned(ws, 16) ? SSM_OK : SSM_ERR_MISALIGNED;
}

// ---------------------------------------------------------------- convolution
ssm_status check_conv(const ssm_conv_desc *d, bool update) {
    if (!d) return SSM_ERR_NULL_ARG;
    if (d->batch < 0 || d->channels < 0) return SSM_ERR_BAD_SHAPE;
    if (d->width < 1 || d->width > SSM_MAX_CONV_WIDTH) return SSM_ERR_UNSUPPORTED;
    if (!io_ok(d->io_dtype) || d->flags != 0 || d->reserved != 0) return SSM_ERR_UNSUPPORTED;
    if (d->x_batch_stride < 0 || d->x_token_stride < 0 || d->dy_batch_stride < 0 ||
        d->dy_token_stride < 0)
        return SSM_ERR_BAD_SHAPE;
    if (!fits(d->batch, d->channels, 16.0)) return SSM_ERR_BAD_SHAPE;
    if (static_cast<double>(d->batch) * d->channels / 256 > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    if (update) return SSM_OK;
    if (d->seqlen < 0 || d->n_seqs < 0) return SSM_ERR_BAD_SHAPE;
    if (d->seqlen > SSM_MAX_SEQLEN) return SSM_ERR_UNSUPPORTED;
    if (d->n_seqs > 0 && d->batch != 1) return SSM_ERR_BAD_SHAPE;
    if (!fits(d->batch, d->seqlen, d->channels, 16.0)) return SSM_ERR_BAD_SHAPE;
    return SSM_OK;
}

// Tokens of one run of the convolution's gradients: long ones, which leave fewer
// partial rows, where there are two wavefronts a SIMD of them all the same.  (Runs
// of 64 against 32: 4 x 2048 x 5376 in bfloat16 72 against 77 us, 8 x 4096 259
// against 270; runs of 16 against 32: 1 x 2048 x 2048 21 against 29 us.)
int64_t conv_run(const ssm_conv_desc *d) {
    const int64_t waves = ceil_div(d->channels, 256) * d->batch;
    for (int64_t run = 64; run > 16; run /= 2)
        if (waves * ceil_div(d->seqlen, run) >= 2048) return run;
    return 16;
}
int64_t conv_runs(const ssm_conv_desc *d) { return d->batch * ceil_div(d->seqlen, conv_run(d)); }

void conv_args(const ssm_conv_desc *d, ssm::ConvArgs *a) {
    a->batch = d->batch; a->L = d->seqlen; a->C = d->channels; a->W = d->width;
    a->bf16 = d->io_dtype == SSM_BF16;
    a->silu = d->silu != 0;
    a->x_batch = d->x_batch_stride; a->x_token = d->x_token_stride;
    a->dy_batch = d->dy_batch_stride; a->dy_token = d->dy_token_stride;
    a->rows = d->n_seqs > 0 ? d->n_seqs : d->batch;
}

// ----------------------------------------------------------------------- norm
ssm_status check_norm(const ssm_norm_desc *d) {
    if (!d) return SSM_ERR_NULL_ARG;
    if (d->rows < 0 || d->d < 1 || d->group_size < 1 || d->d % d->group_size != 0)
        return SSM_ERR_BAD_SHAPE;
    if (d->group_size > ssm::kNormMaxGroup) return SSM_ERR_UNSUPPORTED;
    if (!io_ok(d->io_dtype) || d->flags != 0 || d->reserved != 0) return SSM_ERR_UNSUPPORTED;
    // the residual's type is the activations' or float32
    if (d->residual_dtype != d->io_dtype && d->residual_dtype != SSM_F32) return SSM_ERR_UNSUPPORTED;
    if (d->x_stride < 0 || d->z_stride < 0 || d->residual_stride < 0 || d->dy_stride < 0)
        return SSM_ERR_BAD_SHAPE;
    if (d->quant_block < 0) return SSM_ERR_BAD_SHAPE;
    if (d->quant_block > 0 && d->quant_block < 16 && d->quant_block < d->group_size)
        return SSM_ERR_UNSUPPORTED;
    if (!fits(d->rows, d->d, 4.0)) return SSM_ERR_BAD_SHAPE;
    if (static_cast<double>(d->rows) * (d->d / d->group_size) > kMaxGrid) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

void norm_args(const ssm_norm_desc *d, ssm::NormArgs *a) {
    a->rows = d->rows; a->d = d->d; a->group = d->group_size;
    a->bf16 = d->io_dtype == SSM_BF16;
    a->res_bf16 = d->residual_dtype == SSM_BF16;
    a->eps = d->eps;
    a->x_row = d->x_stride; a->z_row = d->z_stride; a->res_row = d->residual_stride;
    a->dy_row = d->dy_stride;
    a->block = d->quant_block;
}

}  // namespace

extern "C" {

size_t ssm_heads_workspace_bytes(const ssm_heads_desc *desc, int backward) {
    HeadsPlan p;
    if (check_heads(desc, false) != SSM_OK || plan_heads(desc, backward != 0, &p) != SSM_OK) return 0;
    return p.bytes;
}

ssm_status ssm_heads_fwd(const ssm_heads_desc *desc, const void *u, const void *delta,
                         const float *A, const void *B, const void *C, const float *D,
                         const float *delta_bias, const float *initial_state,
                         const int32_t *cu_seqlens, void *y, float *last_state,
                         ssm_stream_t stream) {
    ssm_status st = check_heads(desc, false);
    if (st != SSM_OK) return st;
    if ((cu_seqlens != nullptr) != (desc->n_seqs > 0)) return SSM_ERR_BAD_SHAPE;
    HeadsPlan p;
    if ((st = plan_heads(desc, false, &p)) != SSM_OK) return st;
    if (desc->batch == 0) return SSM_OK;
    if (!A || (desc->seqlen > 0 && (!u || !delta || !B || !C || !y))) return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    if (!aligned(u, e) || !aligned(delta, e) || !aligned(B, e) || !aligned(C, e) || !aligned(y, e) ||
        !aligned(A, 4) || !aligned(D, 4) || !aligned(delta_bias, 4) || !aligned(initial_state, 4) ||
        !aligned(cu_seqlens, 4) || !aligned(last_state, 4))
        return SSM_ERR_MISALIGNED;
    if ((st = check_workspace(desc->workspace, desc->workspace_bytes, p.bytes)) != SSM_OK) return st;
    ssm::HeadsArgs a{};
    heads_args(desc, p, false, &a);
    a.u = u; a.delta = delta; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = delta_bias;
    a.h0 = initial_state; a.cu = cu_seqlens; a.y = y; a.last = last_state;
    return status(ssm::launch_heads_fwd(a, stream));
}

ssm_status ssm_heads_bwd(const ssm_heads_desc *desc, const void *u, const void *delta,
                         const float *A, const void *B, const void *C, const float *D,
                         const float *delta_bias, const float *initial_state,
                         const int32_t *cu_seqlens, const void *dy, const float *dlast, void *du,
                         void *ddelta, float *dA, void *dB, void *dC, float *dD,
                         float *ddelta_bias, float *dh0, ssm_stream_t stream) {
    ssm_status st = check_heads(desc, false);
    if (st != SSM_OK) return st;
    if ((cu_seqlens != nullptr) != (desc->n_seqs > 0)) return SSM_ERR_BAD_SHAPE;
    HeadsPlan p;
    if ((st = plan_heads(desc, true, &p)) != SSM_OK) return st;
    if (!A || !dA) return SSM_ERR_NULL_ARG;
    if (desc->batch * desc->seqlen > 0 &&
        (!u || !delta || !B || !C || !dy || !du || !ddelta || !dB || !dC))
        return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    const void *io[] = {u, delta, B, C, dy, du, ddelta, dB, dC};
    for (const void *q : io)
        if (!aligned(q, e)) return SSM_ERR_MISALIGNED;
    const void *f[] = {A, D, delta_bias, initial_state, cu_seqlens, dlast, dA, dD, ddelta_bias, dh0};
    for (const void *q : f)
        if (!aligned(q, 4)) return SSM_ERR_MISALIGNED;
    if ((st = check_workspace(desc->workspace, desc->workspace_bytes, p.bytes)) != SSM_OK) return st;
    ssm::HeadsArgs a{};
    heads_args(desc, p, true, &a);
    a.u = u; a.delta = delta; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = delta_bias;
    a.h0 = initial_state; a.cu = cu_seqlens; a.dy = dy; a.dlast = dlast;
    a.du = du; a.ddelta = ddelta; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dbias = ddelta_bias;
    a.dh0 = dh0;
    return status(ssm::launch_heads_bwd(a, stream));
}

ssm_status ssm_heads_update(const ssm_heads_desc *desc, float *state, const int32_t *slots,
                            int64_t n_slots, const void *u, const void *delta, const float *A,
                            const void *B, const void *C, const float *D, const float *delta_bias,
                            void *y, ssm_stream_t stream) {
    const ssm_status st = check_heads(desc, true);
    if (st != SSM_OK) return st;
    if (n_slots < 0 || (!slots && desc->batch > n_slots)) return SSM_ERR_BAD_SHAPE;
    if (!fits(n_slots, desc->heads, desc->head_dim, 4.0 * desc->d_state)) return SSM_ERR_BAD_SHAPE;
    if (desc->batch == 0) return SSM_OK;
    // at most one workgroup a channel
    if (static_cast<double>(desc->batch) * desc->heads * desc->head_dim > kMaxGrid)
        return SSM_ERR_UNSUPPORTED;
    if (!state || !u || !delta || !A || !B || !C || !y) return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    if (!aligned(u, e) || !aligned(delta, e) || !aligned(B, e) || !aligned(C, e) || !aligned(y, e) ||
        !aligned(A, 4) || !aligned(D, 4) || !aligned(delta_bias, 4) || !aligned(state, 4) ||
        !aligned(slots, 4))
        return SSM_ERR_MISALIGNED;
    ssm::HeadsArgs a{};
    HeadsPlan p;
    heads_args(desc, p, false, &a);
    a.u = u; a.delta = delta; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = delta_bias; a.y = y;
    a.state = state; a.slots = slots; a.n_slots = n_slots;
    return status(ssm::launch_heads_update(a, stream));
}

size_t ssm_conv_workspace_bytes(const ssm_conv_desc *desc) {
    if (check_conv(desc, false) != SSM_OK) return 0;
    return align_up(static_cast<size_t>(conv_runs(desc)) * (desc->width + 1) * desc->channels * 4);
}

ssm_status ssm_conv_fwd(const ssm_conv_desc *desc, const void *x, const float *weight,
                        const float *bias, const float *conv_state, const int32_t *cu_seqlens,
                        void *y, float *last_state, ssm_stream_t stream) {
    const ssm_status st = check_conv(desc, false);
    if (st != SSM_OK) return st;
    if ((cu_seqlens != nullptr) != (desc->n_seqs > 0)) return SSM_ERR_BAD_SHAPE;
    if (desc->batch * desc->channels == 0) return SSM_OK;
    if (!weight || (desc->seqlen > 0 && (!x || !y))) return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(conv_state, 4) || !aligned(cu_seqlens, 4) || !aligned(last_state, 4))
        return SSM_ERR_MISALIGNED;
    ssm::ConvArgs a{};
    conv_args(desc, &a);
    a.x = x; a.weight = weight; a.bias = bias; a.state = conv_state; a.cu = cu_seqlens; a.y = y;
    a.last = last_state;
    return status(ssm::launch_conv_fwd(a, stream));
}

ssm_status ssm_conv_bwd(const ssm_conv_desc *desc, const void *x, const float *weight,
                        const float *bias, const float *conv_state, const int32_t *cu_seqlens,
                        const void *dy, void *dx, float *dweight, float *dbias, float *dconv_state,
                        ssm_stream_t stream) {
    ssm_status st = check_conv(desc, false);
    if (st != SSM_OK) return st;
    if ((cu_seqlens != nullptr) != (desc->n_seqs > 0)) return SSM_ERR_BAD_SHAPE;
    if (desc->channels == 0) return SSM_OK;
    if (!weight || !dweight || (desc->batch * desc->seqlen > 0 && (!x || !dy || !dx)))
        return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(conv_state, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(dconv_state, 4))
        return SSM_ERR_MISALIGNED;
    if ((st = check_workspace(desc->workspace, desc->workspace_bytes, ssm_conv_workspace_bytes(desc))) !=
        SSM_OK)
        return st;
    ssm::ConvArgs a{};
    conv_args(desc, &a);
    a.x = x; a.weight = weight; a.bias = bias; a.state = conv_state; a.cu = cu_seqlens; a.dy = dy;
    a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.dstate = dconv_state;
    a.part = static_cast<float *>(desc->workspace);
    a.runs = conv_runs(desc); a.run = conv_run(desc);
    return status(ssm::launch_conv_bwd(a, stream));
}

ssm_status ssm_conv_update(const ssm_conv_desc *desc, float *conv_state, const int32_t *slots,
                           int64_t n_slots, const void *x, const float *weight, const float *bias,
                           void *y, ssm_stream_t stream) {
    const ssm_status st = check_conv(desc, true);
    if (st != SSM_OK) return st;
    if (n_slots < 0 || (!slots && desc->batch > n_slots)) return SSM_ERR_BAD_SHAPE;
    if (!fits(n_slots, desc->channels, 16.0)) return SSM_ERR_BAD_SHAPE;
    if (desc->batch * desc->channels == 0) return SSM_OK;
    if (!x || !weight || !y || (desc->width > 1 && !conv_state)) return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(conv_state, 4) || !aligned(slots, 4))
        return SSM_ERR_MISALIGNED;
    ssm::ConvArgs a{};
    conv_args(desc, &a);
    a.x = x; a.weight = weight; a.bias = bias; a.y = y;
    a.slot_state = conv_state; a.slots = slots; a.n_slots = n_slots;
    return status(ssm::launch_conv_update(a, stream));
}

size_t ssm_norm_workspace_bytes(const ssm_norm_desc *desc) {
    if (check_norm(desc) != SSM_OK) return 0;
    return align_up(static_cast<size_t>(ssm::norm_bwd_blocks(desc->rows, desc->d, desc->group_size)) *
                    desc->d * 4);
}

ssm_status ssm_norm_fwd(const ssm_norm_desc *desc, const void *x, const float *weight,
                        const void *residual, const void *z, void *y, float *scale,
                        void *residual_out, ssm_stream_t stream) {
    const ssm_status st = check_norm(desc);
    if (st != SSM_OK) return st;
    if (desc->rows == 0) return SSM_OK;
    if (!x || !weight || !y || (residual && !residual_out) || (desc->quant_block > 0 && !scale))
        return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype), r = io_size(desc->residual_dtype);
    if (!aligned(x, e) || !aligned(z, e) || !aligned(y, desc->quant_block > 0 ? 1 : e) ||
        !aligned(weight, 4) || !aligned(scale, 4) || !aligned(residual, r) || !aligned(residual_out, r))
        return SSM_ERR_MISALIGNED;
    ssm::NormArgs a{};
    norm_args(desc, &a);
    a.x = x; a.weight = weight; a.residual = residual; a.z = z; a.y = y; a.scale = scale;
    a.residual_out = residual_out;
    return status(ssm::launch_norm_fwd(a, stream));
}

ssm_status ssm_norm_bwd(const ssm_norm_desc *desc, const void *x, const float *weight,
                        const void *z, const void *dy, const void *dresidual, void *dx, void *dz,
                        float *dweight, ssm_stream_t stream) {
    ssm_status st = check_norm(desc);
    if (st != SSM_OK) return st;
    if (desc->quant_block != 0) return SSM_ERR_UNSUPPORTED;
    if (!weight || !dweight || (desc->rows > 0 && (!x || !dy || !dx || (z && !dz))))
        return SSM_ERR_NULL_ARG;
    const size_t e = io_size(desc->io_dtype), r = io_size(desc->residual_dtype);
    if (!aligned(x, r) || !aligned(z, e) || !aligned(dy, e) || !aligned(dresidual, r) ||
        !aligned(dx, r) || !aligned(dz, e) || !aligned(weight, 4) || !aligned(dweight, 4))
        return SSM_ERR_MISALIGNED;
    if ((st = check_workspace(desc->workspace, desc->workspace_bytes, ssm_norm_workspace_bytes(desc))) !=
        SSM_OK)
        return st;
    ssm::NormArgs a{};
    norm_args(desc, &a);
    a.x = x; a.weight = weight; a.z = z; a.dy = dy; a.dresidual = dresidual; a.dx = dx; a.dz = dz;
    a.dweight = dweight;
    a.part = static_cast<float *>(desc->workspace);
    a.nblk = ssm::norm_bwd_blocks(desc->rows, desc->d, desc->group_size);
    return status(ssm::launch_norm_bwd(a, stream));
}

}  // extern "C"
