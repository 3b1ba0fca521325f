"""Plain 64-bit forms of the layer operators, and error bounds derived from
them, for the tests of the scan over heads, the convolution and the norm.

Bounds count roundings.  A value rounded to a type is off by at most half a
step, HALF[type] relative to it; a float32 sum of n terms by at most n 2^-24
of the sum of the terms' magnitudes.  That sum is the same plain form taken of
the inputs' magnitudes: every output and gradient of the scan is a sum of
products of u, B, C, dy and states with positive factors (decays, step sizes).

A step size is good to 4 units of 2^-24 (an exponential, a logarithm, a sum and
a product), so a decay exp(-gap) over a gap of log decays is off by 4 gap 2^-24
of it: a sum by 4 2^-24 of the sum of gap times each term's magnitude.  As
exp(-gap (1 - e)) >= exp(-gap) (1 + gap e), that is at most what the sum of
magnitudes gains, over e, when all log decays shrink by e = 2^-10.
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def spans_of(L, batch, lens):
    """(batch row, first token, one past the last) of each sequence."""
    if lens is None:
        return [(b, 0, L) for b in range(batch)]
    out, at = [], 0
    for n in lens:
        out.append((0, at, at + n))
        at += n
    return out


def step_sizes(delta, bias, softplus):
    v = delta.double() + (0.0 if bias is None else bias.double())
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs())) if softplus else v


def scan(u, w, a, B, C, h0, spans, marks=None):
    """y without the skip term and the last states, token by token in 64 bits:
    h = exp(a) h + w u (x) B, y = h C.  u (b, L, H, P); w, a (b, L, H); B, C
    (b, L, G, N); h0 (rows, H, P, N).  marks: a list that gets, by sequence, the
    states that enter every 32nd token and the last one."""
    per = u.shape[2] // B.shape[2]
    Bh, Ch = B.repeat_interleave(per, 2), C.repeat_interleave(per, 2)
    y, last = {}, []
    for r, (b, i, j) in enumerate(spans):
        h = h0[r]
        kept = [h]
        for t in range(i, j):
            h = (torch.exp(a[b, t])[:, None, None] * h
                 + (w[b, t][:, None] * u[b, t])[:, :, None] * Bh[b, t][:, None, :])
            y[b, t] = (h * Ch[b, t][:, None, :]).sum(-1)
            if (t + 1 - i) % 32 == 0:
                kept.append(h)
        kept.append(h)
        if marks is not None:
            marks.append(kept)
        last.append(h)
    zero = torch.zeros_like(u[0, 0])
    y = torch.stack([torch.stack([y.get((b, t), zero) for t in range(u.shape[1])])
                     for b in range(u.shape[0])])
    return y, torch.stack(last)


def f64(t):
    return None if t is None else t.detach().double().cpu()


def heads_reference(u, delta, A, B, C, D, bias, h0, lens, softplus=True, dy=None, dlast=None):
    """Outputs (and, with dy, gradients) in 64 bits, for each the sum of its
    terms' magnitudes, and under "decays" what the decays' errors add, in units
    of 2^-24."""
    u, delta, A, B, C, D, bias, h0, dy, dlast = map(
        f64, (u, delta, A, B, C, D, bias, h0, dy, dlast))
    spans = spans_of(u.shape[1], u.shape[0], lens)
    H, P, N = u.shape[2], u.shape[3], B.shape[3]
    w = step_sizes(delta, bias, softplus)
    a = w * A
    start = h0 if h0 is not None else torch.zeros(len(spans), H, P, N, dtype=torch.float64)
    ref, size, more = {}, {}, {}
    for out, mag in ((ref, False), (size, True), (more, True)):
        take = (lambda t: t.abs()) if mag else (lambda t: t)
        leaf = [take(t).clone().requires_grad_() for t in (u, B, C, start)]
        shrink = 1 - 2.0 ** -10 if out is more else 1.0
        wl, al = take(w).clone().requires_grad_(), (a * shrink).requires_grad_()
        marks = []
        y, last = scan(leaf[0], wl, al, leaf[1], leaf[2], leaf[3], spans, marks)
        skip = 0.0 if D is None else take(D)[:, None] * leaf[0]
        out["y"], out["last_state"] = (y + skip).detach(), last.detach()
        if dy is None:
            continue
        for kept in marks:
            for h in kept[1:]:
                if h.requires_grad:
                    h.retain_grad()
        loss = (y * take(dy)).sum()
        if dlast is not None:
            loss = loss + (last * take(dlast)).sum()
        loss.backward()
        g = lambda t: torch.zeros_like(t) if t.grad is None else t.grad
        du = g(leaf[0]) + (0.0 if D is None else take(D)[:, None] * take(dy))
        out.update(du=du, dB=g(leaf[1]), dC=g(leaf[2]), dh0=g(leaf[3]))
        out["dD"] = (take(dy) * take(u)).sum((0, 1, 3))
        ga = g(al)
        if mag:
            # the running sums in a sequence are as exact as their largest
            for b, i, j in spans:
                if j > i:
                    ga[b, i:j] = ga[b, i:j].amax(0)
        ddt = g(wl) + (A.abs() if mag else A) * ga
        out["dA"] = (ga * take(w)).sum((0, 1))
        act = torch.sigmoid(delta + (0.0 if bias is None else bias)) if softplus else 1.0
        out["ddelta"] = ddt * act
        out["ddelta_bias"] = out["ddelta"].sum((0, 1))
        if mag:
            # <gradient leaving a chunk, state entering it>, by tokens of the chunk:
            # 2^-13 of it at most is taken from bfloat16 copies
            through = torch.zeros_like(w)
            for (b, i, j), kept in zip(spans, marks):
                for m in range(len(kept) - 1):
                    gh = torch.zeros_like(kept[m + 1]) if kept[m + 1].grad is None else kept[m + 1].grad
                    t0, t1 = i + 32 * m, min(i + 32 * m + 32, j)
                    through[b, t0:t1] = (gh * kept[m]).sum((1, 2)).detach()
            out["through_ddelta"] = A.abs() * through * act
            out["through_dA"] = (w.abs() * through).sum((0, 1))
            out["through_ddelta_bias"] = out["through_ddelta"].sum((0, 1))
    # the decays' share of the error, in units of 2^-24
    size["decays"] = {k: 4 * (more[k] - size[k]).clamp(min=0) * 2.0 ** 10 for k in ref}
    return ref, size


def assert_within(name, got, ref, bound):
    err = (f64(got) - ref).abs()
    assert err.shape == bound.shape, (name, err.shape, bound.shape)
    assert torch.isfinite(f64(got)).all(), f"{name}: not finite"
    over = err > bound
    if over.any():
        at = (err - bound).argmax().item()
        raise AssertionError(f"{name}: {int(over.sum())} of {over.numel()} off, worst "
                             f"{err.flatten()[at]:.3e} against {bound.flatten()[at]:.3e}")


def conv_reference(x, weight, bias, state, lens, silu=True, dy=None):
    x, weight, bias, state, dy = map(f64, (x, weight, bias, state, dy))
    b_, L, ch = x.shape
    W = weight.shape[1]
    spans = spans_of(L, b_, lens)
    if state is None:
        state = torch.zeros(len(spans), ch, W - 1, dtype=torch.float64)
    ref, size = {}, {}
    for out, mag in ((ref, False), (size, True)):
        take = (lambda t: t.abs()) if mag else (lambda t: t)
        leaf = [t.clone().requires_grad_() for t in map(take, (x, weight, state))]
        v = torch.zeros_like(x)
        last = torch.zeros(len(spans), ch, W - 1, dtype=torch.float64)
        for r, (b, i, j) in enumerate(spans):
            line = torch.cat([leaf[2][r].T, leaf[0][b, i:j]])
            part = sum(leaf[1][:, k] * line[k:k + j - i] for k in range(W))
            v = v + torch.nn.functional.pad(part, (0, 0, i, L - j))[None] * (
                torch.arange(b_)[:, None, None] == b)
            last[r] = line[j - i:].T.detach()
        if not mag:
            pre = v.detach() + (0.0 if bias is None else bias)
        vb = v if bias is None else v + take(bias)
        act = torch.sigmoid(pre) if silu else torch.ones_like(pre)
        out["y"] = (vb.detach() * act)
        out["last"] = last
        if dy is not None:
            # silu' as the forward's values give it; its magnitude is below 1.1
            slope = act * (1 + pre * (1 - act)) if silu else act
            dv = dy * slope if not mag else dy.abs() * (1.1 * torch.ones_like(slope))
            g = torch.autograd.grad((v * dv).sum(), leaf, allow_unused=True)
            out["dx"], out["dweight"], out["dconv_state"] = (
                torch.zeros_like(t) if q is None else q for t, q in zip(leaf, g))
            out["dbias"] = dv.sum((0, 1))
    return ref, size


def norm_reference(s, weight, z, group, eps=1e-5, dy=None, dresidual=None):
    s, weight, z, dy, dresidual = map(f64, (s, weight, z, dy, dresidual))
    leaf = [t if t is None else t.clone().requires_grad_() for t in (s, weight, z)]
    g = leaf[0] if z is None else leaf[0] * leaf[2] * torch.sigmoid(leaf[2])
    v = g.unflatten(-1, (-1, group))
    n = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)).flatten(-2)
    y = n * leaf[1]
    out = {"y": y.detach(), "n": n.detach()}
    if dy is not None:
        got = torch.autograd.grad((y * dy).sum(), [t for t in leaf if t is not None])
        out["dx"], out["dweight"] = got[0], got[1]
        if dresidual is not None:
            out["dx"] = out["dx"] + dresidual
        if z is not None:
            out["dz"] = got[2]
    return out
