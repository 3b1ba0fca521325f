"""Cases of the layer operators: the scan over heads (prompt, gradients, single
token), the short causal convolution in front of it (the same three) and the
root-mean-square norm behind it (output, gradients).

``run`` computes a case in elementary torch operations in 32 bits, or, where
``own`` is set, through this package's entry points.  ``exact`` computes it
from the definitions in 64 bits: token by token, or as one masked product over
the whole sequence.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8_MAX = 448.0


# ------------------------------------------------------------------- cases

def _heads(op, name, io, batch, L, heads, head_dim, groups, N, lens="", state=False):
    return {"name": name, "op": op, "io": io, "batch": batch, "L": L, "heads": heads,
            "head_dim": head_dim, "groups": groups, "N": N, "lens": lens, "state": state}


def _conv(op, name, io, batch, L, channels, W, lens="", state=False):
    return {"name": name, "op": op, "io": io, "batch": batch, "L": L, "channels": channels,
            "W": W, "lens": lens, "state": state}


def _norm(op, name, io, rows, d, group, residual="", gate=False, block=0):
    return {"name": name, "op": op, "io": io, "rows": rows, "d": d, "group": group,
            "residual": residual, "gate": gate, "block": block}


def listed():
    return [
        # prompts of a 2.8B-sized layer: eight of 2048 tokens, 80 heads of 64
        _heads("heads_fwd", "heads_prompt_bf16", "bf16", 8, 2048, 80, 64, 1, 128),
        # one meeting-length sequence: few rows, a long axis
        _heads("heads_fwd", "heads_long_bf16", "bf16", 1, 65536, 32, 64, 1, 128),
        # ragged prompts packed behind one another, continued from kept states
        _heads("heads_fwd", "heads_packed_f32", "f32", 1, 4099, 20, 64, 2, 64,
               "1,700,33,1024,2,1500,64,775", True),
        # a training step of the 2.8B-sized layer
        _heads("heads_bwd", "heads_train_bf16", "bf16", 4, 2048, 80, 64, 1, 128),
        # one token of one request, and of 256 requests, states in slots
        _heads("heads_update", "heads_token_1_bf16", "bf16", 1, 1, 80, 64, 1, 128),
        _heads("heads_update", "heads_token_256_bf16", "bf16", 256, 1, 80, 64, 1, 128),
        # the convolution in front of the same layer, a training step of it,
        # and one token of 256 requests
        _conv("conv_fwd", "conv_prompt_bf16", "bf16", 8, 2048, 5376, 4),
        _conv("conv_bwd", "conv_train_bf16", "bf16", 4, 2048, 5376, 4),
        _conv("conv_update", "conv_token_256_f32", "f32", 256, 1, 5376, 4),
        # gate and norm behind the scan, in 8 bits for the projection after it
        _norm("norm_fwd", "norm_gated_8bit_bf16", "bf16", 16384, 5120, 5120, gate=True, block=128),
        # the norm in front of the layer for a few decoded tokens: residual
        # kept in float32
        _norm("norm_fwd", "norm_residual_4_bf16", "bf16", 4, 2560, 2560, residual="f32"),
        # a training step of the gated norm, in two groups
        _norm("norm_bwd", "norm_train_bf16", "bf16", 8192, 5120, 2560, gate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, total):
    """Ragged lengths, empty ones among them, that sum to `total`."""
    n = rng.randint(2, 9)
    at = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + at, at + [total]))


def draw(rng):
    op = rng.choice(["heads_fwd", "heads_fwd", "heads_bwd", "heads_bwd", "heads_update",
                     "conv_fwd", "conv_bwd", "conv_update", "norm_fwd", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("heads"):
        groups = rng.choice([1, 1, 1, 2, 4])
        heads = groups * _log_int(rng, 1, 80 // groups)
        head_dim = rng.choice([16, 32, 64, 64, 64, 128, 48, 33])
        N = rng.choice([16, 32, 64, 128, 128, 256, 24, 100])
        if op == "heads_update":
            batch = max(1, min(_log_int(rng, 1, 300), 160_000_000 // (heads * head_dim * N)))
            c = _heads(op, "", io, batch, 1, heads, head_dim, groups, N)
        else:
            batch = rng.randint(1, 8)
            most = 1.0e10 if op == "heads_fwd" else 5.0e9      # batch L heads head_dim N
            if io == "f32":
                most /= 4
            L = _log_int(rng, 1, max(2, min(20000 if op == "heads_fwd" else 3000,
                                            int(most / (batch * heads * head_dim * N)))))
            lens = ""
            if rng.random() < 0.4:
                batch, L = 1, min(batch * L, 8000)
                lens = _cut(rng, L)
            c = _heads(op, "", io, batch, L, heads, head_dim, groups, N, lens, rng.random() < 0.5)
    elif op.startswith("conv"):
        channels = _log_int(rng, 8, 5376)
        if rng.random() < 0.6:
            channels = (channels + 7) // 8 * 8
        W = rng.choice([4, 4, 4, 3, 2, 1])
        if op == "conv_update":
            c = _conv(op, "", io, _log_int(rng, 1, 300), 1, channels, W)
        else:
            batch = rng.randint(1, 8)
            L = _log_int(rng, 1, min(30000, 44_000_000 // (channels * batch)))
            lens = ""
            if rng.random() < 0.4:
                batch, L = 1, min(batch * L, 30000)
                lens = _cut(rng, L)
            c = _conv(op, "", io, batch, L, channels, W, lens, rng.random() < 0.5)
    else:
        group = _log_int(rng, 8, 8192)
        if rng.random() < 0.7:
            group = (group + 7) // 8 * 8
        d = group * rng.choice([1, 1, 1, 2])
        rows = _log_int(rng, 1, min(16384, 42_000_000 // d))
        c = _norm(op, "", io, rows, d, group, rng.choice(["", "io", "f32"]), rng.random() < 0.5,
                  rng.choice([0, 0, 128, group]) if op == "norm_fwd" else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lens(c):
    return [int(v) for v in c["lens"].split(",")] if c["lens"] else None


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    io = TYPES[c["io"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    s = {"case": c}
    lens = _lens(c) if "lens" in c else None
    rows = len(lens) if lens else c.get("batch")
    if lens:
        s["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=DEV)
    if c["op"].startswith("heads"):
        b, L, H, P, G, N = (c[k] for k in ("batch", "L", "heads", "head_dim", "groups", "N"))
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        s["A"] = -uniform(1.0, 16.0, H)
        s["D"] = normal(H)
        s["delta_bias"] = torch.log(torch.expm1(step))
        # u, B and C are pieces of the convolution's output, delta the last
        # columns of the projection's
        xbc = normal(b, L, H * P + 2 * G * N, dtype=io)
        proj = normal(b, L, H * P + H, dtype=io, scale=0.5)
        s["u"] = xbc[..., :H * P].unflatten(-1, (H, P))
        s["B"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["C"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
        s["delta"] = proj[..., H * P:]
        if c["op"] == "heads_update":
            slots = b + 3
            s["state"] = normal(slots, H, P, N)
            s["slots"] = torch.randperm(slots, generator=g, device=DEV)[:b].to(torch.int32)
            for k in ("u", "B", "C", "delta"):
                s[k] = s[k][:, 0]
        else:
            s["h0"] = normal(rows, H, P, N) if c["state"] else None
            if c["op"] == "heads_bwd":
                s["dy"] = normal(b, L, H, P, dtype=io)
                s["dlast"] = normal(rows, H, P, N) if c["state"] else None
    elif c["op"].startswith("conv"):
        b, L, ch, W = (c[k] for k in ("batch", "L", "channels", "W"))
        s["weight"] = uniform(-1.0, 1.0, ch, W) / math.sqrt(W)
        s["bias"] = normal(ch, scale=0.1)
        # the convolution's input lies between other columns of the projection
        proj = normal(b, L, ch + 64, dtype=io)
        s["x"] = proj[..., 32:32 + ch]
        if c["op"] == "conv_update":
            slots = b + 3
            s["conv_state"] = normal(slots, ch, W - 1)
            s["slots"] = torch.randperm(slots, generator=g, device=DEV)[:b].to(torch.int32)
            s["x"] = s["x"][:, 0]
        else:
            s["conv_state"] = normal(rows, ch, W - 1) if c["state"] else None
            if c["op"] == "conv_bwd":
                s["dy"] = normal(b, L, ch, dtype=io)
    else:
        r, d = c["rows"], c["d"]
        res = {"": None, "io": io, "f32": torch.float32}[c["residual"]]
        s["weight"] = 1.0 + normal(d, scale=0.1)
        # the gate lies beside other columns of the projection
        s["z"] = normal(r, d + 64, dtype=io)[:, :d] if c["gate"] else None
        if c["op"] == "norm_fwd":
            s["x"] = normal(r, d, dtype=io)
            s["residual"] = normal(r, d, dtype=res, scale=2.0) if res else None
        else:
            # what was normed: the sum with the residual, in its type
            s["x"] = normal(r, d, dtype=res or io, scale=2.0)
            s["dresidual"] = normal(r, d, dtype=res) if res else None
            s["dy"] = normal(r, d, dtype=io)
    return s


# -------------------------------------------------------------- plain forms

def _silu(v):
    return v * torch.sigmoid(v)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _pad_index(lens):
    """Places (sequence, token) -> packed token, and which of them are real."""
    n = torch.tensor(lens, device=DEV)
    at = torch.cumsum(n, 0) - n
    t = torch.arange(max(max(lens), 1), device=DEV)
    real = t[None, :] < n[:, None]
    return torch.where(real, at[:, None] + t[None, :], 0), real


def _scan_dense(u, dt, A, B, C, D, h0):
    """The scan of rows of one length in pieces of 128 tokens: u (b, L, H, P),
    dt (b, L, H) the step sizes, B and C (b, L, G, N), all float32.  A piece
    with step sizes of zero leaves the state as it is."""
    b, L, H, P = u.shape
    G, N = B.shape[2:]
    Q = 128
    J = -(-L // Q)
    fill = J * Q - L

    def pieces(v):
        v = torch.cat([v, v.new_zeros((b, fill) + v.shape[2:])], 1) if fill else v
        return v.reshape((b, J, Q) + v.shape[2:])

    uq, dq = pieces(u), pieces(dt).permute(0, 1, 3, 2)                # (b,J,H,Q)
    Bq = pieces(B).permute(0, 1, 3, 2, 4)                             # (b,J,G,Q,N)
    Cq = pieces(C).permute(0, 1, 3, 2, 4)
    uq = uq.permute(0, 1, 3, 2, 4)                                    # (b,J,H,Q,P)
    s = torch.cumsum(dq.double() * A.double()[:, None], -1)           # log decay in the piece
    lower = torch.ones(Q, Q, dtype=torch.bool, device=u.device).tril()
    gap = torch.where(lower, s[..., :, None] - s[..., None, :], -math.inf)
    M = torch.exp(gap.float()) * dq[..., None, :]
    M = (M.unflatten(2, (G, H // G)) * (Cq @ Bq.transpose(-1, -2))[:, :, :, None]).flatten(2, 3)
    y = M @ uq
    tail = torch.exp((s[..., -1:] - s).float()) * dq                  # to the piece's end
    Bh = Bq[:, :, :, None].expand(b, J, G, H // G, Q, N).reshape(b, J, H, Q, N)
    add = (uq * tail[..., None]).transpose(-1, -2) @ Bh               # (b,J,H,P,N)
    # states entering the pieces, and the one after the last
    S = torch.cumsum(s[..., -1], 1).permute(0, 2, 1)                  # (b,H,J)
    S = torch.cat([S.new_zeros(b, H, 1), S], -1)
    low = torch.ones(J + 1, J + 1, dtype=torch.bool, device=u.device).tril()
    carry = torch.exp(torch.where(low, S[..., :, None] - S[..., None, :], -math.inf).float())
    first = h0 if h0 is not None else add.new_zeros(b, H, P, N)
    every = torch.cat([first[:, None], add], 1).permute(0, 2, 1, 3, 4).flatten(3)
    h = (carry @ every).unflatten(-1, (P, N)).permute(0, 2, 1, 3, 4)  # (b,J+1,H,P,N)
    Ch = Cq[:, :, :, None].expand(b, J, G, H // G, Q, N).reshape(b, J, H, Q, N)
    y = y + torch.exp(s.float())[..., None] * (Ch @ h[:, :-1].transpose(-1, -2))
    y = y.permute(0, 1, 3, 2, 4).reshape(b, J * Q, H, P)[:, :L] + D[:, None] * u
    return y, h[:, -1]


def _scan(u, delta, A, B, C, D, bias, h0, lens):
    dt = _softplus(delta + bias)
    if lens is None:
        return _scan_dense(u, dt, A, B, C, D, h0)
    at, real = _pad_index(lens)
    y, last = _scan_dense(u[0, at], dt[0, at] * real[..., None], A, B[0, at], C[0, at], D, h0)
    return y[real][None], last


def _taps(x, state, W, lens):
    """The W inputs that each token's output is made of: (b, L, channels, W)."""
    if lens is None:
        b, L, ch = x.shape
        before = x.new_zeros(b, W - 1, ch) if state is None else state.transpose(1, 2)
        return torch.cat([before, x], 1).unfold(1, W, 1)
    at, real = _pad_index(lens)
    return _taps(x[0, at], state, W, None)[real][None]


def _conv_last(x, state, W, lens):
    """The last W - 1 inputs of each sequence, zeros or the state before it."""
    if lens is None:
        b, L, ch = x.shape
        before = x.new_zeros(b, W - 1, ch) if state is None else state.transpose(1, 2)
        return torch.cat([before, x], 1)[:, L:].transpose(1, 2).contiguous()
    n = torch.tensor(lens, device=DEV)
    at, real = _pad_index(lens)
    before = x.new_zeros(len(lens), W - 1, x.shape[2]) if state is None else state.transpose(1, 2)
    every = torch.cat([before, x[0, at]], 1)
    take = n[:, None] + torch.arange(W - 1, device=DEV)
    return every[torch.arange(len(lens), device=DEV)[:, None], take].transpose(1, 2).contiguous()


def _normed(x, weight, z, group):
    g = x if z is None else x * _silu(z)
    v = g.unflatten(-1, (-1, group))
    return (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5)).flatten(-2) * weight


def _grads(out, wrt, by):
    return torch.autograd.grad(out, wrt, by)


def _leaf(v):
    return None if v is None else v.float().detach().requires_grad_()


def _plain(s):
    c = s["case"]
    io = TYPES[c["io"]]
    f = {k: v.float() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    lens = _lens(c) if "lens" in c else None
    if c["op"] == "heads_fwd":
        y, last = _scan(f["u"], f["delta"], f["A"], f["B"], f["C"], f["D"], f["delta_bias"],
                        f["h0"], lens)
        return {"y": y.to(io), "last_state": last}
    if c["op"] == "heads_bwd":
        p = {k: _leaf(s[k]) for k in ("u", "delta", "A", "B", "C", "D", "delta_bias", "h0")}
        y, last = _scan(p["u"], p["delta"], p["A"], p["B"], p["C"], p["D"], p["delta_bias"],
                        p["h0"], lens)
        outs, by = [y], [f["dy"]]
        if s["dlast"] is not None:
            outs, by = [y, last], [f["dy"], s["dlast"]]
        keys = [k for k in p if p[k] is not None]
        d = dict(zip(keys, _grads(outs, [p[k] for k in keys], by)))
        out = {"du": d["u"].to(io), "ddelta": d["delta"].to(io), "dB": d["B"].to(io),
               "dC": d["C"].to(io), "dA": d["A"], "dD": d["D"], "ddelta_bias": d["delta_bias"]}
        if "h0" in d:
            out["dh0"] = d["h0"]
        return out
    if c["op"] == "heads_update":
        at, state = s["slots"].long(), s["state"]
        dt = _softplus(f["delta"] + f["delta_bias"])
        per = c["heads"] // c["groups"]
        B, C = (f[k].repeat_interleave(per, 1)[:, :, None] for k in ("B", "C"))
        h = (torch.exp(dt * f["A"])[..., None, None] * state[at]
             + (dt[..., None] * f["u"])[..., None] * B)
        state[at] = h
        y = (h * C).sum(-1) + f["D"][:, None] * f["u"]
        return {"y": y.to(io), "state": state}
    if c["op"] == "conv_fwd":
        v = (_taps(f["x"], f["conv_state"], c["W"], lens) * f["weight"]).sum(-1) + f["bias"]
        return {"y": _silu(v).to(io), "last": _conv_last(f["x"], f["conv_state"], c["W"], lens)}
    if c["op"] == "conv_bwd":
        p = {k: _leaf(s[k]) for k in ("x", "weight", "bias", "conv_state")}
        v = (_taps(p["x"], p["conv_state"], c["W"], lens) * p["weight"]).sum(-1) + p["bias"]
        keys = [k for k in p if p[k] is not None]
        d = dict(zip(keys, _grads([_silu(v)], [p[k] for k in keys], [f["dy"]])))
        out = {"dx": d["x"].to(io), "dweight": d["weight"], "dbias": d["bias"]}
        if "conv_state" in d:
            out["dconv_state"] = d["conv_state"]
        return out
    if c["op"] == "conv_update":
        at, state = s["slots"].long(), s["conv_state"]
        taps = torch.cat([state[at], f["x"][..., None]], -1)
        state[at] = taps[..., 1:]
        return {"y": _silu((taps * f["weight"]).sum(-1) + f["bias"]).to(io), "conv_state": state}
    if c["op"] == "norm_fwd":
        out = {}
        x = f["x"]
        if s["residual"] is not None:
            out["residual"] = (x + f["residual"]).to(s["residual"].dtype)
            x = out["residual"].float()
        y = _normed(x, f["weight"], f["z"], c["group"])
        if not c["block"]:
            return {**out, "y": y.to(io)}
        # 8 bits: one scale for each block of a group, the last block of a
        # group may be short
        v = y.unflatten(-1, (-1, c["group"]))
        n = -(-c["group"] // c["block"])
        v = torch.cat([v, v.new_zeros(v.shape[:-1] + (n * c["block"] - c["group"],))], -1)
        v = v.unflatten(-1, (n, c["block"]))
        most = v.abs().amax(-1, keepdim=True)
        q = (v * (FP8_MAX / most)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        q = q.flatten(-2)[..., :c["group"]].reshape(y.shape).contiguous()
        return {**out, "y": q, "scale": (most / FP8_MAX).reshape(y.shape[0], -1)}
    # norm_bwd
    p = {k: _leaf(s[k]) for k in ("x", "weight", "z")}
    keys = [k for k in p if p[k] is not None]
    y = _normed(p["x"], p["weight"], p["z"], c["group"])
    d = dict(zip(keys, _grads([y], [p[k] for k in keys], [f["dy"]])))
    dx = d["x"] if s["dresidual"] is None else d["x"] + f["dresidual"]
    out = {"dx": dx.to(s["x"].dtype), "dweight": d["weight"]}
    if "z" in d:
        out["dz"] = d["z"].to(io)
    return out


# ------------------------------------------------------------ the package's

def _own(s):
    import selective_state_space_fwd_amd as ssm
    op = s["case"]["op"]
    if op == "heads_fwd":
        y, last = ssm.ssm_heads_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"],
                                    s["delta_bias"], initial_state=s["h0"],
                                    cu_seqlens=s.get("cu"))
        return {"y": y, "last_state": last}
    if op == "heads_bwd":
        d = ssm.ssm_heads_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dy"], s["D"],
                              s["delta_bias"], initial_state=s["h0"], dlast=s["dlast"],
                              cu_seqlens=s.get("cu"))
        return {k: v for k, v in d.items() if v is not None}
    if op == "heads_update":
        y = ssm.ssm_heads_update(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"],
                                 s["delta_bias"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "conv_fwd":
        y, last = ssm.ssm_conv_fwd(s["x"], s["weight"], s["bias"], conv_state=s["conv_state"],
                                   cu_seqlens=s.get("cu"))
        return {"y": y, "last": last}
    if op == "conv_bwd":
        d = ssm.ssm_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], conv_state=s["conv_state"],
                             cu_seqlens=s.get("cu"))
        return {k: v for k, v in d.items() if v is not None}
    if op == "conv_update":
        y = ssm.ssm_conv_update(s["conv_state"], s["x"], s["weight"], s["bias"],
                                slots=s["slots"])
        return {"y": y, "conv_state": s["conv_state"]}
    group = s["case"]["group"]
    if op == "norm_fwd":
        y, scale, residual = ssm.ssm_norm_fwd(s["x"], s["weight"], residual=s["residual"],
                                              z=s["z"], group_size=group,
                                              quant_block=s["case"]["block"])
        out = {"y": y, "scale": scale, "residual": residual}
        return {k: v for k, v in out.items() if v is not None}
    d = ssm.ssm_norm_bwd(s["x"], s["weight"], s["dy"], z=s["z"], dresidual=s["dresidual"],
                         group_size=group)
    return {k: v for k, v in d.items() if v is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the work

def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    rows = len(_lens(c)) if c.get("lens") else c.get("batch", 0)
    if c["op"].startswith("heads"):
        b, L, H, P, G, N = (c[k] for k in ("batch", "L", "heads", "head_dim", "groups", "N"))
        T = b * L
        inputs = T * (H * P + H + 2 * G * N) * e
        if c["op"] == "heads_update":
            return {"bytes": inputs + T * H * P * e + 2 * T * H * P * N * 4,
                    "flops": 7 * T * H * P * N}
        state = rows * H * P * N * 4
        # the recurrence itself: the state's update and the output, a product
        # and a sum each for every token, channel and state
        if c["op"] == "heads_fwd":
            return {"bytes": inputs + T * H * P * e + state * (2 if c["state"] else 1),
                    "flops": 4 * T * H * P * N}
        # states again, their gradients, and the gradients of u, B and C
        return {"bytes": 2 * inputs + T * H * P * e + (3 * state if c["state"] else 0),
                "flops": 10 * T * H * P * N}
    if c["op"].startswith("conv"):
        n = c["batch"] * c["L"] * c["channels"]
        state = rows * c["channels"] * (c["W"] - 1) * 4
        if c["op"] == "conv_fwd":
            return {"bytes": 2 * n * e + state * (2 if c["state"] else 1),
                    "flops": n * (2 * c["W"] + 5)}
        if c["op"] == "conv_update":
            return {"bytes": 2 * n * e + 2 * state, "flops": n * (2 * c["W"] + 5)}
        return {"bytes": 3 * n * e + (2 * state if c["state"] else 0),
                "flops": n * (6 * c["W"] + 10)}
    n = c["rows"] * c["d"]
    r = {"": 0, "io": e, "f32": 4}[c["residual"]]
    z = e if c["gate"] else 0
    if c["op"] == "norm_fwd":
        out = 1 + 4 / c["block"] if c["block"] else e
        return {"bytes": n * (e + z + 2 * r + out) + c["d"] * 4, "flops": 12 * n}
    return {"bytes": n * (2 * (r or e) + e + 2 * z + r) + 2 * c["d"] * 4, "flops": 24 * n}


# ------------------------------------------------------ definitions, 64 bits

def _exact_silu(v):
    return v / (1 + torch.exp(-v))


def _exact_scan(u, dt, A, B, C, D, h):
    """Token by token: h = exp(dt A) h + dt u B', y = h C + D u."""
    b, L, H, P = u.shape
    per = H // B.shape[2]
    y = torch.empty_like(u)
    decay = torch.exp(dt * A)
    w = dt[..., None] * u
    for t in range(L):
        Bt = B[:, t].repeat_interleave(per, 1)
        Ct = C[:, t].repeat_interleave(per, 1)
        h = torch.addcmul(decay[:, t, :, None, None] * h, w[:, t, :, :, None], Bt[:, :, None, :])
        y[:, t] = torch.matmul(h, Ct[..., None])[..., 0] + D[:, None] * u[:, t]
    return y, h


def _exact_head(u, dt, A, B, C, D, h0):
    """One sequence of one head as a masked product over its whole length:
    u (L, P), dt (L), B and C (L, N), h0 (P, N)."""
    s = torch.cumsum(dt * A, 0)
    seen = torch.ones(len(dt), len(dt), dtype=torch.bool, device=u.device).tril()
    W = torch.where(seen, s[:, None] - s[None, :], -math.inf).exp() * dt
    y = ((C @ B.T) * W) @ u + s.exp()[:, None] * (C @ h0.T) + D * u
    end = s[-1] if len(dt) else s.new_zeros(())
    last = end.exp() * h0 + (u * (dt * torch.exp(end - s))[:, None]).T @ B
    return y, last


def _exact_heads_bwd(s, f, spans):
    H, P = f["u"].shape[2:]
    N = f["B"].shape[3]
    per = H // f["B"].shape[2]
    d = {k: torch.zeros_like(f[k]) for k in ("u", "delta", "A", "B", "C", "D", "delta_bias")}
    d["h0"] = torch.zeros(len(spans), H, P, N, dtype=torch.float64, device=DEV)
    for r, (b, i, j) in enumerate(spans):
        for h in range(H):
            g = h // per
            h0 = f["h0"][r, h] if f["h0"] is not None else d["h0"].new_zeros(P, N)
            leaf = [v.detach().clone().requires_grad_() for v in
                    (f["u"][b, i:j, h], f["delta"][b, i:j, h], f["A"][h], f["B"][b, i:j, g],
                     f["C"][b, i:j, g], f["D"][h], f["delta_bias"][h], h0)]
            u, delta, A, B, C, D, bias, start = leaf
            dt = torch.log1p(torch.exp(delta + bias))
            y, last = _exact_head(u, dt, A, B, C, D, start)
            loss = (y * f["dy"][b, i:j, h]).sum()
            if f["dlast"] is not None:
                loss = loss + (last * f["dlast"][r, h]).sum()
            got = torch.autograd.grad(loss, leaf, allow_unused=True)
            got = [torch.zeros_like(v) if w is None else w for v, w in zip(leaf, got)]
            d["u"][b, i:j, h], d["delta"][b, i:j, h] = got[0], got[1]
            d["A"][h] += got[2]
            d["B"][b, i:j, g] += got[3]
            d["C"][b, i:j, g] += got[4]
            d["D"][h] += got[5]
            d["delta_bias"][h] += got[6]
            d["h0"][r, h] = got[7]
    out = {"d" + k: d[k] for k in ("u", "delta", "A", "B", "C", "D", "delta_bias")}
    if f["h0"] is not None:
        out["dh0"] = d["h0"]
    return out


def _exact_conv(x, weight, bias, state, spans):
    """Sequence by sequence, tap by tap; the pre-activation and the last inputs."""
    ch, W = weight.shape
    v = torch.zeros_like(x) + bias
    last = x.new_zeros(len(spans), ch, W - 1)
    for r, (b, i, j) in enumerate(spans):
        before = x.new_zeros(W - 1, ch) if state is None else state[r].T
        line = torch.cat([before, x[b, i:j]])
        for k in range(W):
            v[b, i:j] = v[b, i:j] + weight[:, k] * line[k:k + j - i]
        last[r] = line[j - i:].T
    return v, last


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if c["op"].startswith(("heads", "conv")):
        lens = _lens(c)
        at = _offsets(lens) if lens else None
        spans = ([(0, i, j) for i, j in zip(at, at[1:])] if lens
                 else [(b, 0, c["L"]) for b in range(c["batch"])])
    if c["op"] == "heads_fwd":
        dt = torch.log1p(torch.exp(f["delta"] + f["delta_bias"]))
        H, P, N = c["heads"], c["head_dim"], c["N"]
        h0 = f["h0"] if f["h0"] is not None else f["u"].new_zeros(len(spans), H, P, N)
        if not lens:
            y, last = _exact_scan(f["u"], dt, f["A"], f["B"], f["C"], f["D"], h0)
            return {"y": y, "last_state": last}
        parts = [_exact_scan(f["u"][:, i:j], dt[:, i:j], f["A"], f["B"][:, i:j], f["C"][:, i:j],
                             f["D"], h0[r:r + 1]) for r, (_, i, j) in enumerate(spans)]
        return {"y": torch.cat([p[0] for p in parts], 1),
                "last_state": torch.cat([p[1] for p in parts])}
    if c["op"] == "heads_bwd":
        return _exact_heads_bwd(s, f, spans)
    if c["op"] == "heads_update":
        dt = torch.log1p(torch.exp(f["delta"] + f["delta_bias"]))
        state = f["state"].clone()
        rows = s["slots"].long()
        y, h = _exact_scan(f["u"][:, None], dt[:, None], f["A"], f["B"][:, None], f["C"][:, None],
                           f["D"], state[rows])
        state[rows] = h
        return {"y": y[:, 0], "state": state}
    if c["op"] == "conv_fwd":
        v, last = _exact_conv(f["x"], f["weight"], f["bias"], f["conv_state"], spans)
        return {"y": _exact_silu(v), "last": last}
    if c["op"] == "conv_bwd":
        v, _ = _exact_conv(f["x"], f["weight"], f["bias"], f["conv_state"], spans)
        sig = 1 / (1 + torch.exp(-v))
        dv = f["dy"] * sig * (1 + v * (1 - sig))
        W = c["W"]
        dx, dw = torch.zeros_like(f["x"]), torch.zeros_like(f["weight"])
        dstate = dx.new_zeros(len(spans), c["channels"], W - 1)
        for r, (b, i, j) in enumerate(spans):
            n = j - i
            before = dx.new_zeros(W - 1, c["channels"])
            if f["conv_state"] is not None:
                before = f["conv_state"][r].T
            line = torch.cat([before, f["x"][b, i:j]])
            dline = torch.zeros_like(line)
            for k in range(W):
                dline[k:k + n] += f["weight"][:, k] * dv[b, i:j]
                dw[:, k] += (line[k:k + n] * dv[b, i:j]).sum(0)
            dx[b, i:j] = dline[W - 1:]
            dstate[r] = dline[:W - 1].T
        out = {"dx": dx, "dweight": dw, "dbias": dv.sum((0, 1))}
        if f["conv_state"] is not None:
            out["dconv_state"] = dstate
        return out
    if c["op"] == "conv_update":
        state = f["conv_state"].clone()
        rows = s["slots"].long()
        v, last = _exact_conv(f["x"][:, None], f["weight"], f["bias"], state[rows], spans)
        state[rows] = last
        return {"y": _exact_silu(v[:, 0]), "conv_state": state}
    x, group = f["x"], c["group"]
    out = {}
    if c["op"] == "norm_fwd" and f["residual"] is not None:
        out["residual"] = x + f["residual"]
        x = out["residual"].to(s["residual"].dtype).double()   # the norm is of the rounded sum
    gate = 1.0 if f["z"] is None else _exact_silu(f["z"])
    v = (x * gate).reshape(c["rows"], -1, group)
    root = torch.sqrt((v * v).sum(-1, keepdim=True) / group + 1e-5)
    n = (v / root).reshape(x.shape)
    if c["op"] == "norm_fwd":
        y = n * f["weight"]
        if not c["block"]:
            return {**out, "y": y}
        q, scales = torch.empty_like(y), []
        for g in range(c["d"] // group):
            for i in range(g * group, (g + 1) * group, c["block"]):
                j = min(i + c["block"], (g + 1) * group)
                sc = y[:, i:j].abs().amax(1) / FP8_MAX
                q[:, i:j] = y[:, i:j] / sc[:, None]
                scales.append(sc)
        return {**out, "y": q, "scale": torch.stack(scales, 1)}
    dn = f["dy"] * f["weight"]
    mean = (dn * n).reshape(v.shape).sum(-1, keepdim=True) / group
    dg = ((dn.reshape(v.shape) - n.reshape(v.shape) * mean) / root).reshape(x.shape)
    dx = dg * gate
    if f["dresidual"] is not None:
        dx = dx + f["dresidual"]
    out = {"dx": dx, "dweight": (f["dy"] * n).sum(0)}
    if f["z"] is not None:
        sig = 1 / (1 + torch.exp(-f["z"]))
        out["dz"] = dg * x * sig * (1 + f["z"] * (1 - sig))
    return out
