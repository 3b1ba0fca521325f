"""The layer operators of libssm: the scan over heads, the short causal
convolution in front of it and the root-mean-square norm, each for prompts,
for single tokens and with its gradients.

Activations are token-major: (batch, tokens, ...), the channels of a token
side by side, as a projection leaves them.  Inputs may be columns of a wider
tensor (any distance from token to token); outputs are dense.  Gradients of
activations have the activations' type, those of parameters and states are
float32.  Like the scan's, these functions check and marshal only: every step
runs in the HIP kernels of libssm.

    y, last_conv = ssm_conv_fwd(x, weight, bias)
    y, last = ssm_heads_fwd(u, delta, A, B, C, D, delta_bias)
    y, scale, residual = ssm_norm_fwd(x, weight, residual=r, z=z, quant_block=128)
"""
from __future__ import annotations

import ctypes

__all__ = ["ssm_heads_fwd", "ssm_heads_bwd", "ssm_heads_update",
           "ssm_conv_fwd", "ssm_conv_bwd", "ssm_conv_update", "ssm_norm_fwd", "ssm_norm_bwd"]

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class HeadsDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in (
        "batch", "seqlen", "heads", "head_dim", "groups", "d_state", "n_seqs",
        "u_batch_stride", "u_token_stride", "delta_batch_stride", "delta_token_stride",
        "B_batch_stride", "B_token_stride", "C_batch_stride", "C_token_stride",
        "dy_batch_stride", "dy_token_stride")] + [
        ("io_dtype", _i32), ("softplus", _i32), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t), ("flags", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32)]


class ConvDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in (
        "batch", "seqlen", "channels", "n_seqs", "x_batch_stride", "x_token_stride",
        "dy_batch_stride", "dy_token_stride")] + [
        ("width", _i32), ("io_dtype", _i32), ("silu", _i32), ("reserved", _i32),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("flags", ctypes.c_uint64)]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in (
        "rows", "d", "group_size", "quant_block", "x_stride", "z_stride", "residual_stride",
        "dy_stride")] + [
        ("io_dtype", _i32), ("residual_dtype", _i32), ("eps", ctypes.c_float),
        ("reserved", _i32), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("flags", ctypes.c_uint64)]


def declare(lib):
    """Argument and result types of the layer entry points."""
    vp, sz = _vp, ctypes.c_size_t
    hd, cd, nd = (ctypes.POINTER(t) for t in (HeadsDesc, ConvDesc, NormDesc))
    for name, args, res in (
            ("ssm_heads_workspace_bytes", [hd, ctypes.c_int], sz),
            ("ssm_heads_fwd", [hd] + [vp] * 12, ctypes.c_int),
            ("ssm_heads_bwd", [hd] + [vp] * 20, ctypes.c_int),
            ("ssm_heads_update", [hd, vp, vp, _i64] + [vp] * 9, ctypes.c_int),
            ("ssm_conv_workspace_bytes", [cd], sz),
            ("ssm_conv_fwd", [cd] + [vp] * 8, ctypes.c_int),
            ("ssm_conv_bwd", [cd] + [vp] * 11, ctypes.c_int),
            ("ssm_conv_update", [cd, vp, vp, _i64] + [vp] * 5, ctypes.c_int),
            ("ssm_norm_workspace_bytes", [nd], sz),
            ("ssm_norm_fwd", [nd] + [vp] * 8, ctypes.c_int),
            ("ssm_norm_bwd", [nd] + [vp] * 9, ctypes.c_int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


from . import PreparedCall, _check, _io_code, load_library  # noqa: E402

_torch = None


def _t():
    """torch, imported by the first call."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


class _LayerCall(PreparedCall):
    """A PreparedCall that makes the tensors' device current for the launch."""

    __slots__ = ("_device",)

    def __call__(self, profile_events=None, stream=None):
        if profile_events is not None:
            raise ValueError("the layer entry points record no events")
        cuda = _t().cuda
        if self._device.index == cuda.current_device():
            return super().__call__(None, stream)
        with cuda.device(self._device):
            return super().__call__(None, stream)


def _issue(prepare, fn, desc, args, keep, result, device):
    cuda = _t().cuda
    stream = cuda.current_stream(device).cuda_stream
    if prepare:
        call = _LayerCall(fn, desc, args + (stream,), keep, result)
        call._device = device
        return call
    if device.index == cuda.current_device():
        status = fn(ctypes.byref(desc), *args, stream)
    else:
        with cuda.device(device):
            status = fn(ctypes.byref(desc), *args, stream)
    if status:
        _check(status)
    return result


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t, name, shape, dtype, device):
    """Checks a shape (a tuple), a type and a device."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")


def _expect(t, name, shape, dtype, device):
    if t is None:
        return
    _like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, dtype, device, inner):
    """Checks an activation whose last `inner` dimensions lie side by side, as
    columns of rows any distance apart; returns its leading strides."""
    _like(t, name, shape, dtype, device)
    st, want, n = t.stride(), 1, len(shape)
    for i in range(n - 1, n - 1 - inner, -1):
        if st[i] != want and shape[i] != 1:
            raise ValueError(f"{name}: the last {inner} dimension(s) must be contiguous")
        want *= shape[i]
    # the distance between rows of which there is one does not matter
    lead = st[:n - inner]
    return lead if 1 not in shape[:n - inner] else tuple(
        0 if shape[i] == 1 else lead[i] for i in range(n - inner))


def _offsets(cu_seqlens, batch, device):
    if cu_seqlens is None:
        return 0, batch
    torch = _t()
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold n_seqs + 1 >= 2 offsets")
    n = cu_seqlens.numel() - 1
    _expect(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, device)
    if batch != 1:
        raise ValueError("packed sequences lie in one batch row")
    return n, n


def _room(need, workspace, desc, device):
    if need == 0:
        return None
    if workspace is None:
        workspace = _t().empty(need, dtype=_t().uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on {device}")
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a GPU tensor, got {t.device}")
    return t.device


# ------------------------------------------------------------ scan over heads

def _heads_desc(u, delta, A, B, C, D, delta_bias, softplus, tokens):
    """Checks what every form of the scan over heads takes; tokens: whether a
    token dimension follows the batch's."""
    torch = _t()
    if u.dim() != 3 + tokens:
        raise ValueError(f"u: expected {3 + tokens} dimensions, got {tuple(u.shape)}")
    if B.dim() != 3 + tokens:
        raise ValueError(f"B: expected {3 + tokens} dimensions, got {tuple(B.shape)}")
    lead = tuple(u.shape[:1 + tokens])
    H, P = u.shape[-2:]
    G, N = B.shape[-2:]
    dev, io = _cuda(u, "u"), u.dtype
    us = _rows(u, "u", lead + (H, P), io, dev, 2)
    ds = _rows(delta, "delta", lead + (H,), io, dev, 1)
    bs = _rows(B, "B", lead + (G, N), io, dev, 2)
    cs = _rows(C, "C", lead + (G, N), io, dev, 2)
    f32 = torch.float32
    _expect(A, "A", (H,), f32, dev)
    _expect(D, "D", (H,), f32, dev)
    _expect(delta_bias, "delta_bias", (H,), f32, dev)
    if not tokens:
        us, ds, bs, cs = us + (0,), ds + (0,), bs + (0,), cs + (0,)
    desc = HeadsDesc(lead[0], lead[1] if tokens else 1, H, P, G, N, 0, us[0], us[1], ds[0], ds[1],
                     bs[0], bs[1], cs[0], cs[1], 0, 0, _io_code(io), 1 if softplus else 0)
    return desc, dev, io, lead


def ssm_heads_fwd(u, delta, A, B, C, D=None, delta_bias=None, softplus=True,
                  return_last_state=True, initial_state=None, cu_seqlens=None, y=None,
                  last_state=None, workspace=None, prepare=False):
    """The scan over heads: h_t = exp(dt_t A) h_{t-1} + dt_t u_t (x) B_t,
    y_t = h_t C_t + D u_t, with dt = softplus(delta + delta_bias).

    u: (batch, L, heads, head_dim); delta: (batch, L, heads); B, C: (batch, L,
    groups, d_state), float32 or bfloat16; head h uses group h // (heads //
    groups).  A, D, delta_bias: (heads,) float32.  initial_state: (rows, heads,
    head_dim, d_state) float32, or None for zeros; rows = batch, or the number
    of packed sequences.  cu_seqlens: int32 offsets of sequences packed in one
    batch row; tokens behind the last are left out, and their y as it was.
    prepare: check and marshal only, return a PreparedCall.
    Returns (y, last_state); last_state is None unless requested.
    """
    torch = _t()
    lib = load_library()
    desc, dev, io, lead = _heads_desc(u, delta, A, B, C, D, delta_bias, softplus, 1)
    desc.n_seqs, rows = _offsets(cu_seqlens, lead[0], dev)
    state = (rows, desc.heads, desc.head_dim, desc.d_state)
    _expect(initial_state, "initial_state", state, torch.float32, dev)
    if y is None:
        y = u.new_empty(u.shape)
    _expect(y, "y", u.shape, io, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty(state, dtype=torch.float32, device=dev)
    _expect(last_state, "last_state", state, torch.float32, dev)
    need = lib.ssm_heads_workspace_bytes(ctypes.byref(desc), 0)
    workspace = _room(need, workspace, desc, dev)
    args = tuple(map(_ptr, (u, delta, A, B, C, D, delta_bias, initial_state, cu_seqlens, y,
                            last_state)))
    keep = (u, delta, A, B, C, D, delta_bias, initial_state, cu_seqlens, workspace)
    return _issue(prepare, lib.ssm_heads_fwd, desc, args, keep, (y, last_state), dev)


def ssm_heads_bwd(u, delta, A, B, C, dy, D=None, delta_bias=None, softplus=True,
                  initial_state=None, dlast=None, cu_seqlens=None, workspace=None, prepare=False):
    """Gradients of sum(dy * y) + sum(dlast * last_state) of ssm_heads_fwd.

    Returns a dict: du, ddelta (of the raw delta), dB, dC in the inputs' type;
    dA, dD (None without D), ddelta_bias (None without delta_bias), dh0 (None
    without initial_state) float32.  Nothing of the forward call is needed;
    other arguments as there.
    """
    torch = _t()
    lib = load_library()
    desc, dev, io, lead = _heads_desc(u, delta, A, B, C, D, delta_bias, softplus, 1)
    desc.dy_batch_stride, desc.dy_token_stride = _rows(dy, "dy", tuple(u.shape), io, dev, 2)
    desc.n_seqs, rows = _offsets(cu_seqlens, lead[0], dev)
    state = (rows, desc.heads, desc.head_dim, desc.d_state)
    _expect(initial_state, "initial_state", state, torch.float32, dev)
    _expect(dlast, "dlast", state, torch.float32, dev)

    def new(like, dtype, wanted=True):
        return torch.empty(like, dtype=dtype, device=dev) if wanted else None

    f32, H = torch.float32, (desc.heads,)
    out = {"du": new(u.shape, io), "ddelta": new(delta.shape, io), "dA": new(H, f32),
           "dB": new(B.shape, io), "dC": new(C.shape, io), "dD": new(H, f32, D is not None),
           "ddelta_bias": new(H, f32, delta_bias is not None),
           "dh0": new(state, f32, initial_state is not None)}
    need = lib.ssm_heads_workspace_bytes(ctypes.byref(desc), 1)
    workspace = _room(need, workspace, desc, dev)
    args = tuple(map(_ptr, (u, delta, A, B, C, D, delta_bias, initial_state, cu_seqlens, dy,
                            dlast, out["du"], out["ddelta"], out["dA"], out["dB"], out["dC"],
                            out["dD"], out["ddelta_bias"], out["dh0"])))
    keep = (u, delta, A, B, C, D, delta_bias, initial_state, cu_seqlens, dy, dlast, workspace)
    return _issue(prepare, lib.ssm_heads_bwd, desc, args, keep, out, dev)


def _slots(slots, batch, n_slots, dev):
    _expect(slots, "slots", (batch,), _t().int32, dev)
    if slots is None and batch > n_slots:
        raise ValueError(f"{batch} rows, but {n_slots} states")


def ssm_heads_update(state, u, delta, A, B, C, D=None, delta_bias=None, softplus=True,
                     slots=None, y=None, prepare=False):
    """One token of the scan over heads, ``state`` (n_slots, heads, head_dim,
    d_state) float32 updated in place.

    u: (rows, heads, head_dim); delta: (rows, heads); B, C: (rows, groups,
    d_state).  slots: int32 (rows,), the state of each row (None: row i is slot
    i); a row whose slot lies outside 0 .. n_slots - 1 is skipped, its y left
    as it was; slots of one call must differ.  Returns y (rows, heads, head_dim).
    """
    torch = _t()
    lib = load_library()
    desc, dev, io, lead = _heads_desc(u, delta, A, B, C, D, delta_bias, softplus, 0)
    n = state.shape[0]
    _expect(state, "state", (n, desc.heads, desc.head_dim, desc.d_state), torch.float32, dev)
    _slots(slots, lead[0], n, dev)
    if y is None:
        y = u.new_empty(u.shape)
    _expect(y, "y", u.shape, io, dev)
    args = (_ptr(state), _ptr(slots), n) + tuple(map(_ptr, (u, delta, A, B, C, D, delta_bias, y)))
    keep = (state, slots, u, delta, A, B, C, D, delta_bias)
    return _issue(prepare, lib.ssm_heads_update, desc, args, keep, y, dev)


# --------------------------------------------------------------- convolution

def _conv_desc(x, weight, bias, silu, tokens):
    torch = _t()
    if x.dim() != 2 + tokens:
        raise ValueError(f"x: expected {2 + tokens} dimensions, got {tuple(x.shape)}")
    ch = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != ch:
        raise ValueError(f"weight must be (channels, width), got {tuple(weight.shape)}")
    dev, io, W = _cuda(x, "x"), x.dtype, weight.shape[1]
    st = _rows(x, "x", tuple(x.shape), io, dev, 1)
    desc = ConvDesc(x.shape[0], x.shape[1] if tokens else 1, ch, 0, st[0], st[1] if tokens else 0,
                    0, 0, W, _io_code(io), 1 if silu else 0)
    _expect(weight, "weight", (ch, W), torch.float32, dev)
    _expect(bias, "bias", (ch,), torch.float32, dev)
    return desc, dev, io


def ssm_conv_fwd(x, weight, bias=None, silu=True, conv_state=None, cu_seqlens=None,
                 return_last_state=True, y=None, last_state=None, prepare=False):
    """The short causal depthwise convolution: y_t = silu(bias + sum_k
    weight[:, k] x_{t-(W-1)+k}); silu False: without the activation.

    x: (batch, L, channels); weight: (channels, W) float32, W <= 4; conv_state:
    (rows, channels, W - 1) float32 inputs before each sequence, None for
    zeros; cu_seqlens as in ssm_heads_fwd.  Returns (y, last_state), the latter
    the conv_state behind each sequence (None unless requested).
    """
    torch = _t()
    lib = load_library()
    desc, dev, io = _conv_desc(x, weight, bias, silu, 1)
    desc.n_seqs, rows = _offsets(cu_seqlens, desc.batch, dev)
    state = (rows, desc.channels, desc.width - 1)
    _expect(conv_state, "conv_state", state, torch.float32, dev)
    if y is None:
        y = x.new_empty(x.shape)
    _expect(y, "y", x.shape, io, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty(state, dtype=torch.float32, device=dev)
    _expect(last_state, "last_state", state, torch.float32, dev)
    args = tuple(map(_ptr, (x, weight, bias, conv_state, cu_seqlens, y, last_state)))
    keep = (x, weight, bias, conv_state, cu_seqlens)
    return _issue(prepare, lib.ssm_conv_fwd, desc, args, keep, (y, last_state), dev)


def ssm_conv_bwd(x, weight, dy, bias=None, silu=True, conv_state=None, cu_seqlens=None,
                 workspace=None, prepare=False):
    """Gradients of sum(dy * y) of ssm_conv_fwd: a dict of dx (in x's type) and
    float32 dweight, dbias (None without bias), dconv_state (None without
    conv_state)."""
    torch = _t()
    lib = load_library()
    desc, dev, io = _conv_desc(x, weight, bias, silu, 1)
    desc.dy_batch_stride, desc.dy_token_stride = _rows(dy, "dy", tuple(x.shape), io, dev, 1)
    desc.n_seqs, rows = _offsets(cu_seqlens, desc.batch, dev)
    _expect(conv_state, "conv_state", (rows, desc.channels, desc.width - 1), torch.float32, dev)

    def new(like, wanted=True, dtype=torch.float32):
        return torch.empty(like, dtype=dtype, device=dev) if wanted else None

    out = {"dx": new(x.shape, dtype=io), "dweight": new(weight.shape),
           "dbias": new((desc.channels,), bias is not None),
           "dconv_state": new((rows, desc.channels, desc.width - 1), conv_state is not None)}
    workspace = _room(lib.ssm_conv_workspace_bytes(ctypes.byref(desc)), workspace, desc, dev)
    args = tuple(map(_ptr, (x, weight, bias, conv_state, cu_seqlens, dy, out["dx"],
                            out["dweight"], out["dbias"], out["dconv_state"])))
    keep = (x, weight, bias, conv_state, cu_seqlens, dy, workspace)
    return _issue(prepare, lib.ssm_conv_bwd, desc, args, keep, out, dev)


def ssm_conv_update(conv_state, x, weight, bias=None, silu=True, slots=None, y=None,
                    prepare=False):
    """One token of the convolution: x (rows, channels); conv_state (n_slots,
    channels, W - 1) float32 moves on by one in place; slots as in
    ssm_heads_update.  Returns y (rows, channels)."""
    torch = _t()
    lib = load_library()
    desc, dev, io = _conv_desc(x, weight, bias, silu, 0)
    n = conv_state.shape[0]
    _expect(conv_state, "conv_state", (n, desc.channels, desc.width - 1), torch.float32, dev)
    _slots(slots, desc.batch, n, dev)
    if y is None:
        y = x.new_empty(x.shape)
    _expect(y, "y", x.shape, io, dev)
    args = (_ptr(conv_state), _ptr(slots), n) + tuple(map(_ptr, (x, weight, bias, y)))
    keep = (conv_state, slots, x, weight, bias)
    return _issue(prepare, lib.ssm_conv_update, desc, args, keep, y, dev)


# ---------------------------------------------------------------------- norm

def _norm_desc(x, weight, io, res, group_size, eps):
    torch = _t()
    if x.dim() != 2:
        raise ValueError(f"x: expected (rows, d), got {tuple(x.shape)}")
    rows, d = x.shape
    dev = _cuda(x, "x")
    group_size = group_size or d
    if group_size < 0 or d % group_size:
        raise ValueError(f"group_size {group_size} does not divide {d}")
    xs = _rows(x, "x", (rows, d), x.dtype, dev, 1)[0]
    desc = NormDesc(rows, d, group_size, 0, xs, 0, 0, 0, _io_code(io), _io_code(res), eps)
    _expect(weight, "weight", (d,), torch.float32, dev)
    return desc, dev


def ssm_norm_fwd(x, weight, residual=None, z=None, eps=1e-5, group_size=0, quant_block=0, y=None,
                 scale=None, residual_out=None, prepare=False):
    """Root-mean-square norm: s = x + residual, g = s * silu(z),
    y = g / sqrt(mean(g * g) + eps) * weight, the mean over each group of
    group_size values (0: the row).

    x, z: (rows, d), float32 or bfloat16; residual: (rows, d) in x's type or
    float32; weight: (d,) float32.  quant_block > 0: y is float8_e4m3fn with
    one float32 scale for each quant_block values of a group (the last block of
    a group may be short): y * scale is the result.  residual_out may be the
    residual.  Returns (y, scale, s): scale None without quant_block, s (in the
    residual's type) None without residual.
    """
    torch = _t()
    lib = load_library()
    desc, dev = _norm_desc(x, weight, x.dtype, x.dtype if residual is None else residual.dtype,
                           group_size, eps)
    shape, io = tuple(x.shape), x.dtype
    if z is not None:
        desc.z_stride = _rows(z, "z", shape, io, dev, 1)[0]
    if residual is not None:
        desc.residual_stride = _rows(residual, "residual", shape, residual.dtype, dev, 1)[0]
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=dev)
        _expect(residual_out, "residual_out", shape, residual.dtype, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    desc.quant_block = quant_block
    yt = torch.float8_e4m3fn if quant_block else io
    if y is None:
        y = torch.empty(shape, dtype=yt, device=dev)
    _expect(y, "y", shape, yt, dev)
    if quant_block > 0:
        blocks = -(-desc.group_size // quant_block) * (desc.d // desc.group_size)
        if scale is None:
            scale = torch.empty((desc.rows, blocks), dtype=torch.float32, device=dev)
        _expect(scale, "scale", (desc.rows, blocks), torch.float32, dev)
    elif scale is not None:
        raise ValueError("scale without quant_block")
    args = tuple(map(_ptr, (x, weight, residual, z, y, scale, residual_out)))
    return _issue(prepare, lib.ssm_norm_fwd, desc, args, (x, weight, residual, z),
                  (y, scale, residual_out), dev)


def ssm_norm_bwd(x, weight, dy, z=None, dresidual=None, eps=1e-5, group_size=0, workspace=None,
                 prepare=False):
    """Gradients of sum(dy * y) + sum(dresidual * s) of ssm_norm_fwd for x = s,
    what was normed: its returned sum, or its x without a residual.

    x may be float32 beside a bfloat16 dy; dresidual has x's type.  Returns a
    dict: dx (the gradient of x and of the residual alike, in x's type), dz
    (None without z, in dy's), dweight float32.
    """
    torch = _t()
    lib = load_library()
    desc, dev = _norm_desc(x, weight, dy.dtype, x.dtype, group_size, eps)
    shape, io = tuple(x.shape), dy.dtype
    desc.dy_stride = _rows(dy, "dy", shape, io, dev, 1)[0]
    if z is not None:
        desc.z_stride = _rows(z, "z", shape, io, dev, 1)[0]
    _expect(dresidual, "dresidual", shape, x.dtype, dev)
    out = {"dx": torch.empty(shape, dtype=x.dtype, device=dev),
           "dz": torch.empty(shape, dtype=io, device=dev) if z is not None else None,
           "dweight": torch.empty((desc.d,), dtype=torch.float32, device=dev)}
    workspace = _room(lib.ssm_norm_workspace_bytes(ctypes.byref(desc)), workspace, desc, dev)
    args = tuple(map(_ptr, (x, weight, z, dy, dresidual, out["dx"], out["dz"], out["dweight"])))
    keep = (x, weight, z, dy, dresidual, workspace)
    return _issue(prepare, lib.ssm_norm_bwd, desc, args, keep, out, dev)
