"""Host-side checks of the layer operators' C entry points and of their Python
binding: every refusal comes before a launch.  No kernel runs here."""
import ctypes

import pytest
import torch

import selective_state_space_fwd_amd as ssm
from selective_state_space_fwd_amd.layer import ConvDesc, HeadsDesc, NormDesc

OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4, 5
PTR = 4096          # an address that only its alignment is looked at of


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def heads(**kw):
    base = dict(batch=2, seqlen=300, heads=8, head_dim=64, groups=2, d_state=128, u_token_stride=512,
                u_batch_stride=512 * 300, delta_token_stride=8, delta_batch_stride=2400,
                B_token_stride=256, B_batch_stride=256 * 300, C_token_stride=256,
                C_batch_stride=256 * 300, dy_token_stride=512, dy_batch_stride=512 * 300,
                io_dtype=1, softplus=1, workspace=PTR, workspace_bytes=1 << 40)
    base.update(kw)
    return HeadsDesc(**base)


def fwd(lib, d, cu=None, **kw):
    p = dict(u=PTR, delta=PTR, A=PTR, B=PTR, C=PTR, D=None, bias=None, h0=None, cu=cu, y=PTR, last=PTR)
    p.update(kw)
    return lib.ssm_heads_fwd(ctypes.byref(d) if d is not None else None, *p.values(), None)


def bwd(lib, d, cu=None, **kw):
    p = dict(u=PTR, delta=PTR, A=PTR, B=PTR, C=PTR, D=None, bias=None, h0=None, cu=cu, dy=PTR,
             dlast=None, du=PTR, ddelta=PTR, dA=PTR, dB=PTR, dC=PTR, dD=None, dbias=None, dh0=None)
    p.update(kw)
    return lib.ssm_heads_bwd(ctypes.byref(d), *p.values(), None)


def update(lib, d, n_slots=8, **kw):
    p = dict(state=PTR, slots=PTR, n=n_slots, u=PTR, delta=PTR, A=PTR, B=PTR, C=PTR, D=None,
             bias=None, y=PTR)
    p.update(kw)
    return lib.ssm_heads_update(ctypes.byref(d), *p.values(), None)


BAD_HEADS = [
    (dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(heads=0), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=3), SHAPE),
    (dict(d_state=0), UNSUPPORTED), (dict(d_state=257), UNSUPPORTED),
    (dict(head_dim=257), UNSUPPORTED), (dict(heads=65536, groups=1), UNSUPPORTED),
    (dict(seqlen=(1 << 25) + 1), UNSUPPORTED), (dict(io_dtype=2), UNSUPPORTED),
    (dict(flags=1), UNSUPPORTED), (dict(reserved=1), UNSUPPORTED), (dict(n_seqs=-1), SHAPE),
    (dict(n_seqs=3), SHAPE), (dict(u_token_stride=-1), SHAPE), (dict(C_batch_stride=-1), SHAPE),
]


@pytest.mark.parametrize("kw,want", BAD_HEADS)
def test_heads_bad_descriptors(lib, kw, want):
    d = heads(**kw)
    assert fwd(lib, d) == want and bwd(lib, d) == want
    assert lib.ssm_heads_workspace_bytes(ctypes.byref(d), 0) == 0
    if not any(k in kw for k in ("seqlen", "n_seqs")):
        assert update(lib, d) == want


def test_heads_null_misaligned_and_workspace(lib):
    assert fwd(lib, None) == NULL
    for k in ("u", "delta", "A", "B", "C", "y"):
        assert fwd(lib, heads(), **{k: None}) == NULL
    for k in ("u", "delta", "A", "B", "C", "dy", "du", "ddelta", "dA", "dB", "dC"):
        assert bwd(lib, heads(), **{k: None}) == NULL
    for k in ("state", "u", "delta", "A", "B", "C", "y"):
        assert update(lib, heads(), **{k: None}) == NULL
    assert fwd(lib, heads(), u=PTR + 1) == MISALIGNED
    assert fwd(lib, heads(), A=PTR + 2) == MISALIGNED
    assert bwd(lib, heads(), dh0=PTR + 2) == MISALIGNED
    assert update(lib, heads(), slots=PTR + 2) == MISALIGNED
    # packed: cu_seqlens exactly with n_seqs, in one batch row
    assert fwd(lib, heads(batch=1, n_seqs=2)) == SHAPE
    assert fwd(lib, heads(batch=1), cu=PTR) == SHAPE
    need = lib.ssm_heads_workspace_bytes(ctypes.byref(heads()), 1)
    assert need > 0
    assert bwd(lib, heads(workspace_bytes=need - 1)) == WORKSPACE
    assert bwd(lib, heads(workspace=None)) == WORKSPACE
    assert bwd(lib, heads(workspace=PTR + 8)) == MISALIGNED
    assert bwd(lib, heads(batch=70000, seqlen=1)) == UNSUPPORTED
    assert update(lib, heads(batch=9), n_slots=8, slots=None) == SHAPE
    assert update(lib, heads(), n_slots=-1) == SHAPE
    # nothing to do
    assert fwd(lib, heads(batch=0)) == OK and update(lib, heads(batch=0)) == OK


def conv(**kw):
    base = dict(batch=2, seqlen=100, channels=64, x_batch_stride=6400, x_token_stride=64,
                dy_batch_stride=6400, dy_token_stride=64, width=4, io_dtype=0, silu=1,
                workspace=PTR, workspace_bytes=1 << 40)
    base.update(kw)
    return ConvDesc(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), SHAPE), (dict(channels=-1), SHAPE), (dict(width=0), UNSUPPORTED),
    (dict(width=5), UNSUPPORTED), (dict(io_dtype=7), UNSUPPORTED), (dict(flags=1), UNSUPPORTED),
    (dict(reserved=1), UNSUPPORTED), (dict(x_token_stride=-1), SHAPE), (dict(n_seqs=2), SHAPE),
    (dict(seqlen=(1 << 25) + 1), UNSUPPORTED)])
def test_conv_bad_descriptors(lib, kw, want):
    d = conv(**kw)
    assert lib.ssm_conv_fwd(ctypes.byref(d), PTR, PTR, None, None, None, PTR, None, None) == want
    assert lib.ssm_conv_bwd(ctypes.byref(d), PTR, PTR, None, None, None, PTR, PTR, PTR, None, None,
                            None) == want


def test_conv_null_misaligned_and_workspace(lib):
    d = ctypes.byref(conv())
    assert lib.ssm_conv_fwd(None, PTR, PTR, None, None, None, PTR, None, None) == NULL
    assert lib.ssm_conv_fwd(d, None, PTR, None, None, None, PTR, None, None) == NULL
    assert lib.ssm_conv_fwd(d, PTR, None, None, None, None, PTR, None, None) == NULL
    assert lib.ssm_conv_fwd(d, PTR + 2, PTR, None, None, None, PTR, None, None) == MISALIGNED
    assert lib.ssm_conv_fwd(d, PTR, PTR, None, None, PTR, PTR, None, None) == SHAPE
    assert lib.ssm_conv_bwd(d, PTR, PTR, None, None, None, PTR, PTR, None, None, None, None) == NULL
    e = ctypes.byref(conv(workspace_bytes=lib.ssm_conv_workspace_bytes(d) - 1))
    assert lib.ssm_conv_bwd(e, PTR, PTR, None, None, None, PTR, PTR, PTR, None, None, None) == WORKSPACE
    assert lib.ssm_conv_update(d, None, None, 4, PTR, PTR, None, PTR, None) == NULL
    assert lib.ssm_conv_update(d, PTR, None, 1, PTR, PTR, None, PTR, None) == SHAPE


def norm(**kw):
    base = dict(rows=5, d=256, group_size=128, x_stride=256, z_stride=256, residual_stride=256,
                dy_stride=256, io_dtype=1, residual_dtype=1, eps=1e-5, workspace=PTR,
                workspace_bytes=1 << 40)
    base.update(kw)
    return NormDesc(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(d=0), SHAPE), (dict(group_size=0), SHAPE),
    (dict(group_size=100), SHAPE), (dict(d=16385, group_size=16385), UNSUPPORTED),
    (dict(io_dtype=3), UNSUPPORTED), (dict(io_dtype=0, residual_dtype=1), UNSUPPORTED),
    (dict(quant_block=-1), SHAPE), (dict(quant_block=8), UNSUPPORTED), (dict(flags=2), UNSUPPORTED),
    (dict(x_stride=-4), SHAPE)])
def test_norm_bad_descriptors(lib, kw, want):
    d = ctypes.byref(norm(**kw))
    assert lib.ssm_norm_fwd(d, PTR, PTR, None, None, PTR, PTR, None, None) == want
    assert lib.ssm_norm_bwd(d, PTR, PTR, None, PTR, None, PTR, None, PTR, None) == want


def test_norm_null_misaligned_and_workspace(lib):
    d = ctypes.byref(norm())
    assert lib.ssm_norm_fwd(None, PTR, PTR, None, None, PTR, None, None, None) == NULL
    assert lib.ssm_norm_fwd(d, PTR, PTR, PTR, None, PTR, None, None, None) == NULL
    q = ctypes.byref(norm(quant_block=32))
    assert lib.ssm_norm_fwd(q, PTR, PTR, None, None, PTR, None, None, None) == NULL
    assert lib.ssm_norm_bwd(q, PTR, PTR, None, PTR, None, PTR, None, PTR, None) == UNSUPPORTED
    assert lib.ssm_norm_fwd(d, PTR + 1, PTR, None, None, PTR, None, None, None) == MISALIGNED
    assert lib.ssm_norm_bwd(d, PTR, PTR, PTR, PTR, None, PTR, None, PTR, None) == NULL
    e = ctypes.byref(norm(workspace_bytes=8))
    assert lib.ssm_norm_bwd(e, PTR, PTR, None, PTR, None, PTR, None, PTR, None) == WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_ranks():
    u, x = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(u, torch.zeros(1, 4, 2), torch.zeros(2), torch.zeros(1, 4, 1, 16),
                          torch.zeros(1, 4, 1, 16))
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(x, x, x, x, x)
    with pytest.raises(ValueError):
        ssm.ssm_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        ssm.ssm_norm_fwd(torch.zeros(2, 8), torch.zeros(8))
    assert {"ssm_heads_fwd", "ssm_heads_bwd", "ssm_heads_update", "ssm_conv_fwd", "ssm_conv_bwd",
            "ssm_conv_update", "ssm_norm_fwd", "ssm_norm_bwd"} <= set(ssm.__all__)
