"""The short convolution and the root-mean-square norm against their plain
forms in 64 bits, and the layer's operators together: a prompt continued token
by token, a training step, both captured in graphs."""
import sys

import pytest
import torch

import layer_testutil as lt
import selective_state_space_fwd_amd as ssm
from ssm_testutil import floored_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.load_library()
    return torch.device("cuda:0")


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def act(dev, io, rows, n, seed, pad=0, odd=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    count = 1
    for r in rows:
        count *= r
    flat = torch.zeros(count * (n + pad) + odd, dtype=lt.IO[io], device=dev)
    v = flat[odd:].view(*rows, n + pad)[..., :n]
    v.copy_((torch.randn(*rows, n, generator=g) * scale).to(lt.IO[io]))
    return v


def f32(dev, *shape, seed=0, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dev)


# -------------------------------------------------------------- convolution

# a silu, its argument's and its own roundings, in steps of 2^-24 of the
# magnitudes; exp2 and the reciprocal are good to an ulp, the exponent's
# product to |v| / 2 ulps (|v| < 40 here)
SILU = 48 * 2.0 ** -24


def check_conv(dev, io, batch, L, ch, W, lens=None, state=True, silu=True, bias=True, pad=0, odd=0):
    say(f"conv {io} {batch} {L} {ch} W={W} lens={lens} state={state} silu={silu} pad={pad} odd={odd}")
    rows = len(lens) if lens is not None else batch
    x, dy = act(dev, io, (batch, L), ch, 1, pad, odd), act(dev, io, (batch, L), ch, 2, pad, odd)
    w = f32(dev, ch, W, seed=3)
    b = f32(dev, ch, seed=4) if bias else None
    st = f32(dev, rows, ch, W - 1, seed=5) if state else None
    cu = None
    if lens is not None:
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    used = L if lens is None else sum(lens)
    y, last = ssm.ssm_conv_fwd(x, w, b, silu=silu, conv_state=st, cu_seqlens=cu)
    out = ssm.ssm_conv_bwd(x, w, dy, b, silu=silu, conv_state=st, cu_seqlens=cu)
    torch.cuda.synchronize()
    ref, size = lt.conv_reference(x[:, :used], w, b, st, lens, silu, dy=dy[:, :used])
    half = lt.HALF[lt.IO[io]]
    e = (W + 2) * 2.0 ** -24 + SILU
    lt.assert_within("y", y[:, :used], ref["y"], half * ref["y"].abs() + e * size["y"] * 1.1 + 1e-30)
    assert torch.equal(lt.f64(last), ref["last"])
    # dv is off by e of its size, and by e of v's size through silu'' (below 0.5)
    g = 2 * e + (W + 2) * 2.0 ** -24
    vsize = size["y"].max() * 2 + 1
    lt.assert_within("dx", out["dx"][:, :used], ref["dx"], half * ref["dx"].abs() + g * vsize * size["dx"] + 1e-30)
    n = 2.0 ** -24 * (40 + batch * L / 64)      # a run, then 16 lanes, then a tree
    for k in ("dweight", "dbias", "dconv_state"):
        if out[k] is not None:
            lt.assert_within(k, out[k], ref[k], (g * vsize + n) * size[k] + 1e-30)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("L", [1, 2, 3, 15, 16, 17, 64, 65, 100])
def test_conv_lengths(dev, io, W, L):
    check_conv(dev, io, 2, L, 24, W)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1, 0, 2, 3, 4, 40, 0], [0, 0, 70], [33, 31, 1], [90]])
@pytest.mark.parametrize("state", [True, False])
def test_conv_packed(dev, io, lens, state):
    check_conv(dev, io, 1, sum(lens), 40, 4, lens=lens, state=state)
    check_conv(dev, io, 1, sum(lens) + 5, 40, 4, lens=lens, state=state)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("ch,pad,odd", [(1, 0, 0), (7, 0, 0), (24, 3, 0), (24, 0, 1), (520, 8, 0),
                                        (1001, 1, 1), (260, 4, 4)])
def test_conv_channels_and_strides(dev, io, ch, pad, odd):
    check_conv(dev, io, 2, 40, ch, 4, pad=pad, odd=odd)


@pytest.mark.parametrize("io,lens", [("f32", [1000, 0, 63, 64, 973]), ("bf16", [2000, 1, 129, 2860]),
                                     ("bf16", [3001, 23, 24, 2960])])
def test_conv_many_channels(dev, io, lens):
    """Runs of 24 tokens, and of 32 and 64 in the gradients; sequences end inside them."""
    check_conv(dev, io, 1, sum(lens), 8196, 4, lens=lens)


def test_conv_without_options(dev):
    check_conv(dev, "f32", 2, 40, 24, 4, state=False, silu=False, bias=False)


def test_conv_no_tokens_and_tokens_behind(dev):
    w, st = f32(dev, 8, 4), f32(dev, 2, 8, 3)
    x = torch.zeros(2, 0, 8, device=dev)
    y, last = ssm.ssm_conv_fwd(x, w, conv_state=st)
    out = ssm.ssm_conv_bwd(x, w, x, conv_state=st)
    torch.cuda.synchronize()
    assert y.shape == x.shape and torch.equal(last, st)
    assert not out["dweight"].any() and not out["dconv_state"].any()
    x = torch.full((1, 20, 8), float("nan"), device=dev)
    x[:, :12] = 1.0
    y = torch.full_like(x, 7.0)
    cu = torch.tensor([0, 5, 12], dtype=torch.int32, device=dev)
    _, last = ssm.ssm_conv_fwd(x, w, cu_seqlens=cu, y=y)
    torch.cuda.synchronize()
    assert (y[:, 12:] == 7.0).all() and torch.isfinite(y).all() and (last == 1.0).all()
    for bad in ([0, 15, 5], [-3, 4, 20], [0, 400, 800]):
        ssm.ssm_conv_fwd(x, w, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=dev))
        ssm.ssm_conv_bwd(x, w, x, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("rows,ch,odd", [(1, 8, 0), (5, 1000, 0), (3, 13, 1)])
def test_conv_update(dev, io, W, rows, ch, odd):
    x = act(dev, io, (rows,), ch, 1, 2 * odd, odd)
    w, b = f32(dev, ch, W, seed=2), f32(dev, ch, seed=3)
    state = f32(dev, rows + 3, ch, W - 1, seed=4)
    before = state.clone()
    slots = torch.randperm(rows + 3, generator=torch.Generator().manual_seed(5))[:rows]
    y = torch.full((rows + 1, ch), 7.0, dtype=lt.IO[io], device=dev)
    with_bad = torch.cat([slots, torch.tensor([-1])]).to(torch.int32).to(dev)
    ssm.ssm_conv_update(state, torch.cat([x, x[:1]]), w, b, slots=with_bad, y=y)
    torch.cuda.synchronize()
    ref, size = lt.conv_reference(x[:, None], w, b, before[slots.to(dev)], None)
    half = lt.HALF[lt.IO[io]]
    lt.assert_within("y", y[:rows], ref["y"][:, 0],
                     half * ref["y"][:, 0].abs() + ((W + 2) * 2.0 ** -24 + SILU) * 1.1 * size["y"][:, 0] + 1e-30)
    assert (y[rows:] == 7.0).all()
    assert torch.equal(lt.f64(state[slots.to(dev)]), ref["last"])
    rest = [i for i in range(rows + 3) if i not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])


# --------------------------------------------------------------------- norm

def check_norm(dev, io, rows, d, group, res=None, gate=False, block=0, pad=0, odd=0):
    say(f"norm {io} {rows} {d} group={group} res={res} gate={gate} block={block} pad={pad} odd={odd}")
    x = act(dev, io, (rows,), d, 1, pad, odd)
    z = act(dev, io, (rows,), d, 2, pad, odd) if gate else None
    r = act(dev, res, (rows,), d, 3, pad, odd, 2.0) if res else None
    w = f32(dev, d, seed=4)
    y, scale, s = ssm.ssm_norm_fwd(x, w, residual=r, z=z, group_size=group, quant_block=block)
    torch.cuda.synchronize()
    if res:
        exact = lt.f64(x) + lt.f64(r)
        # the sum in float32, then the residual's type
        lt.assert_within("residual", s, exact, (lt.HALF[lt.IO[res]] * (1 + 2.0 ** -24) + 2.0 ** -24) * exact.abs())
    base = s if res else x
    dy = act(dev, io, (rows,), d, 5, pad, odd)
    dr = f32(dev, rows, d, seed=6).to(base.dtype) if res else None
    ref = lt.norm_reference(base, w, z, group, dy=dy, dresidual=dr)
    half = lt.HALF[lt.IO[io]]
    # the mean square: a lane's terms, the workgroup's tree; half of it in the
    # root; then the gate's silu and six products
    n = (group / 512 + 40) * 2.0 ** -24 + SILU
    if not block:
        lt.assert_within("y", y, ref["y"], half * ref["y"].abs() + n * ref["y"].abs() * (1 + half) + 1e-30)
    else:
        v = ref["y"].unflatten(-1, (-1, group))
        k = -(-group // block)
        v = torch.nn.functional.pad(v, (0, k * block - group)).unflatten(-1, (k, block))
        most = v.abs().amax(-1)
        lt.assert_within("scale", scale, (most / 448).reshape(rows, -1), (n + 2.0 ** -23) * (most / 448).reshape(rows, -1))
        got = lt.f64(scale).reshape(most.shape)[..., None].expand(v.shape).flatten(-2)[..., :group]
        got = got.reshape(rows, d) * lt.f64(y.float())
        # half a step of 3 bits, or of the smallest numbers (2^-9 of a step of 1 / 448)
        room = (2.0 ** -4 + 2 * n) * ref["y"].abs() + (
            2.0 ** -10 / 448 * most[..., None]).expand(v.shape).flatten(-2)[..., :group].reshape(rows, d)
        lt.assert_within("8 bits", got, ref["y"], room * (1 + 1e-6) + 1e-30)
        return
    out = ssm.ssm_norm_bwd(base, w, dy, z=z, dresidual=dr, group_size=group)
    torch.cuda.synchronize()
    # dg = rs (dn - n mean(dn n)): both terms' magnitudes
    dn = (lt.f64(dy) * lt.f64(w)).abs()
    nn = ref["n"].abs()
    mean = (dn * nn).unflatten(-1, (-1, group)).mean(-1, keepdim=True).expand(rows, d // group, group).flatten(-2)
    gate_ = torch.ones_like(dn) if z is None else (lt.f64(z) * torch.sigmoid(lt.f64(z))).abs()
    g = lt.f64(base) * (1 if z is None else lt.f64(z) * torch.sigmoid(lt.f64(z)))
    rs = (1 / torch.sqrt((g * g).unflatten(-1, (-1, group)).mean(-1, keepdim=True) + 1e-5)
          ).expand(rows, d // group, group).flatten(-2)
    dg = rs * (dn + nn * mean)
    own = lt.HALF[base.dtype]
    extra = 0 if dr is None else lt.f64(dr).abs()
    lt.assert_within("dx", out["dx"], ref["dx"], own * ref["dx"].abs() + 3 * n * (dg * gate_ + extra) + 1e-30)
    if z is not None:
        slope = 1.1 * lt.f64(base).abs()
        lt.assert_within("dz", out["dz"], ref["dz"], half * ref["dz"].abs() + 4 * n * dg * slope + 1e-30)
    m = n + 2.0 ** -24 * (rows + 16)
    lt.assert_within("dweight", out["dweight"], ref["dweight"], m * (lt.f64(dy).abs() * nn).sum(0) + 1e-30)


@pytest.mark.parametrize("io,res", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"),
                                    ("bf16", "f32")])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rows,d,group", [(1, 1, 1), (3, 8, 8), (5, 100, 50), (2, 2560, 2560),
                                          (7, 1000, 1000), (4, 4096, 512), (3, 5003, 5003)])
def test_norm(dev, io, res, gate, rows, d, group):
    check_norm(dev, io, rows, d, group, res, gate)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16384, 8192, 16383])
def test_norm_wide_rows(dev, io, d):
    check_norm(dev, io, 2, d, d, None, True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_norm_more_groups_than_a_grid_has_rows(dev, io):
    check_norm(dev, io, 3, 140000, 2, None, True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad,odd", [(8, 0), (1, 0), (0, 1), (3, 5)])
def test_norm_strides_and_alignment(dev, io, pad, odd):
    check_norm(dev, io, 5, 264, 132, "f32", True, pad=pad, odd=odd)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,group,block", [(256, 256, 128), (5120, 2560, 128), (300, 300, 128),
                                           (300, 100, 64), (129, 129, 16), (64, 64, 64),
                                           (40, 20, 20), (1000, 1000, 1000), (7, 7, 7), (512, 256, 32),
                                           (100, 100, 33)])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_eight_bits(dev, io, d, group, block, gate):
    check_norm(dev, io, 4, d, group, None, gate, block)
    check_norm(dev, io, 3, d, group, "f32", gate, block, pad=1, odd=1)


def test_norm_eight_bits_of_zeros_and_infinities(dev):
    x = f32(dev, 3, 256, seed=1)
    w = torch.ones(256, device=dev)
    w[:128] = 0.0                               # a block of zeros
    x[2, 200] = float("nan")
    y, scale, _ = ssm.ssm_norm_fwd(x, w, quant_block=128)
    torch.cuda.synchronize()
    assert (scale[:2, 0] == 0).all() and (y[:2, :128].float() == 0).all()
    assert torch.isfinite(scale[:2]).all() and (y[:2, 128:].float().abs().amax(1) == 448).all()
    assert torch.isnan(scale[2]).all() and torch.isnan(y[2].float()).all()


def test_norm_residual_in_place_and_no_rows(dev):
    x, w, r = f32(dev, 4, 64, seed=1), f32(dev, 64, seed=2), f32(dev, 4, 64, seed=3)
    want = ssm.ssm_norm_fwd(x, w, residual=r)
    keep = r.clone()
    y, _, s = ssm.ssm_norm_fwd(x, w, residual=r, residual_out=r)
    torch.cuda.synchronize()
    assert s is r and torch.equal(y, want[0]) and torch.equal(r, want[2]) and torch.equal(r, x + keep)
    y, _, _ = ssm.ssm_norm_fwd(x[:0], w)
    out = ssm.ssm_norm_bwd(x[:0], w, x[:0])
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and not out["dweight"].any()


def test_refusals(dev):
    x, w = torch.zeros(1, 4, 8, device=dev), torch.zeros(8, 4, device=dev)
    with pytest.raises(ssm.SsmError):
        ssm.ssm_conv_fwd(x, torch.zeros(8, 5, device=dev))
    with pytest.raises(ValueError):
        ssm.ssm_conv_fwd(x.transpose(1, 2), torch.zeros(4, 4, device=dev))
    with pytest.raises(ValueError):
        ssm.ssm_conv_fwd(x, w, conv_state=torch.zeros(2, 8, 3, device=dev))
    with pytest.raises(TypeError):
        ssm.ssm_conv_bwd(x, w, x.to(torch.bfloat16))
    n = torch.zeros(2, 8, device=dev)
    with pytest.raises(ValueError):
        ssm.ssm_norm_fwd(n, torch.zeros(8, device=dev), group_size=3)
    with pytest.raises(ValueError):
        ssm.ssm_norm_fwd(n, torch.zeros(8, device=dev), scale=torch.zeros(2, 1, device=dev))
    with pytest.raises(ssm.SsmError):
        ssm.ssm_norm_fwd(n, torch.zeros(8, device=dev), residual=n.to(torch.bfloat16))
    with pytest.raises(ssm.SsmError):
        ssm.ssm_norm_fwd(torch.zeros(1, 64, device=dev), torch.zeros(64, device=dev), quant_block=8)


# ----------------------------------------------------------------- together

H, P, G, N, W = 4, 32, 2, 16, 4
DI, CH = H * P, H * P + 2 * G * N


def layer_params(dev):
    return dict(cw=f32(dev, CH, W, seed=1, scale=0.5), cb=f32(dev, CH, seed=2, scale=0.1),
                A=-torch.rand(H, generator=torch.Generator().manual_seed(3)).to(dev) - 0.1,
                D=f32(dev, H, seed=4), bias=f32(dev, H, seed=5) - 2.0,
                nw=1 + f32(dev, DI, seed=6, scale=0.1))


def split(p):
    """The projection's columns: gate, convolution input, step sizes."""
    return p[..., :DI], p[..., DI:DI + CH], p[..., DI + CH:]


def prompt(q, proj, conv_state=None, h0=None):
    z, x, delta = split(proj)
    v, conv = ssm.ssm_conv_fwd(x, q["cw"], q["cb"], conv_state=conv_state)
    u, B, C = (v[..., a:b].unflatten(-1, s) for a, b, s in
               ((0, DI, (H, P)), (DI, DI + G * N, (G, N)), (DI + G * N, CH, (G, N))))
    y, last = ssm.ssm_heads_fwd(u, delta, q["A"], B, C, q["D"], q["bias"], initial_state=h0)
    b, L = proj.shape[:2]
    o, scale, _ = ssm.ssm_norm_fwd(y.reshape(b * L, DI), q["nw"], z=z.reshape(b * L, DI), group_size=DI // G)
    return o.view(b, L, DI), conv, last


def token(q, proj, conv_state, state, slots):
    z, x, delta = split(proj)
    v = ssm.ssm_conv_update(conv_state, x, q["cw"], q["cb"], slots=slots)
    u, B, C = (v[..., a:b].unflatten(-1, s) for a, b, s in
               ((0, DI, (H, P)), (DI, DI + G * N, (G, N)), (DI + G * N, CH, (G, N))))
    y = ssm.ssm_heads_update(state, u, delta, q["A"], B, C, q["D"], q["bias"], slots=slots)
    return ssm.ssm_norm_fwd(y.reshape(-1, DI), q["nw"], z=z, group_size=DI // G)[0]


def test_prompt_then_tokens_is_the_longer_prompt(dev):
    """A prompt's states go into slots and tokens continue from there: the
    outputs and states are those of one longer prompt (float32: 1e-4 of the
    outputs' size, the bar of every float32 result here)."""
    q = layer_params(dev)
    proj = act(dev, "f32", (2, 90), DI + CH + H, 9)
    want, conv_w, last_w = prompt(q, proj)
    head, conv, last = prompt(q, proj[:, :70])
    slots = torch.tensor([3, 0], dtype=torch.int32, device=dev)
    cpool, pool = torch.zeros(5, CH, W - 1, device=dev), torch.zeros(5, H, P, N, device=dev)
    cpool[slots.long()], pool[slots.long()] = conv, last
    outs = [head] + [token(q, proj[:, t], cpool, pool, slots)[:, None] for t in range(70, 90)]
    torch.cuda.synchronize()
    got = torch.cat(outs, 1)
    for a, b in ((got, want), (pool[slots.long()], last_w)):
        err = floored_err(lt.f64(a).numpy(), lt.f64(b).numpy())
        say(f"prompt and tokens: {err:.2e}")
        assert err <= 1e-4
    assert torch.equal(cpool[slots.long()], conv_w)
    assert not pool[[1, 2, 4]].any() and not cpool[[1, 2, 4]].any()


def test_two_prompts_behind_one_another(dev):
    """States carried from one call into the next."""
    q = layer_params(dev)
    proj = act(dev, "f32", (2, 130), DI + CH + H, 10)
    want = prompt(q, proj)
    first = prompt(q, proj[:, :61])
    second = prompt(q, proj[:, 61:], first[1], first[2])
    torch.cuda.synchronize()
    for a, b in ((torch.cat([first[0], second[0]], 1), want[0]), (second[2], want[2])):
        assert floored_err(lt.f64(a).numpy(), lt.f64(b).numpy()) <= 1e-4
    assert torch.equal(second[1], want[1])


def step(q, proj, dout):
    """A training step of the layer between its projections: the gradients of
    sum(dout * out) with respect to proj and the parameters."""
    z, x, delta = split(proj)
    b, L = proj.shape[:2]
    v, _ = ssm.ssm_conv_fwd(x, q["cw"], q["cb"], return_last_state=False)
    u, B, C = (v[..., a:e].unflatten(-1, s) for a, e, s in
               ((0, DI, (H, P)), (DI, DI + G * N, (G, N)), (DI + G * N, CH, (G, N))))
    y, _ = ssm.ssm_heads_fwd(u, delta, q["A"], B, C, q["D"], q["bias"], return_last_state=False)
    yz, zz = y.reshape(b * L, DI), z.reshape(b * L, DI)
    o = ssm.ssm_norm_fwd(yz, q["nw"], z=zz, group_size=DI // G)[0]
    n = ssm.ssm_norm_bwd(yz, q["nw"], dout.reshape(b * L, DI), z=zz, group_size=DI // G)
    h = ssm.ssm_heads_bwd(u, delta, q["A"], B, C, n["dx"].view(b, L, H, P), q["D"], q["bias"])
    dv = torch.cat([h["du"].flatten(-2), h["dB"].flatten(-2), h["dC"].flatten(-2)], -1)
    c = ssm.ssm_conv_bwd(x, q["cw"], dv, q["cb"])
    dproj = torch.cat([n["dz"].view(b, L, DI), c["dx"], h["ddelta"]], -1)
    return o, dproj, c["dweight"], c["dbias"], h["dA"], h["dD"], h["ddelta_bias"], n["dweight"]


def test_training_step_against_differences(dev):
    """The layer's whole gradient against a difference of its output along a
    random direction (float32; a step of 2^-9 along a direction of unit-sized
    values: the second-order error of the central difference, about h^2, and
    the outputs' 1e-6 over h both stay below 2e-3 of the sum's size)."""
    q = layer_params(dev)
    proj = act(dev, "f32", (1, 75), DI + CH + H, 11)
    dout = act(dev, "f32", (1, 75), DI, 12)
    got = step(q, proj, dout)
    h = 2.0 ** -9
    names = ("cw", "cb", "A", "D", "bias", "nw")
    for k, name in enumerate(("proj",) + names):
        base = proj if name == "proj" else q[name]
        dirn = f32(dev, *base.shape, seed=20 + k)
        if name == "A":
            dirn = dirn * 0.1
        side = []
        for s in (-1, 1):
            q2 = q if name == "proj" else {**q, name: q[name] + s * h * dirn}
            p2 = proj + s * h * dirn if name == "proj" else proj
            o = prompt(q2, p2.contiguous())[0]
            side.append((o.double() * dout.double()).sum())
        torch.cuda.synchronize()
        want = float((side[1] - side[0]) / (2 * h))
        terms = got[1 + k].double() * dirn.double()
        have, size = float(terms.sum()), float(terms.norm())
        say(f"along {name}: {have:.5f} {want:.5f} (size {size:.3f})")
        assert abs(have - want) <= 5e-3 * (size + abs(want)), name


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_graphs_of_a_step_and_of_a_token(dev, io):
    """Both captured, replayed on new inputs between eager work, and equal to
    the eager calls' bits every time."""
    q = layer_params(dev)
    proj, dout = act(dev, io, (2, 70), DI + CH + H, 13), act(dev, io, (2, 70), DI, 14)
    slots = torch.tensor([2, 0], dtype=torch.int32, device=dev)
    cpool, pool = f32(dev, 3, CH, W - 1, seed=15), f32(dev, 3, H, P, N, seed=16)
    tok = act(dev, io, (2,), DI + CH + H, 17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(q, proj, dout)
        token(q, tok, cpool.clone(), pool.clone(), slots)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train = step(q, proj, dout)
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        out = token(q, tok, cpool, pool, slots)
    for k in range(3):
        proj.copy_(act(dev, io, (2, 70), DI + CH + H, 30 + k))
        tok.copy_(act(dev, io, (2,), DI + CH + H, 40 + k))
        c, p = cpool.clone(), pool.clone()
        want = step(q, proj, dout)
        want2 = token(q, tok, c, p, slots)
        torch.cuda.synchronize()
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(train, want)), k
        assert torch.equal(out, want2) and torch.equal(cpool, c) and torch.equal(pool, p), k


def test_prepared_calls(dev):
    """A prepared call launches the same work on new contents."""
    q = layer_params(dev)
    proj = act(dev, "bf16", (2, 50), DI + CH + H, 18)
    _, x, delta = split(proj)
    conv = ssm.ssm_conv_fwd(x, q["cw"], q["cb"], prepare=True)
    v, _ = conv()
    u, B, C = (v[..., a:b].unflatten(-1, s) for a, b, s in
               ((0, DI, (H, P)), (DI, DI + G * N, (G, N)), (DI + G * N, CH, (G, N))))
    scan = ssm.ssm_heads_fwd(u, delta, q["A"], B, C, q["D"], q["bias"], prepare=True)
    y, _ = scan()
    for k in range(2):
        proj.copy_(act(dev, "bf16", (2, 50), DI + CH + H, 50 + k))
        conv()
        scan()
        want_v = ssm.ssm_conv_fwd(x, q["cw"], q["cb"])[0]
        want = ssm.ssm_heads_fwd(u, delta, q["A"], B, C, q["D"], q["bias"])[0]
        torch.cuda.synchronize()
        assert torch.equal(v, want_v) and torch.equal(y, want)


def test_two_steps_at_once_on_two_streams(dev):
    q = layer_params(dev)
    a, b = act(dev, "bf16", (1, 300), DI + CH + H, 19), act(dev, "bf16", (1, 300), DI + CH + H, 20)
    dout = act(dev, "bf16", (1, 300), DI, 21)
    want = step(q, a, dout), step(q, b, dout)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        g1 = step(q, a, dout)
    with torch.cuda.stream(s2):
        g2 = step(q, b, dout)
    torch.cuda.synchronize()
    for x, y in zip(want, (g1, g2)):
        assert all(torch.equal(i, j) for i, j in zip(x, y))
