"""The scan over heads (prompt, gradients, single token) against its plain form
in 64 bits, with bounds that count roundings (layer_testutil)."""
import sys

import pytest
import torch

import layer_testutil as lt
import selective_state_space_fwd_amd as ssm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.load_library()
    return torch.device("cuda:0")


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def make(dev, io, batch, L, H, P, G, N, lens=None, state=True, seed=0, skip=True, bias=True,
         decay=4.0, pad=0, odd=0):
    """Inputs; pad: columns between the tokens of u, B, C and delta, odd: values
    that each of them lies behind an aligned place."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    rows = len(lens) if lens is not None else batch

    def act(*shape):
        n = 1
        for s in shape[2:]:
            n *= s
        flat = torch.zeros(batch * L * (n + pad) + odd, dtype=lt.IO[io], device=dev)
        v = flat[odd:].view(batch, L, n + pad)[..., :n]
        v.copy_(r(batch, L, n).to(lt.IO[io]))
        return v.unflatten(-1, shape[2:]) if len(shape) > 3 else v

    t = dict(u=act(batch, L, H, P), delta=act(batch, L, H), B=act(batch, L, G, N),
             C=act(batch, L, G, N), dy=act(batch, L, H, P))
    t["A"] = -(torch.rand(H, generator=g) * decay + 0.05).to(dev)
    t["D"] = r(H).to(dev) if skip else None
    t["delta_bias"] = (r(H) - 2.0).to(dev) if bias else None
    t["h0"] = r(rows, H, P, N).to(dev) if state else None
    t["dlast"] = r(rows, H, P, N).to(dev) if state else None
    t["cu"] = None
    if lens is not None:
        at = torch.tensor([0] + lens).cumsum(0)
        t["cu"] = at.to(torch.int32).to(dev)
    return t


def run_fwd(t, softplus=True):
    return ssm.ssm_heads_fwd(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"], t["delta_bias"],
                             softplus=softplus, initial_state=t["h0"], cu_seqlens=t["cu"])


def run_bwd(t, softplus=True):
    return ssm.ssm_heads_bwd(t["u"], t["delta"], t["A"], t["B"], t["C"], t["dy"], t["D"],
                             t["delta_bias"], softplus=softplus, initial_state=t["h0"],
                             dlast=t["dlast"], cu_seqlens=t["cu"])


def check(dev, io, shape, lens=None, softplus=True, gradients=True, **kw):
    batch, L, H, P, G, N = shape
    say(f"heads {io} {shape} lens={lens} {kw}")
    t = make(dev, io, batch, L, H, P, G, N, lens, **kw)
    used = L if lens is None else sum(lens)
    cut = lambda k: t[k][:, :used]
    ref, size = lt.heads_reference(cut("u"), cut("delta"), t["A"], cut("B"), cut("C"), t["D"],
                                   t["delta_bias"], t["h0"], lens, softplus,
                                   dy=cut("dy") if gradients else None, dlast=t["dlast"])
    half = lt.HALF[lt.IO[io]]
    # float32 sums: over states, channels, the tokens of a chunk, the chunks, the
    # heads of a group and the roundings on the way (decays, step sizes, terms)
    f32 = (N + P + 64 + L // 32 + H + 64) * 2.0 ** -24
    dec = {k: 2.0 ** -24 * v for k, v in size["decays"].items()}
    y, last = run_fwd(t, softplus)
    torch.cuda.synchronize()
    # y: its own rounding; one of each decayed product and of each state value
    two = half if io == "bf16" else 0.0
    lt.assert_within("y", y[:, :used], ref["y"], half * ref["y"].abs() + ((two + f32) * size["y"] + dec["y"]) * (1 + half))
    lt.assert_within("last_state", last, ref["last_state"], f32 * size["last_state"] + dec["last_state"] + 1e-30)
    if not gradients:
        return
    out = run_bwd(t, softplus)
    torch.cuda.synchronize()
    for k in ("du", "dB", "dC"):
        lt.assert_within(k, out[k][:, :used], ref[k],
                         half * ref[k].abs() + ((two + f32) * size[k] + dec[k]) * (1 + half) + 1e-30)
    # the decays' gradients are float32 sums throughout; <gh, h_in> of a chunk
    # that keeps below 2^-13 comes from values of one rounding each
    few = 2 * two * 2.0 ** -13
    for k, own in (("ddelta", half), ("dA", 0.0), ("ddelta_bias", 0.0)):
        if out[k] is None:
            continue
        got = out[k][:, :used] if k == "ddelta" else out[k]
        n = f32 if k == "ddelta" else f32 + 2.0 ** -24 * 8      # the last sums run in 64 bits
        lt.assert_within(k, got, ref[k], own * ref[k].abs() +
                         (n * size[k] + dec[k] + few * size["through_" + k]) * (1 + own) + 1e-30)
    if t["D"] is not None:
        lt.assert_within("dD", out["dD"], ref["dD"], (f32 + 8 * 2.0 ** -24) * size["dD"] + 1e-30)
    if t["h0"] is not None:
        lt.assert_within("dh0", out["dh0"], ref["dh0"], f32 * size["dh0"] + dec["dh0"] + 1e-30)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 130])
def test_lengths(dev, io, L):
    check(dev, io, (2, L, 3, 64, 1, 64), seed=L)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H,P,G,N", [(1, 1, 1, 1), (4, 16, 2, 16), (6, 33, 2, 24), (3, 48, 3, 100),
                                     (2, 128, 1, 128), (5, 32, 1, 130), (2, 80, 1, 256),
                                     (9, 8, 3, 64), (2, 256, 1, 32)])
def test_head_layouts(dev, io, H, P, G, N):
    check(dev, io, (1, 70, H, P, G, N), seed=P + N)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[40, 0, 1, 64, 65, 0, 3], [0, 0, 100, 0], [1, 1, 1, 2], [200]])
@pytest.mark.parametrize("N", [128, 20])
def test_packed_sequences(dev, io, lens, N):
    check(dev, io, (1, sum(lens), 3, 64, 1, N), lens=lens, seed=len(lens))
    check(dev, io, (1, sum(lens) + 9, 3, 64, 1, N), lens=lens, seed=len(lens), state=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 900, 2, 64, 1, 64), (2, 700, 1, 32, 1, 128)])
@pytest.mark.parametrize("state", [True, False])
def test_ranges_of_a_long_row(dev, io, shape, state):
    """Few heads: the row is cut into ranges joined by their states."""
    check(dev, io, shape, seed=7, state=state, decay=0.5)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_ranges_of_packed_sequences(dev, io):
    check(dev, io, (1, 1000, 2, 64, 1, 64), lens=[300, 0, 5, 450, 245], seed=3, decay=0.5)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad,odd", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(dev, io, pad, odd):
    check(dev, io, (2, 70, 4, 64, 2, 64), seed=pad + odd, pad=pad, odd=odd)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_options(dev, io):
    check(dev, io, (2, 70, 3, 64, 1, 64), skip=False, bias=False, state=False, seed=1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [1e-3, 60.0, 2000.0])
def test_slow_and_fast_decays(dev, io, decay):
    """From states that last to ones that are gone within a token."""
    check(dev, io, (1, 200, 3, 64, 1, 64), seed=5, decay=decay)


def test_step_sizes_given(dev):
    """Without softplus: step sizes of zero leave the state alone."""
    t = make(dev, "f32", 1, 66, 2, 64, 1, 64, bias=False, seed=9)
    t["delta"].copy_(t["delta"].abs() * 0.1)
    t["delta"][:, 10:20] = 0.0
    ref, size = lt.heads_reference(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"], None,
                                   t["h0"], None, False)
    y, last = run_fwd(t, softplus=False)
    torch.cuda.synchronize()
    f32 = 500 * 2.0 ** -24
    lt.assert_within("y", y, ref["y"], f32 * size["y"])
    lt.assert_within("last_state", last, ref["last_state"], f32 * size["last_state"])


def test_no_tokens(dev):
    t = make(dev, "f32", 2, 0, 2, 16, 1, 16)
    y, last = run_fwd(t)
    out = run_bwd(t)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 2, 16) and torch.equal(last, t["h0"])
    assert torch.equal(out["dh0"], t["dlast"]) and not out["dA"].any() and not out["dD"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_tokens_behind_the_last_sequence_stay(dev, io):
    t = make(dev, io, 1, 80, 2, 64, 1, 64, lens=[30, 20])
    t["u"][:, 50:] = float("nan")
    y = torch.full_like(t["u"].contiguous(), 7.0)
    got, last = ssm.ssm_heads_fwd(t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"],
                                  t["delta_bias"], initial_state=t["h0"], cu_seqlens=t["cu"], y=y)
    torch.cuda.synchronize()
    assert got is y and (y[:, 50:] == 7.0).all() and torch.isfinite(y).all()
    assert torch.isfinite(last).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_infinities_stay_in_their_sequence(dev, io):
    """A NaN of one sequence reaches neither its neighbours nor their states."""
    lens = [20, 70, 33]
    t = make(dev, io, 1, sum(lens), 2, 64, 1, 64, lens=lens, seed=2)
    y0, l0 = run_fwd(t)
    g0 = run_bwd(t)
    t["u"][0, 40] = float("nan")
    t["h0"][1] = float("inf")
    y1, l1 = run_fwd(t)
    g1 = run_bwd(t)
    torch.cuda.synchronize()
    for a, b in ((0, 20), (90, 123)):
        assert torch.equal(y0[:, a:b], y1[:, a:b])
        assert torch.equal(g0["du"][:, a:b], g1["du"][:, a:b])
        assert torch.equal(g0["dB"][:, a:b], g1["dB"][:, a:b])
        assert torch.equal(g0["ddelta"][:, a:b], g1["ddelta"][:, a:b])
    assert torch.equal(l0[[0, 2]], l1[[0, 2]]) and torch.equal(g0["dh0"][[0, 2]], g1["dh0"][[0, 2]])
    assert not torch.isfinite(y1[:, 40]).any()


def test_malformed_offsets_stay_inside(dev):
    """Offsets that break the rules give no error and no access outside."""
    t = make(dev, "f32", 1, 50, 2, 16, 1, 16, lens=[20, 30])
    for bad in ([0, 40, 20], [-5, 10, 50], [0, 1000, 2000], [50, 50, 50]):
        t["cu"] = torch.tensor(bad, dtype=torch.int32, device=dev)
        run_fwd(t)
        run_bwd(t)
        torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_same_bits_again_and_on_another_stream(dev, io):
    t = make(dev, io, 2, 300, 5, 64, 1, 128, seed=4)
    first = (run_fwd(t), run_bwd(t))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = (run_fwd(t), run_bwd(t))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[0], again[0]))
    assert all(torch.equal(first[1][k], again[1][k]) for k in first[1])


# ------------------------------------------------------------- single token

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,H,P,G,N", [(1, 1, 1, 1, 1), (1, 4, 64, 1, 128), (5, 6, 33, 2, 24),
                                          (3, 3, 48, 3, 101), (40, 80, 64, 1, 128), (2, 2, 256, 1, 256),
                                          (40, 16, 33, 2, 6), (20, 32, 200, 1, 101)])
def test_update(dev, io, rows, H, P, G, N):
    say(f"update {io} {rows} {H} {P} {G} {N}")
    t = make(dev, io, rows, 1, H, P, G, N, seed=rows + N)
    for k in ("u", "delta", "B", "C"):
        t[k] = t[k][:, 0]
    n = rows + 2
    state = torch.randn(n, H, P, N, generator=torch.Generator().manual_seed(1)).to(dev)
    before = state.clone()
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:rows].to(torch.int32).to(dev)
    y = ssm.ssm_heads_update(state, t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"],
                             t["delta_bias"], slots=slots)
    torch.cuda.synchronize()
    ref, size = lt.heads_reference(*(t[k][:, None] for k in ("u", "delta")), t["A"],
                                   *(t[k][:, None] for k in ("B", "C")), t["D"], t["delta_bias"],
                                   before[slots.long()], None)
    f32 = (N + 16) * 2.0 ** -24
    half = lt.HALF[lt.IO[io]]
    lt.assert_within("y", y, ref["y"][:, 0], half * ref["y"][:, 0].abs() +
                     (f32 * size["y"][:, 0] + 2.0 ** -24 * size["decays"]["y"][:, 0]) * (1 + half))
    lt.assert_within("state", state[slots.long()], ref["last_state"],
                     f32 * size["last_state"] + 2.0 ** -24 * size["decays"]["last_state"])
    rest = [i for i in range(n) if i not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])


def test_update_skips_rows_without_a_slot(dev):
    t = make(dev, "f32", 4, 1, 2, 16, 1, 16)
    for k in ("u", "delta", "B", "C"):
        t[k] = t[k][:, 0]
    state = torch.randn(3, 2, 16, 16, device=dev)
    before, y = state.clone(), torch.full((4, 2, 16), 7.0, device=dev)
    slots = torch.tensor([1, -1, 3, 1 << 30], dtype=torch.int32, device=dev)
    ssm.ssm_heads_update(state, t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"],
                         t["delta_bias"], slots=slots, y=y)
    torch.cuda.synchronize()
    assert (y[1:] == 7.0).all() and torch.equal(state[[0, 2]], before[[0, 2]])
    assert not torch.equal(state[1], before[1])


def test_update_past_32_bit_offsets(dev):
    """A slot that begins behind 2^31 values of the state pool."""
    H, P, N = 80, 64, 128
    n = (1 << 31) // (H * P * N) + 3
    state = torch.empty(n, H, P, N, device=dev)
    state[-1] = 0.5
    t = make(dev, "bf16", 1, 1, H, P, 1, N)
    for k in ("u", "delta", "B", "C"):
        t[k] = t[k][:, 0]
    slots = torch.tensor([n - 1], dtype=torch.int32, device=dev)
    y = ssm.ssm_heads_update(state, t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"],
                             t["delta_bias"], slots=slots)
    small = torch.full((1, H, P, N), 0.5, device=dev)
    want = ssm.ssm_heads_update(small, t["u"], t["delta"], t["A"], t["B"], t["C"], t["D"],
                                t["delta_bias"])
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(state[-1], small[0])


# ----------------------------------------------------------------- refusals

def test_binding_refusals(dev):
    t = make(dev, "f32", 2, 8, 2, 16, 1, 16)
    ok = dict(u=t["u"], delta=t["delta"], A=t["A"], B=t["B"], C=t["C"])
    with pytest.raises(TypeError):
        ssm.ssm_heads_fwd(**{**ok, "B": t["B"].to(torch.bfloat16)})
    with pytest.raises(TypeError):
        ssm.ssm_heads_fwd(**{**ok, "u": t["u"].to(torch.float16)})
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(**{**ok, "A": t["A"][:1]})
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(**{**ok, "u": t["u"].transpose(2, 3).contiguous().transpose(2, 3)})
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(**ok, initial_state=t["h0"][:1])
    with pytest.raises(ValueError):
        ssm.ssm_heads_fwd(**ok, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        ssm.ssm_heads_update(torch.zeros(1, 2, 16, 16, device=dev), t["u"][:, 0], t["delta"][:, 0],
                             t["A"], t["B"][:, 0], t["C"][:, 0])
    with pytest.raises(ssm.SsmError):
        b3 = torch.zeros(2, 8, 3, 16, device=dev)
        ssm.ssm_heads_fwd(t["u"], t["delta"], t["A"], b3, b3)
