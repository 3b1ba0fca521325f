"""The plain 64-bit forms that the layer operators are held to, against
differences and against each other (CPU)."""
import math

import pytest
import torch

import layer_testutil as lt


def rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("lens", [None, [2, 0, 3]])
def test_scan_gradients_against_differences(lens):
    b, L, H, P, G, N = (1, 5, 2, 2, 1, 3)
    spans = lt.spans_of(L, b, lens)
    u, B, C = rand(b, L, H, P, seed=1), rand(b, L, G, N, seed=2), rand(b, L, G, N, seed=3)
    w, a = rand(b, L, H, seed=4).abs() + 0.1, -rand(b, L, H, seed=5).abs()
    h0 = rand(len(spans), H, P, N, seed=6)
    args = [t.requires_grad_() for t in (u, w, a, B, C, h0)]
    assert torch.autograd.gradcheck(lambda *t: lt.scan(*t, spans), args)


def test_scan_is_the_unrolled_sum():
    b, L, H, P, N = 1, 7, 1, 2, 3
    u, B, C = rand(b, L, H, P, seed=1), rand(b, L, 1, N, seed=2), rand(b, L, 1, N, seed=3)
    w, a = rand(b, L, H, seed=4).abs(), -rand(b, L, H, seed=5).abs()
    y, _ = lt.scan(u, w, a, B, C, torch.zeros(1, H, P, N, dtype=torch.float64), lt.spans_of(L, b, None))
    for t in range(L):
        want = sum(torch.exp(a[0, s + 1:t + 1, 0].sum()) * w[0, s, 0] * u[0, s, 0]
                   * (C[0, t, 0] @ B[0, s, 0]) for s in range(t + 1))
        assert torch.allclose(y[0, t, 0], want, rtol=1e-12, atol=1e-12)


def test_heads_reference_gradients_against_differences():
    """dA, ddelta and ddelta_bias as heads_reference puts them together."""
    b, L, H, P, G, N = 2, 4, 2, 2, 2, 2
    t = {"u": rand(b, L, H, P, seed=1), "delta": rand(b, L, H, seed=2), "A": -rand(H, seed=3).abs(),
         "B": rand(b, L, G, N, seed=4), "C": rand(b, L, G, N, seed=5), "D": rand(H, seed=6),
         "bias": rand(H, seed=7), "h0": rand(b, H, P, N, seed=8)}
    dy, dlast = rand(b, L, H, P, seed=9), rand(b, H, P, N, seed=10)

    def loss(**kw):
        r, _ = lt.heads_reference(**{**t, **kw}, lens=None)
        return float((r["y"] * dy).sum() + (r["last_state"] * dlast).sum())

    got, size = lt.heads_reference(**t, lens=None, dy=dy, dlast=dlast)
    h = 1e-6
    for name, key in (("A", "dA"), ("delta", "ddelta"), ("bias", "ddelta_bias"), ("D", "dD"),
                      ("u", "du"), ("h0", "dh0")):
        flat = t[name].flatten()
        for i in range(0, flat.numel(), max(1, flat.numel() // 5)):
            e = torch.zeros_like(flat)
            e[i] = h
            e = e.view_as(t[name])
            want = (loss(**{name: t[name] + e}) - loss(**{name: t[name] - e})) / (2 * h)
            assert math.isclose(got[key].flatten()[i], want, rel_tol=1e-5, abs_tol=1e-6), (name, i)
    for k in got:
        assert (size["decays"][k] >= 0).all() and (size[k] >= got[k].abs() - 1e-12).all(), k


def test_conv_and_norm_gradients_against_differences():
    x, w, bias = rand(1, 6, 3, seed=1), rand(3, 4, seed=2), rand(3, seed=3)
    state, dy = rand(3, 3, 3, seed=4), rand(1, 6, 3, seed=5)
    lens = [1, 0, 5]
    got, _ = lt.conv_reference(x, w, bias, state, lens, dy=dy)
    h = 1e-6
    for k, (name, key) in enumerate((("x", "dx"), ("weight", "dweight"), ("bias", "dbias"),
                                     ("state", "dconv_state"))):
        args = {"x": x, "weight": w, "bias": bias, "state": state}
        flat = args[name].flatten()
        for i in range(0, flat.numel(), 2):
            e = torch.zeros_like(flat)
            e[i] = h
            lo, hi = (lt.conv_reference(**{**args, name: args[name] + s * e.view_as(args[name])},
                                        lens=lens)[0]["y"] for s in (-1, 1))
            want = float(((hi - lo) * dy).sum()) / (2 * h)
            assert math.isclose(got[key].flatten()[i], want, rel_tol=1e-5, abs_tol=1e-7), (name, i)
    s, wt, z = rand(2, 6, seed=1), rand(6, seed=2), rand(2, 6, seed=3)
    dy, dr = rand(2, 6, seed=4), rand(2, 6, seed=5)
    got = lt.norm_reference(s, wt, z, 3, dy=dy, dresidual=dr)
    for name, key in (("s", "dx"), ("weight", "dweight"), ("z", "dz")):
        args = {"s": s, "weight": wt, "z": z}
        flat = args[name].flatten()
        for i in range(flat.numel()):
            e = torch.zeros_like(flat)
            e[i] = h
            e = e.view_as(args[name])
            lo, hi = (lt.norm_reference(**{**args, name: args[name] + q * e}, group=3)["y"]
                      for q in (-1, 1))
            want = float(((hi - lo) * dy).sum()) / (2 * h)
            if name == "s":
                want += float(dr.flatten()[i])
            assert math.isclose(got[key].flatten()[i], want, rel_tol=1e-4, abs_tol=1e-6), (name, i)
