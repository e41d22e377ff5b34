"""Pins of the layer-operator oracle (oracle/layer_oracle.py) to things other
than itself: torch's fp64 routines and autograd, and central differences of
its own forwards (no GPU)."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O


def _rand(shape, seed, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


def _t(a):
    return torch.tensor(a, dtype=torch.float64, requires_grad=True)


def _torch_act(z, act):
    F = torch.nn.functional
    return F.gelu(z) if act == "gelu" else F.silu(z) if act == "silu" else z


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_activations_match_torch_and_their_differences(act):
    z = np.linspace(-9, 9, 181)
    np.testing.assert_allclose(O.act_value(z, act), _torch_act(torch.tensor(z), act).numpy(),
                               rtol=1e-12, atol=1e-15)
    h = 1e-5
    diff = (O.act_value(z + h, act) - O.act_value(z - h, act)) / (2 * h)
    np.testing.assert_allclose(O.act_slope(z, act), diff, rtol=0, atol=1e-9)


@pytest.mark.parametrize("rows,C", [(1, 1), (3, 2), (7, 13)])
def test_layer_norm_matches_torch_autograd(rows, C):
    x, g, b = _rand((rows, C), 1, 2.0) + 3, _rand(C, 2), _rand(C, 3)
    dy, dres = _rand((rows, C), 4), _rand((rows, C), 5)
    tx, tg, tb = _t(x), _t(g), _t(b)
    ty = torch.nn.functional.layer_norm(tx, (C,), tg, tb, 1e-5)
    y, mean, rstd = O.layer_norm_fwd(x, g, b, 1e-5)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=0, atol=1e-11)
    (ty * torch.tensor(dy)).sum().backward()
    dx, dg, db = O.layer_norm_bwd(x, dy, mean, rstd, g, dres)
    np.testing.assert_allclose(dx, tx.grad.numpy() + dres, rtol=0, atol=1e-9)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=0, atol=1e-10)
    np.testing.assert_allclose(db, tb.grad.numpy(), rtol=0, atol=1e-10)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_matches_torch_autograd(act):
    x, w, b, r = _rand((5, 6), 1), _rand((4, 6), 2), _rand(4, 3), _rand((5, 4), 4)
    dy, add = _rand((5, 4), 5), _rand((5, 6), 6)
    tx, tw, tb = _t(x), _t(w), _t(b)
    ty = _torch_act(torch.nn.functional.linear(tx, tw, tb), act) + torch.tensor(r)
    y, z = O.linear_fwd(x, w, b, act, r)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=0, atol=1e-12)
    (ty * torch.tensor(dy)).sum().backward()
    dx, dw, db = O.linear_bwd(x, w, dy, act, z, add)
    np.testing.assert_allclose(dx, tx.grad.numpy() + add, rtol=0, atol=1e-11)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=0, atol=1e-11)
    np.testing.assert_allclose(db, tb.grad.numpy(), rtol=0, atol=1e-11)


def _ffn(C=4, H=5, rows=6):
    return (_rand((rows, C), 1), _rand((2, H, C), 2), _rand((2, H), 3), _rand((C, H), 4),
            _rand(C, 5), _rand((rows, C), 6))


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_gated_ffn_matches_torch_autograd(act):
    x, wi, bi, wo, bo, dy = _ffn()
    add = _rand(x.shape, 7)
    tx, twi, tbi, two, tbo = map(_t, (x, wi, bi, wo, bo))
    F = torch.nn.functional
    ty = F.linear(_torch_act(F.linear(tx, twi[0], tbi[0]), act) * F.linear(tx, twi[1], tbi[1]),
                  two, tbo)
    np.testing.assert_allclose(O.gated_ffn_fwd(x, wi, bi, wo, bo, act), ty.detach().numpy(),
                               rtol=0, atol=1e-12)
    (ty * torch.tensor(dy)).sum().backward()
    got = O.gated_ffn_bwd(x, wi, bi, wo, dy, act, add)
    for a, t, extra in zip(got, (tx, twi, tbi, two, tbo), (add, 0, 0, 0, 0)):
        np.testing.assert_allclose(a, t.grad.numpy() + extra, rtol=0, atol=1e-11)


def _difference(f, a, dy, h=1e-6):
    """d sum(f(a) dy) / da by central differences."""
    g = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        p, m = a.copy(), a.copy()
        p[i] += h
        m[i] -= h
        g[i] = ((f(p) - f(m)) * dy).sum() / (2 * h)
    return g


def test_backwards_match_central_differences():
    x, wi, bi, wo, bo, dy = _ffn(C=3, H=4, rows=3)
    dx, dwi, dbi, dwo, dbo = O.gated_ffn_bwd(x, wi, bi, wo, dy, "gelu")
    f = O.gated_ffn_fwd
    for got, arg, fn in ((dx, x, lambda v: f(v, wi, bi, wo, bo, "gelu")),
                         (dwi, wi, lambda v: f(x, v, bi, wo, bo, "gelu")),
                         (dbi, bi, lambda v: f(x, wi, v, wo, bo, "gelu")),
                         (dwo, wo, lambda v: f(x, wi, bi, v, bo, "gelu")),
                         (dbo, bo, lambda v: f(x, wi, bi, wo, v, "gelu"))):
        np.testing.assert_allclose(got, _difference(fn, arg, dy), rtol=0, atol=2e-8)
    g, b = _rand(3, 8), _rand(3, 9)
    _, mean, rstd = O.layer_norm_fwd(x, g, b)
    dx, dg, db = O.layer_norm_bwd(x, dy, mean, rstd, g)
    n = O.layer_norm_fwd
    for got, arg, fn in ((dx, x, lambda v: n(v, g, b)[0]), (dg, g, lambda v: n(x, v, b)[0]),
                         (db, b, lambda v: n(x, g, v)[0])):
        np.testing.assert_allclose(got, _difference(fn, arg, dy), rtol=0, atol=2e-7)
    w, bias = _rand((2, 3), 10), _rand(2, 11)
    d2 = _rand((3, 2), 12)
    _, z = O.linear_fwd(x, w, bias, "silu")
    dx, dw, db = O.linear_bwd(x, w, d2, "silu", z)
    lin = lambda *a: O.linear_fwd(*a, "silu")[0]
    for got, arg, fn in ((dx, x, lambda v: lin(v, w, bias)), (dw, w, lambda v: lin(x, v, bias)),
                         (db, bias, lambda v: lin(x, w, v))):
        np.testing.assert_allclose(got, _difference(fn, arg, d2), rtol=0, atol=2e-8)


def test_a_wrong_sign_or_a_missing_term_is_caught():
    # the comparisons above tell a plausible mistake from the right formula
    x, wi, bi, wo, bo, dy = _ffn(C=3, H=4, rows=3)
    g, u = x @ wi[0].T + bi[0], x @ wi[1].T + bi[1]
    dh = dy @ wo
    right = O.gated_ffn_bwd(x, wi, bi, wo, dy, "silu")[0]
    swapped = (dh * O.act_value(g, "silu")) @ wi[0] + (dh * u * O.act_slope(g, "silu")) @ wi[1]
    assert np.abs(right - swapped).max() > 1e-2
    _, mean, rstd = O.layer_norm_fwd(x)
    full = O.layer_norm_bwd(x, dy, mean, rstd)[0]
    no_mean = rstd[:, None] * dy
    assert np.abs(full - no_mean).max() > 1e-2


def test_every_function_of_the_oracle_is_pinned_here():
    import re
    text = open(__file__).read()
    assert [n for n in O.__all__ if not re.search(r"\bO\.%s\b" % n, text)] == []
