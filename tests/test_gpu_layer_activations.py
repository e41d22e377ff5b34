"""gelu and silu over all values that have a normal bf16 result, through every
kernel that forms them: the tiled product's epilogue, the few-row kernel, the
feed-forward block's forms and the backward.

Bounds, relative to the exact value: H = 2^-8 for the one rounding to bf16, and
2^-14 for the approximation in fp32: a polynomial good to 4.6e-6 (a quarter of
2^-16), a reciprocal and an exponential of an ulp or two, and the exponent's own
rounding, |x| 2^-24 2 for x up to 126 (1.5e-5 = 2^-16): below 2^-14 in sum.
Against bf16 steps that is 1 / 64.  Values whose exponential falls below the
smallest normal fp32 are flushed to zero.
"""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
import windowed_attention_implicit_b200 as R

pytestmark = pytest.mark.gpu

bf, f32 = torch.bfloat16, torch.float32
H, APPROX = 2.0 ** -8, 2.0 ** -14
TINY = 2.0 ** -126


def _z():
    """Every bf16 value from 2^-10 to 96 in size, both signs, and zeros: 8192 in all."""
    b = torch.arange(0x3A80, 0x42C1, dtype=torch.int32)
    z = torch.cat([b, b + 0x8000])
    z = torch.cat([z, torch.zeros(8192 - z.numel(), dtype=torch.int32)])
    return (z << 16).view(f32).to(bf)


def _np(t):
    return t.detach().double().cpu().numpy()


def _done():
    torch.cuda.synchronize()
    code, site = R.rib_last_status()
    assert code == 0, f"{R.rib_status_string(code)} at site {site}"


def _check(got, z, act, what):
    got, want = _np(got).ravel(), O.act_value(_np(z).ravel(), act)
    # the product |z| e^-(...) of a flushed exponential: nothing of it is left
    lost = np.maximum(np.abs(_np(z).ravel()), 1) * TINY
    err = np.abs(got - want)
    bound = (H + APPROX) * np.abs(want) + lost
    i = np.argmax(err / bound)
    assert err[i] <= bound[i], (what, _np(z).ravel()[i], got[i], want[i])


@pytest.mark.parametrize("rows", [1, 2, 4, 8, 64, 512])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_value_for_any_number_of_rows(act, rows):
    eye = torch.eye(16, dtype=bf).cuda()
    for part in _z().view(-1, rows, 16):
        y, _ = R.rib_linear_fwd(part.cuda(), eye, act=act)
        _done()
        _check(y, part, act, f"{rows} rows")


@pytest.mark.parametrize("rows", [4, 512, 20000])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_value_in_the_feed_forward(act, rows):
    """Few rows, two products and one kernel: u is 1, so y is act(x) rounded to
    bf16 as h and not changed after that."""
    z = _z()
    x = z.repeat(-(-rows * 16 // z.numel()))[:rows * 16].view(rows, 16)
    if rows == 4:   # where gelu's tail is
        x = torch.linspace(-13, -0.5, 64).to(bf).view(rows, 16)
    assert (R.rib_gated_ffn_fwd_workspace(rows, 16, 16) == 0) == (rows == 20000)
    eye = torch.eye(16, dtype=bf)
    w_in, b_in = torch.stack([eye, torch.zeros_like(eye)]), torch.stack([torch.zeros(16), torch.ones(16)])
    y = R.rib_gated_ffn_fwd(x.cuda(), R.GatedFfn.from_params(w_in, b_in, eye, None), act=act)
    _done()
    _check(y, x, act, "feed-forward")


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_value_in_the_feed_forward_backward(act):
    """dw_out = dy^T h with one row of dy set is that row of h."""
    z = _z()
    x = z.view(-1, 128)
    C = 128
    eye = torch.eye(C, dtype=bf)
    ffn = R.GatedFfn.from_params(torch.stack([eye, torch.zeros_like(eye)]),
                                 torch.stack([torch.zeros(C), torch.ones(C)]), eye, None)
    for r in range(x.shape[0]):
        dy = torch.zeros(x.shape, dtype=bf)
        dy[r, 0] = 1
        g = R.rib_gated_ffn_bwd(x.cuda(), ffn, dy.cuda(), act=act)
        _done()
        _check(g["dw_out"][0], x[r], act, f"row {r}")


@pytest.mark.parametrize("rows", [4, 300])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slope_in_its_tail(act, rows):
    """The slope's tail in relative terms too: z phi is much the larger part of it
    there.  Where it passes through zero (gelu's at -0.75, silu's at -1.28) the
    bound is that of its parts."""
    z = torch.cat([torch.linspace(-12.5, -1.5, rows * 8), torch.linspace(-1.5, 8, rows * 8)]).to(bf).view(rows, 16)
    one, eye = torch.ones_like(z).cuda(), torch.eye(16, dtype=bf).cuda()
    g = R.rib_linear_bwd(z.cuda(), eye, one, act=act, pre=z.cuda())
    _done()
    Z = _np(z)
    want = O.act_slope(Z, act)
    parts = np.abs(want) + 2 * np.abs(O.act_value(Z, act))
    err = np.abs(_np(g["dx"]) - want)
    # rounded as dz and, unchanged by the product with ones and zeros, as dx
    assert (err <= H * (np.abs(want) + APPROX * parts) + APPROX * parts).all()


@pytest.mark.parametrize("rows", [1, 4, 8, 9, 300])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_infinite_values_give_the_limits(act, rows):
    """An infinite pre-activation, here from the bias: 0 and infinity, and slopes
    0 and 1, however many rows there are; the other columns stay as they are."""
    inf = float("inf")
    eye = torch.eye(16, dtype=bf).cuda()
    x = torch.linspace(-3, 3, rows * 16).to(bf).view(rows, 16).cuda()
    b = torch.zeros(16, device="cuda")
    clean, _ = R.rib_linear_fwd(x, eye, b, act=act)
    b[3], b[8] = -inf, inf
    y, pre = R.rib_linear_fwd(x, eye, b, act=act, save_pre=True)
    g = R.rib_linear_bwd(x, eye, torch.ones_like(x), act=act, pre=pre)
    _done()
    rest = [i for i in range(16) if i not in (3, 8)]
    assert (y[:, 3] == 0).all() and (y[:, 8] == inf).all() and torch.equal(y[:, rest], clean[:, rest])
    assert (g["dx"][:, 3] == 0).all() and (g["dx"][:, 8] == 1).all() and torch.isfinite(g["dx"]).all()
    assert g["db"][3] == 0 and g["db"][8] == rows
