"""The layer norm's pipelines over many blocks: every warp goes several times
around its ring of stages, so that stages are used again, the barriers' parities
flip, the next block's statistics are fetched ahead and the sums of gamma's and
beta's gradients run over blocks.  Against the fp64 oracle, elementwise, with the
bounds of test_gpu_layer_ops."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
import windowed_attention_implicit_b200 as R
from tests.test_gpu_layer_ops import H, U, _done, _ln_case, _ln_fwd_bounds, _np, _rand, _within, bf, f32

pytestmark = pytest.mark.gpu

# Blocks a warp, forward and backward, on 148 SMs.  Whole vectors: 96 and 192
# channels bf16 4 and 8, fp32 8 and 16; 512 4 and 11, 8 and 23; 768 4 and 8, 6 and 17.
# Single elements (odd sizes, blocks that begin off a 16-byte address): 10 4 and 5, 4
# and 7; 33 4 and 9, 12 and 18; 125 4 and 11, 8 and 21; 333 3 and 6, 4 and 11; 601 4
# and 11, 7 and 15 with two stages; 903 4 and 7.
SHAPES = [(150003, 96), (75001, 192), (40000, 512), (20000, 768), (606001, 10), (460003, 33),
          (150001, 125), (30001, 333), (30001, 601), (20003, 903)]
DTYPES = [bf, f32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_forward_around_the_ring(rows, C, dtype):
    x, g, b = _ln_case(rows, C, dtype)
    xd, gd, bd = x.cuda(), g.cuda(), b.cuda()
    y, mean, rstd = R.rib_layer_norm_fwd(xd, gd, bd)
    R.rib_layer_norm_fwd(xd, gd, bd, y=xd)   # in place
    _done()
    assert torch.equal(xd, y)
    ref, bound = _ln_fwd_bounds(x, g, b, 1e-5, H if dtype == bf else 2 * U)
    for got, r, e, n in zip((y, mean, rstd), ref, bound, ("y", "mean", "rstd")):
        _within(got, r, e, n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_backward_around_the_ring(rows, C, dtype):
    x, g, _ = _ln_case(rows, C, dtype)
    dy, dres = _rand((rows, C), 11, dtype=dtype), _rand((rows, C), 12, dtype=dtype)
    X, mu = _np(x), None
    mean = torch.tensor(X.mean(1), dtype=f32)
    mu = _np(mean)[:, None]
    rstd = torch.tensor(1 / np.sqrt(((X - mu) ** 2).mean(1) + 1e-5), dtype=f32)
    d = [t.cuda() for t in (x, dy, mean, rstd, g)]
    got = R.rib_layer_norm_bwd(*d, dres=dres.cuda())
    over_dres, over_dy = dres.cuda(), d[1].clone()
    same = R.rib_layer_norm_bwd(*d, dres=over_dres, dx=over_dres)
    R.rib_layer_norm_bwd(d[0], over_dy, *d[2:], dres=dres.cuda(), dx=over_dy)
    bare = R.rib_layer_norm_bwd(*d)                       # two arrays a stage
    zero = R.rib_layer_norm_bwd(*d, dres=torch.zeros_like(d[0]))
    _done()
    assert torch.equal(over_dres, got["dx"]) and torch.equal(over_dy, got["dx"])
    assert all(torch.equal(same[n], got[n]) for n in got)
    assert all(torch.equal(bare[n], zero[n]) for n in bare)
    dx, dg, db = O.layer_norm_bwd(x, dy, mean, rstd, g, dres)
    D, G, A, rs = _np(dy), _np(g), _np(dres), _np(rstd)[:, None]
    xh, gd = (X - mu) * rs, D * G
    exh = 2 * U * np.abs(xh) + 2 * U * rs * (np.abs(X) + np.abs(mu))
    m1, m2 = gd.mean(1, keepdims=True), (gd * xh).mean(1, keepdims=True)
    e1 = 70 * U * np.abs(gd).mean(1, keepdims=True)
    e2 = 70 * U * np.abs(gd * xh).mean(1, keepdims=True) + (np.abs(gd) * exh).mean(1, keepdims=True)
    ex = rs * (e1 + np.abs(xh) * e2 + exh * np.abs(m2) +
               6 * U * (np.abs(gd) + np.abs(m1) + np.abs(xh * m2))) + 2 * U * (np.abs(A) + np.abs(dx))
    half = H if dtype == bf else 2 * U
    _within(got["dx"], dx, ex + half * (np.abs(dx) + ex), "dx")
    n = (rows + 32) * U
    _within(got["dgamma"], dg, n * np.abs(D * xh).sum(0) + (np.abs(D) * exh).sum(0), "dgamma")
    _within(got["dbeta"], db, n * np.abs(D).sum(0), "dbeta")


@pytest.mark.parametrize("C", [192, 333, 1025])
def test_backward_of_rows_of_tiny_spread(C):
    """fp32 rows of spread 1e-24 without an eps: rstd is 1e24, whose square is
    beyond fp32, while dx, about 1e24, is not."""
    rows = 64
    x = _rand((rows, C), 5, 1.0, f32) * 1e-24
    dy = _rand((rows, C), 6, 1.0, f32)
    X = _np(x)
    mean = torch.tensor(X.mean(1), dtype=f32)
    mu = _np(mean)[:, None]
    rstd = torch.tensor(1 / np.sqrt(((X - mu) ** 2).mean(1)), dtype=f32)
    got = R.rib_layer_norm_bwd(x.cuda(), dy.cuda(), mean.cuda(), rstd.cuda())
    _done()
    dx, dg, db = O.layer_norm_bwd(x, dy, mean, rstd, None, None)
    D, rs = _np(dy), _np(rstd)[:, None]
    xh = (X - mu) * rs
    exh = 2 * U * np.abs(xh) + 2 * U * rs * (np.abs(X) + np.abs(mu))
    m1, m2 = D.mean(1, keepdims=True), (D * xh).mean(1, keepdims=True)
    e1 = 70 * U * np.abs(D).mean(1, keepdims=True)
    e2 = 70 * U * np.abs(D * xh).mean(1, keepdims=True) + (np.abs(D) * exh).mean(1, keepdims=True)
    ex = rs * (e1 + np.abs(xh) * e2 + exh * np.abs(m2) + 6 * U * (np.abs(D) + np.abs(m1) + np.abs(xh * m2)))
    _within(got["dx"], dx, ex + 2 * U * (2 * np.abs(dx) + ex), "dx")
    n = (rows + 32) * U
    _within(got["dgamma"], dg, n * np.abs(D * xh).sum(0) + (np.abs(D) * exh).sum(0), "dgamma")
    _within(got["dbeta"], db, n * np.abs(D).sum(0), "dbeta")
