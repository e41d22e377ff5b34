"""The gated feed-forward's forward in one kernel, at the widths, hidden sizes and
row counts where its tiles, chunks and last MMA steps end, against the fp64 oracle
with the bounds of test_gpu_layer_ops."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
import windowed_attention_implicit_b200 as R
from tests.test_gpu_layer_ops import H, _done, _ffn_case, _ffn_dev, _ffn_inner, _mma, _np, _within

pytestmark = pytest.mark.gpu

# The one kernel runs where there are at least three row tiles of 256 for each 64
# hidden channels.  Channels around whole k-steps and whole column units, hidden
# sizes around whole chunks and whole MMA steps, rows of one to three tiles a CTA
# pair with a last tile of one row, of half a pair and of all of it.
SHAPES = [(513, 256, 8), (513, 8, 64), (513, 192, 16), (1281, 64, 72), (1409, 128, 128), (1537, 200, 120),
          (1536, 232, 96), (2049, 72, 136), (2176, 136, 192), (4000, 256, 248), (769, 96, 24), (3073, 192, 200),
          (19201, 32, 320), (38145, 64, 40), (37889, 256, 16), (57000, 192, 72)]


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("rows,C,Hd", SHAPES)
def test_one_kernel_forward(rows, C, Hd, act):
    assert R.rib_gated_ffn_fwd_workspace(rows, C, Hd) == 0
    x, wi, bi, wo, bo, r = _ffn_case(rows, C, Hd)
    full, none = _ffn_dev(wi, bi, wo, bo), _ffn_dev(wi, None, wo, None)
    xd, rd = x.cuda(), r.cuda()
    y = R.rib_gated_ffn_fwd(xd, full, act=act, residual=rd)
    again = R.rib_gated_ffn_fwd(xd, full, act=act, residual=rd)
    bare = R.rib_gated_ffn_fwd(xd, none, act=act)
    _done()
    assert torch.equal(y, again)
    for got, b1, b2, res in ((y, bi, bo, r), (bare, None, None, None)):
        ref = O.gated_ffn_fwd(x, wi, b1, wo, b2, act, res)
        *_, h, _, _, _, eh = _ffn_inner(x, wi, b1, act)
        W = np.abs(_np(wo)).T
        extra = (0 if b2 is None else np.abs(_np(b2))) + (0 if res is None else np.abs(_np(res)))
        e = eh @ W + _mma(Hd) * (np.abs(h) @ W + extra)
        _within(got, ref, e + H * (np.abs(ref) + e), "y", H)


def test_many_calls_give_the_same_bits():
    """Hand-overs between the CTAs of a pair that came early now and then would show
    as a difference between calls."""
    x, wi, bi, wo, bo, r = _ffn_case(40000, 192, 384)
    ffn, x, r = _ffn_dev(wi, bi, wo, bo), x.cuda(), r.cuda()
    want = R.rib_gated_ffn_fwd(x, ffn, residual=r)
    y = torch.empty_like(want)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        R.rib_gated_ffn_fwd(x, ffn, residual=r, y=y)
        bad += (y != want).sum()
    _done()
    assert int(bad) == 0


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("rows,C,Hd", [(1, 1024, 2816), (2, 16, 1512), (1, 8, 8), (3, 96, 384), (5, 192, 768),
                                       (8, 64, 256)])
def test_few_rows_keep_h_in_fp32(rows, C, Hd, act):
    """Without the tensor cores h is not rounded: what separates y from the formula
    is y's own rounding, fp32 sums of at most (C + Hd) terms and the activation's
    error, which the tiled form's bounds have beside a rounding of every h."""
    x, wi, bi, wo, bo, r = _ffn_case(rows, C, Hd)
    y = R.rib_gated_ffn_fwd(x.cuda(), _ffn_dev(wi, bi, wo, bo), act=act, residual=r.cuda())
    _done()
    ref = O.gated_ffn_fwd(x, wi, bi, wo, bo, act, r)
    *_, h, _, _, _, eh = _ffn_inner(x, wi, bi, act)
    eh = (eh - H * np.abs(h)) / (1 + H)          # without the rounding of h
    W = np.abs(_np(wo)).T
    e = eh @ W + _mma(Hd) * (np.abs(h) @ W + np.abs(_np(bo)) + np.abs(_np(r)))
    _within(y, ref, e + H * (np.abs(ref) + e), "y")
