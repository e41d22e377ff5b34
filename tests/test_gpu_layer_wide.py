"""The feed-forward's backward at many channels, whose sums over the channels are
cut into pieces: values against the fp64 oracle, and the drift of its fp32 sums."""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
import windowed_attention_implicit_b200 as R
from tests.test_gpu_layer_ops import _done, _ffn_case, _ffn_dev, _np, bf

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def _rel(got, ref):
    return np.linalg.norm(_np(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("rows,C,Hd", [(700, 1600, 264), (300, 2048, 72), (2500, 520, 200), (40000, 584, 64),
                                       (1, 776, 1032), (129, 768, 64), (65, 4096, 40)])
def test_wide_backward(rows, C, Hd, act):
    """An output rounded to bf16 has a 2-norm error of at most H / sqrt 3 per rounding,
    and two roundings lie between it and the formula (h, dg or du, and its own):
    below H.

    The bias gradients are fp32 sums of dg and du.  A truncating addition loses 0.36
    units in the last place, 2^-23, of the running sum on average (half a step, whose
    size is 0.72 of the value), and the running sum of a chain of n grows as
    sqrt(k / n): n 2/3 0.36 2^-23 of the result, 0.69e-6 for the 24 additions of a
    piece.  dg and du carry the drift of two such factors, the fp32 arithmetic behind
    them a few 2^-24: 1.8e-6.  (Chains of all the channels drift by 3.7e-6 at 2048.)"""
    x, wi, bi, wo, bo, dy = _ffn_case(rows, C, Hd)
    ffn = _ffn_dev(wi, bi, wo, bo)
    args = x.cuda(), ffn, dy.cuda()
    got = R.rib_gated_ffn_bwd(*args, act=act, dw_dtype=bf)
    again = R.rib_gated_ffn_bwd(*args, act=act, dw_dtype=bf)
    _done()
    assert all(torch.equal(got[k], again[k]) for k in got)
    ref = dict(zip(("dx", "dw_in", "db_in", "dw_out", "db_out"), O.gated_ffn_bwd(x, wi, bi, wo, dy, act)))
    for n in ("dx", "dw_in", "dw_out"):
        assert _rel(got[n], ref[n]) <= H, (n, _rel(got[n], ref[n]))
    assert _rel(got["db_in"], ref["db_in"]) <= 1.8e-6, _rel(got["db_in"], ref["db_in"])
    assert _rel(got["db_out"], ref["db_out"]) <= 1.8e-6
