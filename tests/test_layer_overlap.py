"""Outputs that overlap what a layer operator still reads are refused, also where
they only begin inside it; an output in the place of an input that allows it
gives what it gives elsewhere."""
import pytest
import torch

import rib_inputs as I
import windowed_attention_implicit_b200 as R
from tests.test_layer_ops_host import ARG, FAKE, ffn_bwd, ffn_fwd, lin_bwd, lin_fwd, ln_bwd, ln_fwd
from windowed_attention_implicit_b200 import _abi

bf, f32 = torch.bfloat16, torch.float32

# output, the input (or output) it runs into; 4 rows of 96 channels are 768 bytes, so
# 256 bytes further on is inside, and 1 << 20 apart is not
PARTIAL = [
    (ln_fwd, "y", "x"), (ln_fwd, "mean", "x"), (ln_fwd, "rstd", "y"), (ln_fwd, "y", "gamma"),
    (lin_fwd, "y", "x"), (lin_fwd, "pre", "x"), (lin_fwd, "y", "residual"), (lin_fwd, "y", "pre"),
    (lin_fwd, "pre", "residual"), (lin_bwd, "dx", "x"), (lin_bwd, "dx", "dy"), (lin_bwd, "dx", "dx_add"),
    (ffn_fwd, "y", "x"), (ffn_fwd, "y", "residual"), (ffn_bwd, "dx", "x"), (ffn_bwd, "dx", "dy"),
    (ffn_bwd, "dx", "dx_add"),
]
BUFFERS = {
    ln_fwd: ("x", "gamma", "beta", "y", "mean", "rstd"),
    lin_fwd: ("x", "w", "bias", "residual", "pre", "y"),
    lin_bwd: ("x", "w", "pre", "dy", "dx_add", "dx", "dw", "db"),
    ffn_fwd: ("x", "w_in", "b_in", "w_out", "b_out", "residual", "y"),
    ffn_bwd: ("x", "w_in", "b_in", "w_out", "dy", "dx_add", "dx", "dw_in", "db_in", "dw_out", "db_out"),
}


@pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in pointers: only where nothing can be launched")
@pytest.mark.parametrize("fn,out,other", PARTIAL, ids=[f"{f.__name__}-{o}-{i}" for f, o, i in PARTIAL])
def test_a_partial_overlap_is_refused(fn, out, other):
    apart = {n: FAKE + ((i + 1) << 20) for i, n in enumerate(BUFFERS[fn])}
    assert fn(**apart) not in (_abi.RIB_OK, ARG)    # only the missing device is left to refuse
    for shift in (256,) if out in ("mean", "rstd") else (256, -256):   # those are 16 bytes long
        assert fn(**{**apart, out: apart[other] + shift}) == ARG
    assert fn(**{**apart, out: apart[other] + (1 << 19)}) not in (_abi.RIB_OK, ARG)


def _case():
    r = lambda i, *s, std=1.0: I.randn(s, seed=i, std=std).to(bf).cuda()
    return dict(x=r(1, 64, 64), dy=r(2, 64, 64), w=r(3, 64, 64, std=0.1), w_in=r(5, 2, 64, 64, std=0.1),
                w_out=r(6, 64, 64, std=0.1))


def _refused(fn, *a, **kw):
    with pytest.raises(R.RibError) as e:
        fn(*a, **kw)
    assert e.value.code == ARG


@pytest.mark.gpu
def test_overlaps_are_refused_before_a_launch():
    c = _case()
    x, dy, w = c["x"], c["dy"], c["w"]
    ffn = R.GatedFfn(c["w_in"], None, c["w_out"], None)
    flat = torch.zeros(3 * 64 * 64, dtype=bf, device="cuda")
    flat[:4096] = x.view(-1)
    head, inside = flat[:4096].view(64, 64), flat[2048:2048 + 4096].view(64, 64)
    before = flat.clone()
    g = torch.ones(64, device="cuda")
    y, mean, rstd = R.rib_layer_norm_fwd(x, g)
    _refused(R.rib_layer_norm_fwd, head, g, y=inside)
    stats = torch.zeros(96, device="cuda")
    _refused(R.rib_layer_norm_fwd, head, mean=stats[:64], rstd=stats[32:])
    _refused(R.rib_layer_norm_bwd, head, dy, mean, rstd, dx=inside)
    _refused(R.rib_layer_norm_bwd, x, head, mean, rstd, dx=inside)
    _refused(R.rib_layer_norm_bwd, x, dy, mean, rstd, dres=head, dx=inside)
    _refused(R.rib_layer_norm_bwd, x, dy, mean, rstd, dgamma=stats[:64], dbeta=stats[32:])
    _refused(R.rib_linear_fwd, head, w, y=inside)
    _refused(R.rib_linear_fwd, x, head, y=inside)
    _refused(R.rib_linear_fwd, x, w, residual=head, y=inside)
    _refused(R.rib_linear_fwd, x[:2], head, y=inside[:2])       # few rows
    _refused(R.rib_linear_bwd, x, head, dy, dx=inside)
    _refused(R.rib_linear_bwd, head, w, dy, dw=inside)
    _refused(R.rib_linear_bwd, x, w, head, dw=inside)
    _refused(R.rib_linear_bwd, x, w, dy, dx=head, dw=inside)
    _refused(R.rib_gated_ffn_fwd, head, ffn, y=inside)
    _refused(R.rib_gated_ffn_fwd, x, R.GatedFfn(c["w_in"], None, head, None), y=inside)
    _refused(R.rib_gated_ffn_bwd, x, ffn, head, dx=inside, dw_dtype=bf)
    _refused(R.rib_gated_ffn_bwd, head, ffn, dy, dw_out=inside, dw_dtype=bf)
    _refused(R.rib_gated_ffn_bwd, x, ffn, dy, dx=head, dw_out=inside)
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and R.rib_last_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 64, 300, 20001])
def test_outputs_in_the_place_of_inputs(rows):
    """dx over x, dy and dres; the feed-forward's y over x and over x that is the
    residual too, in its few-row, two-product and one-kernel forms."""
    for C in (64, 33):
        for dt in (bf, f32):
            x, dy, add = (I.randn((rows, C), seed=i).to(dt).cuda() for i in (1, 2, 3))
            _, mean, rstd = R.rib_layer_norm_fwd(x)
            want = R.rib_layer_norm_bwd(x, dy, mean, rstd, dres=add)
            for n in range(3):
                t = [x.clone(), dy.clone(), add.clone()]
                got = R.rib_layer_norm_bwd(t[0], t[1], mean, rstd, dres=t[2], dx=t[n])
                assert got["dx"].data_ptr() == t[n].data_ptr()
                assert all(torch.equal(got[k], want[k]) for k in want)
    c = _case()
    ffn = R.GatedFfn(c["w_in"], None, c["w_out"], None)
    x = I.randn((rows, 64), seed=9).to(bf).cuda()
    plain, res = R.rib_gated_ffn_fwd(x, ffn), R.rib_gated_ffn_fwd(x, ffn, residual=x)
    a, b = x.clone(), x.clone()
    R.rib_gated_ffn_fwd(a, ffn, y=a)
    R.rib_gated_ffn_fwd(b, ffn, residual=b, y=b)
    torch.cuda.synchronize()
    assert torch.equal(a, plain) and torch.equal(b, res)
    assert R.rib_last_status()[0] == 0


def test_no_rows_looks_at_no_map():
    """A map without rows may have any address, an odd one too."""
    odd = FAKE + 1
    assert ln_fwd(rows=0, x=odd, y=odd, gamma=odd) == _abi.RIB_OK
    assert ln_bwd(rows=0, x=odd, dy=odd, dx=odd, mean=odd, dgamma=None, dbeta=None) == _abi.RIB_OK
    assert lin_fwd(rows=0, x=odd, w=odd, y=odd) == _abi.RIB_OK
    assert lin_bwd(rows=0, x=odd, w=odd, pre=odd, dy=odd, dx_add=odd, dx=odd, dw=None, db=None) == _abi.RIB_OK
    assert ffn_fwd(rows=0, x=odd, y=odd, residual=odd) == _abi.RIB_OK
    # the sums are written: refused where they lie, before anything is
    assert lin_bwd(rows=0, x=odd, dw=odd, db=None) == _abi.RIB_ERR_ALIGN
    assert ffn_bwd(rows=0, x=odd, dy=odd, dx=odd, dw_in=odd) == _abi.RIB_ERR_ALIGN


@pytest.mark.gpu
def test_statistics_and_sums_that_nobody_wants_may_share_a_buffer():
    x, dy = (I.randn((300, 96), seed=i).to(bf).cuda() for i in (1, 2))
    y, mean, rstd = R.rib_layer_norm_fwd(x)
    bin_ = torch.empty(300, device="cuda")
    y2, _, _ = R.rib_layer_norm_fwd(x, mean=bin_, rstd=bin_)
    g = R.rib_layer_norm_bwd(x, dy, mean, rstd)
    h = R.rib_layer_norm_bwd(x, dy, mean, rstd, dgamma=bin_[:96], dbeta=bin_[:96])
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(g["dx"], h["dx"])


def test_a_feed_forward_workspace_for_a_few_more_rows_serves_fewer():
    """Up to eight rows h is fp32, above bf16: the sizes still do not fall from
    eight rows to nine (rows whose products run in one kernel need none)."""
    for C, hidden in ((192, 384), (1024, 2816), (512, 8)):
        sizes = [R.rib_gated_ffn_fwd_workspace(r, C, hidden) for r in range(1, 40)]
        assert sizes == sorted(sizes) and sizes[7] >= 8 * hidden * 2
    # what a call asks for is its own need
    assert ffn_fwd(rows=9, ws=FAKE, wsb=9 * 192 * 2 - 1) == _abi.RIB_ERR_WORKSPACE
    assert ffn_fwd(rows=9, ws=None) == _abi.RIB_ERR_WORKSPACE
