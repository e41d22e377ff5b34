"""CPU checks of the layer operators' entry points: bad arguments are refused
before anything is launched, through the C ABI and in the binding."""
import pytest
import torch

import windowed_attention_implicit_b200 as R
from windowed_attention_implicit_b200 import _abi

FAKE = 1 << 20        # aligned non-null stand-in; never dereferenced
ARG, UNS, ALIGN = _abi.RIB_ERR_ARG, _abi.RIB_ERR_UNSUPPORTED, _abi.RIB_ERR_ALIGN
bf, f32 = torch.bfloat16, torch.float32


def ln_fwd(**kw):
    a = dict(x=FAKE, dtype=0, rows=4, C=96, gamma=FAKE, beta=FAKE, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return R.library().rib_layer_norm_fwd(*a.values(), None)


def ln_bwd(**kw):
    a = dict(x=FAKE, dy=FAKE, dtype=0, rows=4, C=96, mean=FAKE, rstd=FAKE, gamma=FAKE, dres=FAKE, dx=FAKE,
             dgamma=FAKE, dbeta=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return R.library().rib_layer_norm_bwd(*a.values(), None)


def lin_fwd(**kw):
    a = dict(x=FAKE, rows=4, K=96, w=FAKE, N=64, bias=FAKE, act=0, residual=FAKE, pre=FAKE, y=FAKE)
    a.update(kw)
    return R.library().rib_linear_fwd(*a.values(), None)


def lin_bwd(**kw):
    a = dict(x=FAKE, rows=4, K=96, w=FAKE, N=64, act=1, pre=FAKE, dy=FAKE, dx_add=FAKE, dx=FAKE, dw=FAKE,
             dw_dtype=1, db=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return R.library().rib_linear_bwd(*a.values(), None)


def ffn_fwd(**kw):
    a = dict(x=FAKE, rows=4, C=96, hidden=192, w_in=FAKE, b_in=FAKE, w_out=FAKE, b_out=FAKE, act=2,
             residual=FAKE, y=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return R.library().rib_gated_ffn_fwd(*a.values(), None)


def ffn_bwd(**kw):
    a = dict(x=FAKE, rows=4, C=96, hidden=192, w_in=FAKE, b_in=FAKE, w_out=FAKE, act=2, dy=FAKE, dx_add=FAKE,
             dx=FAKE, dw_in=FAKE, db_in=FAKE, dw_out=FAKE, db_out=FAKE, dw_dtype=1, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return R.library().rib_gated_ffn_bwd(*a.values(), None)


BAD = [
    (ln_fwd, dict(dtype=2), ARG), (ln_fwd, dict(rows=-1), ARG), (ln_fwd, dict(C=0), ARG),
    (ln_fwd, dict(C=8193), UNS), (ln_fwd, dict(rows=(1 << 30) + 1), UNS), (ln_fwd, dict(eps=-1e-5), ARG),
    (ln_fwd, dict(eps=float("nan")), ARG), (ln_fwd, dict(x=None), ARG), (ln_fwd, dict(y=None), ARG),
    (ln_fwd, dict(x=FAKE + 1), ALIGN), (ln_fwd, dict(dtype=1, y=FAKE + 2), ALIGN),
    (ln_fwd, dict(gamma=FAKE + 2), ALIGN), (ln_fwd, dict(rstd=FAKE + 1), ALIGN),
    (ln_bwd, dict(dtype=-1), ARG), (ln_bwd, dict(C=-3), ARG), (ln_bwd, dict(C=9000), UNS),
    (ln_bwd, dict(dy=None), ARG), (ln_bwd, dict(mean=None), ARG), (ln_bwd, dict(rstd=None), ARG),
    (ln_bwd, dict(dx=None), ARG), (ln_bwd, dict(dres=FAKE + 1), ALIGN), (ln_bwd, dict(dgamma=FAKE + 2), ALIGN),
    (lin_fwd, dict(K=0), ARG), (lin_fwd, dict(N=-8), ARG), (lin_fwd, dict(rows=-1), ARG),
    (lin_fwd, dict(K=100), UNS), (lin_fwd, dict(N=36), UNS), (lin_fwd, dict(N=65544), UNS),
    (lin_fwd, dict(rows=(1 << 30) + 1), UNS), (lin_fwd, dict(act=3), ARG), (lin_fwd, dict(act=-1), ARG),
    (lin_fwd, dict(x=None), ARG), (lin_fwd, dict(w=None), ARG), (lin_fwd, dict(y=None), ARG),
    (lin_fwd, dict(w=FAKE + 8), ALIGN), (lin_fwd, dict(bias=FAKE + 4), ALIGN), (lin_fwd, dict(pre=FAKE + 8), ALIGN),
    (lin_bwd, dict(dw_dtype=2), ARG), (lin_bwd, dict(act=7), ARG), (lin_bwd, dict(K=12), UNS),
    (lin_bwd, dict(dy=None), ARG), (lin_bwd, dict(pre=None), ARG), (lin_bwd, dict(w=None), ARG),
    (lin_bwd, dict(x=None), ARG), (lin_bwd, dict(dx=FAKE + 8), ALIGN), (lin_bwd, dict(db=FAKE + 4), ALIGN),
    (ffn_fwd, dict(hidden=0), ARG), (ffn_fwd, dict(hidden=20), UNS), (ffn_fwd, dict(C=20), UNS),
    (ffn_fwd, dict(hidden=32776), UNS), (ffn_fwd, dict(act=9), ARG), (ffn_fwd, dict(w_out=None), ARG),
    (ffn_fwd, dict(b_in=FAKE + 4), ALIGN), (ffn_fwd, dict(ws=None), _abi.RIB_ERR_WORKSPACE),
    (ffn_fwd, dict(wsb=4 * 192 * 2 - 1), _abi.RIB_ERR_WORKSPACE), (ffn_fwd, dict(ws=FAKE + 16), ALIGN),
    (ffn_bwd, dict(dw_in=None), ARG), (ffn_bwd, dict(dw_out=None), ARG), (ffn_bwd, dict(dx=None), ARG),
    (ffn_bwd, dict(dw_dtype=5), ARG), (ffn_bwd, dict(rows=-2), ARG), (ffn_bwd, dict(hidden=12), UNS),
    (ffn_bwd, dict(dy=FAKE + 8), ALIGN), (ffn_bwd, dict(rows=0, dw_in=None), ARG),
]


@pytest.mark.parametrize("fn,kw,code", BAD, ids=[f"{f.__name__}-{k}" for f, k, _ in BAD])
def test_refusals(fn, kw, code):
    assert fn(**kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in pointers: only where nothing can be launched")
@pytest.mark.parametrize("fn,outs,clash", [
    (lin_fwd, ("residual", "pre", "y"), [("y", "x"), ("pre", "x"), ("pre", "y"), ("pre", "residual")]),
    (lin_bwd, ("dy", "dx_add", "dx"), [("dx", "x"), ("dx", "dy")]),
    (ffn_bwd, ("dy", "dx_add", "dx"), [("dx", "x"), ("dx", "dy")])])
def test_outputs_over_inputs_that_are_read_later_are_refused(fn, outs, clash):
    apart = {n: FAKE + ((i + 1) << 24) for i, n in enumerate(outs)}
    assert fn(**apart) not in (_abi.RIB_OK, ARG, ALIGN, UNS)    # only the missing device is left to refuse
    for out, other in clash:
        assert fn(**{**apart, out: apart.get(other, FAKE)}) == ARG
    last = {"y": "residual"} if "y" in outs else {"dx": "dx_add"}
    for out, other in last.items():                              # in place of these it may be
        assert fn(**{**apart, out: apart[other]}) not in (_abi.RIB_OK, ARG, ALIGN, UNS)


def test_no_rows_is_valid_and_reads_no_pointer():
    assert ln_fwd(rows=0, x=None, y=None) == _abi.RIB_OK
    assert lin_fwd(rows=0, x=None, w=None, y=None) == _abi.RIB_OK
    assert ffn_fwd(rows=0, x=None, y=None, ws=None) == _abi.RIB_OK
    assert lin_bwd(rows=0, dw=None, db=None, dy=None, ws=None) == _abi.RIB_OK
    assert ln_bwd(rows=0, dgamma=None, dbeta=None, x=None, ws=None) == _abi.RIB_OK


def test_workspace_sizes_of_bad_shapes_are_zero():
    assert R.rib_layer_norm_bwd_workspace(4, 9000) == 0
    assert R.rib_linear_bwd_workspace(4, 12, 16) == 0
    assert R.rib_gated_ffn_fwd_workspace(4, 16, 12) == 0
    assert R.rib_gated_ffn_bwd_workspace(-1, 16, 16) == 0
    assert R.rib_gated_ffn_fwd_workspace(5, 16, 24) >= 5 * 24 * 2


# ------------------------------------------------------------------ the binding

def _z(*shape, dtype=bf, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


def _passes(fn, *a, **kw):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn(*a, **kw)


def _rejects(fn, what, *a, code=ARG, **kw):
    with pytest.raises(R.RibError, match=what) as e:
        fn(*a, **kw)
    assert e.value.code == code


def test_layer_norm_buffers():
    x, g, m = _z(2, 3, 96), _z(96, dtype=f32), _z(2, 3, dtype=f32)
    f, b = R.rib_layer_norm_fwd, R.rib_layer_norm_bwd
    _passes(f, x, g, g, y=_z(2, 3, 96), mean=m, rstd=m)
    _passes(f, x)
    _rejects(f, "gamma holds", x, _z(95, dtype=f32))
    _rejects(f, "y holds", x, y=_z(2, 96))
    _rejects(f, "mean holds", x, mean=_z(2, dtype=f32))
    _rejects(f, "x is torch.float16", x.half(), code=UNS)
    _rejects(f, "channels", _z(4, 0))
    _rejects(f, "is on meta", x, y=_z(2, 3, 96, device="meta"))
    _passes(b, x, x, m, m, g, dres=x, dx=_z(2, 3, 96), dgamma=g, dbeta=g)
    _passes(b, x, x, m, m, weight_grads=False)
    _rejects(b, "dy holds", x, x[:1], m, m)
    _rejects(b, "rstd holds", x, x, m, m[:1])
    _rejects(b, "dres holds", x, x, m, m, dres=x[:1])
    _rejects(b, "dbeta holds", x, x, m, m, g, dbeta=_z(1, dtype=f32))


def test_linear_buffers():
    x, w, b, y = _z(2, 5, 96), _z(64, 96), _z(64, dtype=f32), _z(2, 5, 64)
    f, g = R.rib_linear_fwd, R.rib_linear_bwd
    _passes(f, x, w, b, act="gelu", residual=y, y=y, pre=y)
    _rejects(f, "act 'relu'", x, w, act="relu")
    _rejects(f, r"w must be \[out\]\[96\]", x, _z(64, 95))
    _rejects(f, r"w must be", x, _z(64 * 96))
    _rejects(f, "bias holds", x, w, _z(65, dtype=f32))
    _rejects(f, "residual holds", x, w, residual=y[:1])
    _rejects(f, "pre holds", x, w, pre=y[:1])
    _passes(g, x, w, y, act="silu", pre=y, dx_add=x, dx=x, dw=w, db=b)
    _passes(g, x, w, y)
    _rejects(g, "needs pre", x, w, y, act="gelu")
    _rejects(g, "dy holds", x, w, y[:1])
    _rejects(g, "dx_add holds", x, w, y, dx_add=x[:1])
    _rejects(g, "dw holds", x, w, y, dw=_z(64, 95))
    _rejects(g, "dw is torch.float64", x, w, y, dw_dtype=torch.float64, code=UNS)
    _rejects(g, "db holds", x, w, y, db=_z(1, dtype=f32))


def test_gated_ffn_buffers():
    C, H = 96, 200
    x = _z(2, 5, C)
    ffn = R.GatedFfn.from_params(_z(2, H, C), _z(2, H), _z(C, H), _z(C), device="cpu")
    assert ffn.hidden == H and ffn.b_in.dtype == f32 and ffn.w_in.dtype == bf
    f, g = R.rib_gated_ffn_fwd, R.rib_gated_ffn_bwd
    _passes(f, x, ffn, residual=x, y=_z(2, 5, C))
    _passes(f, x, R.GatedFfn(ffn.w_in, None, ffn.w_out, None), act="gelu")
    _rejects(f, "act 'tanh'", x, ffn, act="tanh")
    _rejects(f, "w_in must be", _z(2, 5, 88), ffn)
    _rejects(f, "w_out must be", x, R.GatedFfn(ffn.w_in, None, _z(H, C), None))
    _rejects(f, "b_in holds", x, R.GatedFfn(ffn.w_in, _z(H, dtype=f32), ffn.w_out, None))
    _rejects(f, "residual holds", x, ffn, residual=x[:1])
    _passes(g, x, ffn, x, dx_add=x, dx=x, dw_in=ffn.w_in, dw_out=ffn.w_out)
    _rejects(g, "dy holds", x, ffn, x[:1])
    _rejects(g, "dw_out holds", x, ffn, x, dw_out=_z(C, C))
    _rejects(g, "db_in holds", x, ffn, x, db_in=_z(H, dtype=f32))
    _rejects(g, "is torch.float16", x, ffn, x, dw_dtype=torch.float16, code=UNS)


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """The library launches on the current device: a call whose x is on
    another GPU stops before a pointer is handed over."""
    class Elsewhere:
        shape, device = torch.Size((4, 16)), torch.device("cuda", 1)
        dim = staticmethod(lambda: 2)
        numel = staticmethod(lambda: 64)
        get_device = staticmethod(lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(R.RibError, match="current device is cuda:0") as e:
        R._Call("rib_linear_fwd", Elsewhere(), None)
    assert e.value.code == ARG


def test_block_weight_gradients_share_one_buffer():
    from windowed_attention_implicit_b200.parallel import FlatGrads
    from windowed_attention_implicit_b200.schedule import BlockWeights
    C, Hd = 16, 24
    z = torch.zeros
    ffn = R.GatedFfn.from_params(z(2, Hd, C), z(2, Hd), z(C, Hd), None, device="cpu")
    w = BlockWeights(z(C), z(C), z(3 * C, C), None, z(C, C), z(C), z(C), z(C), ffn)
    g = FlatGrads.for_block(w).named()
    assert "b_qkv" not in g and "b_out" not in g and g["w_in"].shape == (2, Hd, C)
    assert sum(t.numel() for t in g.values()) == 3 * C * C + C * C + 5 * C + 2 * Hd * C + 2 * Hd + C * Hd
    base = g["norm1_gamma"].data_ptr()
    # at the 16-byte addresses that the projections' gradients need
    assert all((g[n].data_ptr() - base) % 16 == 0 for n in ("w_qkv", "w_proj", "w_in", "w_out", "b_in"))
