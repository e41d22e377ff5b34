"""Layer norm, linear projections and the gated feed-forward block against the
fp64 oracle, elementwise, at the sizes and corners where they can go wrong.

Every comparison has a bound derived from the number formats, computed per
element in fp64 beside the reference:
  H = 2^-8    one rounding to bf16, relative to the value (half a step)
  U = 2^-24   one rounding to fp32; an accumulation of n products on the
              tensor cores adds at most (n / 16 + 24) sums that may truncate,
              2 U each, times the sum of the products' magnitudes
  the activations' errors as their formulas give them: gelu's value is
  max(z, 0) - |z| Q with Q to 0.081 (2^-12 Q + 1e-7) by the fit of its
  polynomial, and below 1e-9 beyond |z| = 6; its slope takes Q to 1.5e-7 / 2;
  silu's logistic and every exponential and reciprocal add a few ulps and the
  exponent's own rounding
Where at least 4096 elements were rounded, the 2-norm error has to be that of
independent roundings too: each has an rms of at most H / sqrt 3, so two of
them stay below H.
"""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
import rib_inputs as I
import windowed_attention_implicit_b200 as R
from windowed_attention_implicit_b200 import _abi

pytestmark = pytest.mark.gpu

H, U = 2.0 ** -8, 2.0 ** -24
bf, f32 = torch.bfloat16, torch.float32


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(shape, seed, std=1.0, dtype=bf):
    return I.randn(shape, seed=seed, std=std, dtype=f32).to(dtype)


def _done():
    torch.cuda.synchronize()
    code, site = R.rib_last_status()
    assert code == 0, f"{R.rib_status_string(code)} at site {site}"


def _within(got, ref, bound, what, rounded=None):
    got = _np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = np.abs(got - ref)
    worst = np.max(err / (bound + 1e-30))
    assert worst <= 1.0, f"{what}: {worst:.3f} of its bound, at {np.unravel_index(np.argmax(err / (bound + 1e-30)), err.shape)}"
    if rounded and ref.size >= 4096:
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= rounded, f"{what}: 2-norm error {rel:.2e}"
    return worst


def _mma(n):
    return (n / 16 + 24) * 2 * U


def _act_err(z, act):
    if act == "gelu":
        q = O.act_value(-np.abs(z), act) / -np.maximum(np.abs(z), 1e-30)
        return np.abs(z) * (1e-8 + (0.081 * 2.0 ** -12 + 1e-5) * q + 2 * U * (z >= 0))
    if act == "silu":
        return (np.abs(z) + 8) * 4 * U * np.abs(O.act_value(z, act))
    return 0 * z


def _slope_err(z, act):
    if act == "gelu":
        return 1e-6 + 0 * z
    if act == "silu":
        return (np.abs(z) + 8) * (1 + np.abs(z)) * 4 * U
    return 0 * z


# ------------------------------------------------------------------ layer norm

LN_SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (33, 96), (1000, 192), (7, 250), (9, 256), (65, 264),
             (17, 512), (10, 1000), (4, 1024), (3, 1032), (6, 1025), (5, 2048), (3, 2056), (2, 4096),
             (3, 4104), (2, 8192), (2, 8191), (20001, 8), (4099, 33),
             # single elements, a row to 8, 16 or 32 lanes
             (9, 3), (70, 10), (20003, 10), (37, 20), (41, 36), (65, 50), (12345, 63), (33, 68), (19, 100), (77, 125),
             (50, 130), (21, 390), (22, 601), (23, 767), (24, 770), (25, 903)]


def _ln_case(rows, C, dtype, seed=3):
    x = (_rand((rows, C), seed, 1.5, f32) + 2.0).to(dtype)
    return x, 1 + _rand((C,), seed + 1, 0.3, f32), _rand((C,), seed + 2, 0.3, f32)


def _ln_fwd_bounds(x, g, b, eps, half):
    x, g, b = _np(x), _np(g), _np(b)
    y, mean, rstd = O.layer_norm_fwd(x, g, b, eps)
    d = x - mean[:, None]
    em = 60 * U * np.abs(x).mean(1)
    ed = em[:, None] + 2 * U * (np.abs(x) + np.abs(mean)[:, None])
    ev = 2 * (np.abs(d) * ed).mean(1) + (ed ** 2).mean(1) + 70 * U * (d * d).mean(1)
    er = 0.5 * rstd ** 3 * ev + 8 * U * rstd
    xh = np.abs(d) * rstd[:, None]
    ey = np.abs(g) * (rstd[:, None] * ed + np.abs(d) * er[:, None]) + 6 * U * (np.abs(g) * xh + np.abs(b))
    return (y, mean, rstd), (ey + half * (np.abs(y) + ey), em + 2 * U * np.abs(mean), er)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layer_norm_forward(rows, C, dtype):
    x, g, b = _ln_case(rows, C, dtype)
    y, mean, rstd = R.rib_layer_norm_fwd(x.cuda(), g.cuda(), b.cuda())
    _done()
    ref, bound = _ln_fwd_bounds(x, g, b, 1e-5, H if dtype == bf else 2 * U)
    for got, r, e, n in zip((y, mean, rstd), ref, bound, ("y", "mean", "rstd")):
        _within(got, r, e, n)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layer_norm_backward(rows, C, dtype):
    x, g, _ = _ln_case(rows, C, dtype)
    dy, dres = _rand((rows, C), 11, dtype=dtype), _rand((rows, C), 12, dtype=dtype)
    _, mean, rstd = O.layer_norm_fwd(x)
    mean, rstd = torch.tensor(mean, dtype=f32), torch.tensor(rstd, dtype=f32)
    got = R.rib_layer_norm_bwd(x.cuda(), dy.cuda(), mean.cuda(), rstd.cuda(), g.cuda(),
                               dres=dres.cuda())
    _done()
    dx, dg, db = O.layer_norm_bwd(x, dy, mean, rstd, g, dres)
    X, D, G, A, mu, rs = _np(x), _np(dy), _np(g), _np(dres), _np(mean)[:, None], _np(rstd)[:, None]
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


def test_layer_norm_optional_arguments():
    x, g, b = (t.cuda() for t in _ln_case(37, 192, bf))
    dy = _rand((37, 192), 5).cuda()
    one, zero = torch.ones_like(g), torch.zeros_like(b)
    y, mean, rstd = R.rib_layer_norm_fwd(x)
    y1, _, _ = R.rib_layer_norm_fwd(x, one, zero)
    got = R.rib_layer_norm_bwd(x, dy, mean, rstd)
    want = R.rib_layer_norm_bwd(x, dy, mean, rstd, one, dres=torch.zeros_like(x))
    only_dx = R.rib_layer_norm_bwd(x, dy, mean, rstd, weight_grads=False)
    y3, _, _ = R.rib_layer_norm_fwd(x.view(37, 2, 96).clone())      # any leading axes
    inplace = x.clone()
    R.rib_layer_norm_fwd(inplace, g, b, y=inplace)
    y2, _, _ = R.rib_layer_norm_fwd(x, g, b)
    d = dy.clone()
    R.rib_layer_norm_bwd(x, d, mean, rstd, dx=d)
    _done()
    assert torch.equal(y, y1) and torch.equal(inplace, y2) and y3.shape == (37, 2, 96)
    assert all(torch.equal(got[k], want[k]) for k in got)
    assert torch.equal(only_dx["dx"], got["dx"]) and only_dx["dgamma"] is None
    assert torch.equal(d, got["dx"])


def test_layer_norm_rows_off_the_vector_alignment():
    """A contiguous view that begins off a 16-byte address takes the
    element-by-element kernels."""
    for dtype in (bf, f32):
        big = (_rand((65 * 96 + 1,), 3, 1.5, f32)).to(dtype).cuda()
        x = big[1:].view(65, 96)
        assert x.data_ptr() % 16 != 0
        g, b = (1 + _rand((96,), 4, 0.3, f32)), _rand((96,), 5, 0.3, f32)
        y, mean, rstd = R.rib_layer_norm_fwd(x, g.cuda(), b.cuda())
        got = R.rib_layer_norm_bwd(x, x, mean, rstd, g.cuda())
        same = R.rib_layer_norm_bwd(x.clone(), x.clone(), mean, rstd, g.cuda())
        _done()
        ref, bound = _ln_fwd_bounds(x, g, b, 1e-5, H if dtype == bf else 2 * U)
        _within(y, ref[0], bound[0], "y")
        tol = (2 * H if dtype == bf else 64 * U) * np.abs(_np(same["dx"])) + 1e-5
        assert (np.abs(_np(got["dx"]) - _np(same["dx"])) <= tol).all()


def test_layer_norm_large_offset_keeps_its_spread():
    """x = 4096 + noise in fp32: the deviations from the mean are formed before
    they are squared, so the variance keeps its digits."""
    x = 4096 + _rand((64, 192), 3, 1.0, f32)
    y, mean, rstd = R.rib_layer_norm_fwd(x.cuda())
    _done()
    ref, bound = _ln_fwd_bounds(x, torch.ones(192), torch.zeros(192), 1e-5, 2 * U)
    _within(y, ref[0], bound[0], "y")
    assert np.abs(_np(rstd) - ref[2]).max() <= 1e-3


@pytest.mark.parametrize("dtype,C", [(bf, 192), (f32, 333), (bf, 4096)])
def test_layer_norm_nan_and_inf_stay_in_their_row(dtype, C):
    x, g, b = _ln_case(9, C, dtype)
    clean, _, _ = R.rib_layer_norm_fwd(x.cuda(), g.cuda(), b.cuda())
    x[3, C // 2], x[6, 0] = float("nan"), float("inf")
    y, mean, rstd = R.rib_layer_norm_fwd(x.cuda(), g.cuda(), b.cuda())
    _done()
    rest = [0, 1, 2, 4, 5, 7, 8]
    assert torch.equal(y[rest], clean[rest])
    assert torch.isnan(y[3]).all() and torch.isnan(mean[3]) and not torch.isfinite(y[6]).any()


# ------------------------------------------------------------------ linear

LINEAR = [(1, 8, 8), (1, 192, 576), (2, 16, 24), (127, 96, 96), (128, 64, 64), (129, 72, 200),
          (257, 192, 576), (300, 520, 264), (1000, 1032, 40), (64, 8, 1032), (513, 264, 2056),
          (38401, 72, 72), (20000, 1032, 64), (40000, 16, 520),
          # few rows (without the tensor cores up to a size), part of a row tile,
          # weight gradients in tiles of 128, 192 and 256 rows
          (3, 96, 288), (4, 4096, 40), (5, 1024, 2048), (7, 256, 72), (8, 64, 4096), (6, 2048, 2056),
          (9, 192, 576), (33, 128, 256), (256, 64, 16), (5000, 192, 192), (4097, 256, 320)]


def _linear_case(rows, K, N, seed=21):
    return (_rand((rows, K), seed), _rand((N, K), seed + 1, K ** -0.5), _rand((N,), seed + 2, 0.5, f32),
            _rand((rows, N), seed + 3))


def _linear_fwd_bounds(x, w, b, act, res):
    y, z = O.linear_fwd(x, w, b, act, res)
    K = x.shape[1]
    s = np.abs(_np(x)) @ np.abs(_np(w)).T
    if b is not None:
        s = s + np.abs(_np(b))
    ez = _mma(K) * s
    e = _act_err(z, act) + 1.13 * ez + 2 * U * (np.abs(y) + (0 if res is None else np.abs(_np(res))))
    return (y, z), (e + H * (np.abs(y) + e), ez + H * (np.abs(z) + ez))


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("rows,K,N", LINEAR)
def test_linear_forward(rows, K, N, act):
    x, w, b, r = _linear_case(rows, K, N)
    y, pre = R.rib_linear_fwd(x.cuda(), w.cuda(), b.cuda(), act=act, residual=r.cuda(), save_pre=True)
    plain, none = R.rib_linear_fwd(x.cuda(), w.cuda(), act=act)
    _done()
    (ry, rz), (by, bz) = _linear_fwd_bounds(x, w, b, act, r)
    _within(y, ry, by, "y", H)
    _within(pre, rz, bz, "pre", H)
    (ry, _), (by, _) = _linear_fwd_bounds(x, w, None, act, None)
    _within(plain, ry, by, "y, nothing added", H)
    assert none is None


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("rows,K,N", LINEAR)
def test_linear_backward(rows, K, N, act):
    x, w, _, dy = _linear_case(rows, K, N)
    pre, add = _rand((rows, N), 31, 1.5), _rand((rows, K), 32)
    p = None if act == "none" else pre
    args = [t.cuda() for t in (x, w, dy)]
    pc = None if p is None else p.cuda()
    got = R.rib_linear_bwd(*args, act=act, pre=pc, dx_add=add.cuda())
    half = R.rib_linear_bwd(*args, act=act, pre=pc, dw_dtype=bf)
    _done()
    X, W, D, A = _np(x), np.abs(_np(w)), _np(dy), _np(add)
    slope = O.act_slope(_np(pre), act)
    dz = D * slope
    ez = np.abs(D) * _slope_err(_np(pre), act) + (0 if act == "none" else 2 * U * np.abs(dz))
    e16 = ez + (0 if act == "none" else H * (np.abs(dz) + ez))
    dx, dw, db = O.linear_bwd(x, w, dy, act, p, add)
    ex = e16 @ W + _mma(N) * (np.abs(dz) @ W + np.abs(A))
    _within(got["dx"], dx, ex + H * (np.abs(dx) + ex), "dx", H)
    ew = e16.T @ np.abs(X) + (_mma(rows) + 200 * U) * (np.abs(dz).T @ np.abs(X))
    _within(got["dw"], dw, ew, "dw", H if act != "none" else None)
    _within(half["dw"], dw, ew + H * (np.abs(dw) + ew), "dw in bf16", H)
    eb = ez.sum(0) + (2 * rows + 300) * U * np.abs(dz).sum(0)
    _within(got["db"], db, eb, "db")
    assert torch.equal(got["db"], half["db"]) and half["dw"].dtype == bf


def test_linear_backward_parts_agree_with_the_whole():
    x, w, _, dy = (t.cuda() for t in _linear_case(700, 96, 288))
    pre = _rand((700, 288), 31).cuda()
    for act, p in (("none", None), ("silu", pre)):
        whole = R.rib_linear_bwd(x, w, dy, act=act, pre=p)
        for part in ("dx", "dw", "db"):
            got = R.rib_linear_bwd(x, w, dy, act=act, pre=p, with_dx=part == "dx",
                                   with_dw=part == "dw", with_db=part == "db")
            _done()
            assert [k for k, v in got.items() if v is not None] == [part]
            if part == "db" and act == "none":   # summed without the tensor cores
                assert torch.allclose(got[part], whole[part], rtol=0, atol=1e-3)
            else:
                assert torch.equal(got[part], whole[part])


def test_linear_outputs_may_take_their_residuals_place():
    x, w, b, r = (t.cuda() for t in _linear_case(1000, 192, 192))
    y, _ = R.rib_linear_fwd(x, w, b, act="gelu", residual=r)
    g = R.rib_linear_bwd(x, w, r, dx_add=x)
    y2, d2 = r.clone(), x.clone()
    R.rib_linear_fwd(x, w, b, act="gelu", residual=y2, y=y2)
    R.rib_linear_bwd(x, w, r, dx_add=d2, dx=d2)
    _done()
    assert torch.equal(y, y2) and torch.equal(g["dx"], d2)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_over_their_whole_range(act):
    """z from -40 to 40 through an identity product, value and slope."""
    z = torch.linspace(-40, 40, 4096).to(bf).view(-1, 16)
    eye = torch.eye(16, dtype=bf)
    y, _ = R.rib_linear_fwd(z.cuda(), eye.cuda(), act=act)
    one = torch.ones_like(z)
    g = R.rib_linear_bwd(z.cuda(), eye.cuda(), one.cuda(), act=act, pre=z.cuda())
    _done()
    Z = _np(z)
    v, s = O.act_value(Z, act), O.act_slope(Z, act)
    # beside the relative half step, absolute floors: gelu's Q is good to
    # 1.5e-7 / 2 in absolute terms; below 2^-126 results flush to zero
    e = _act_err(Z, act) + 2.0 ** -126
    _within(y, v, e + H * (np.abs(v) + e), "value")
    e = _slope_err(Z, act) + 2.0 ** -126
    _within(g["dx"], s, e + 2 * H * (np.abs(s) + e), "slope")


def test_linear_non_finite_rows_stay_apart():
    x, w, b, r = _linear_case(300, 192, 96)
    clean, _ = R.rib_linear_fwd(x.cuda(), w.cuda(), b.cuda(), act="silu", residual=r.cuda())
    x[5, 7], x[200, 0] = float("nan"), float("inf")
    y, _ = R.rib_linear_fwd(x.cuda(), w.cuda(), b.cuda(), act="silu", residual=r.cuda())
    _done()
    rest = [i for i in range(300) if i not in (5, 200)]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[5]).all()


# ------------------------------------------------------------------ gated feed-forward

FFN = [(1, 8, 8), (5, 16, 24), (129, 96, 192), (130, 72, 200), (400, 264, 520), (300, 192, 384),
       (30000, 64, 64), (12000, 520, 72), (1, 192, 1032), (3, 64, 128), (8, 32, 64), (17, 64, 2816),
       # in one kernel: short and ragged row tiles, channels and hidden channels,
       # one to three tiles a CTA pair
       (257, 256, 8), (769, 200, 56), (2000, 72, 128), (2560, 136, 192), (19300, 40, 200),
       (40000, 256, 72), (25000, 16, 344)]


def _ffn_case(rows, C, Hd, seed=41):
    return (_rand((rows, C), seed), _rand((2, Hd, C), seed + 1, C ** -0.5), _rand((2, Hd), seed + 2, 0.3, f32),
            _rand((C, Hd), seed + 3, Hd ** -0.5), _rand((C,), seed + 4, 0.3, f32), _rand((rows, C), seed + 5))


def _ffn_dev(wi, bi, wo, bo):
    return R.GatedFfn.from_params(wi, bi, wo, bo)


def _ffn_inner(x, wi, bi, act):
    X, W = _np(x), _np(wi)
    b = np.zeros(W.shape[:2]) if bi is None else _np(bi)
    g, u = X @ W[0].T + b[0], X @ W[1].T + b[1]
    k = _mma(X.shape[1])
    eg = k * (np.abs(X) @ np.abs(W[0]).T + np.abs(b[0]))
    eu = k * (np.abs(X) @ np.abs(W[1]).T + np.abs(b[1]))
    a = O.act_value(g, act)
    ea = _act_err(g, act) + 1.13 * eg
    h = a * u
    eh = np.abs(u) * ea + np.abs(a) * eu + ea * eu + 2 * U * np.abs(h)
    return g, u, a, h, eg, eu, ea, eh + H * (np.abs(h) + eh)


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("rows,C,Hd", FFN)
def test_gated_ffn_forward(rows, C, Hd, act):
    x, wi, bi, wo, bo, r = _ffn_case(rows, C, Hd)
    y = R.rib_gated_ffn_fwd(x.cuda(), _ffn_dev(wi, bi, wo, bo), act=act, residual=r.cuda())
    bare = R.rib_gated_ffn_fwd(x.cuda(), _ffn_dev(wi, None, wo, None), act=act)
    _done()
    for got, b1, b2, res in ((y, bi, bo, r), (bare, None, None, None)):
        ref = O.gated_ffn_fwd(x, wi, b1, wo, b2, act, res)
        *_, h, _, _, _, eh = _ffn_inner(x, wi, b1, act)
        W = np.abs(_np(wo)).T
        extra = (0 if b2 is None else np.abs(_np(b2))) + (0 if res is None else np.abs(_np(res)))
        e = eh @ W + _mma(Hd) * (np.abs(h) @ W + extra)
        _within(got, ref, e + H * (np.abs(ref) + e), "y", H)


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("rows,C,Hd", FFN)
def test_gated_ffn_backward(rows, C, Hd, act):
    x, wi, bi, wo, bo, dy = _ffn_case(rows, C, Hd)
    add = _rand((rows, C), 51)
    ffn = _ffn_dev(wi, bi, wo, bo)
    got = R.rib_gated_ffn_bwd(x.cuda(), ffn, dy.cuda(), act=act, dx_add=add.cuda())
    half = R.rib_gated_ffn_bwd(x.cuda(), _ffn_dev(wi, None, wo, None), dy.cuda(), act=act, dw_dtype=bf)
    _done()
    assert half["db_in"] is None and half["db_out"] is None
    for out, b, extra, bias in ((got, bi, add, True), (half, None, None, False)):
        dx, dwi, dbi, dwo, dbo = O.gated_ffn_bwd(x, wi, b, wo, dy, act, extra)
        g, u, a, h, eg, eu, ea, eh16 = _ffn_inner(x, wi, b, act)
        X, D, W, Wo = np.abs(_np(x)), np.abs(_np(dy)), np.abs(_np(wi)), np.abs(_np(wo))
        dh = _np(dy) @ _np(wo)
        edh = _mma(C) * (D @ Wo)
        sl = O.act_slope(g, act)
        esl = _slope_err(g, act) + (0 if act == "none" else 0.8 * eg)
        dg, du = dh * u * sl, dh * a
        edg = 1.01 * (np.abs(u * sl) * edh + np.abs(dh) * (np.abs(sl) * eu + np.abs(u) * esl)) + 4 * U * np.abs(dg)
        edu = 1.01 * (np.abs(a) * edh + np.abs(dh) * ea) + 4 * U * np.abs(du)
        eg16, eu16 = edg + H * (np.abs(dg) + edg), edu + H * (np.abs(du) + edu)
        A = 0 if extra is None else np.abs(_np(extra))
        e = eg16 @ W[0] + eu16 @ W[1] + _mma(2 * Hd) * (np.abs(dg) @ W[0] + np.abs(du) @ W[1] + A)
        _within(out["dx"], dx, e + H * (np.abs(dx) + e), "dx", H)
        k = _mma(rows) + 200 * U
        ei = np.stack([eg16.T @ X + k * (np.abs(dg).T @ X), eu16.T @ X + k * (np.abs(du).T @ X)])
        eo = D.T @ eh16 + k * (D.T @ np.abs(h))
        if not bias:
            ei, eo = ei + H * (np.abs(dwi) + ei), eo + H * (np.abs(dwo) + eo)
        _within(out["dw_in"], dwi, ei, "dw_in", H)
        _within(out["dw_out"], dwo, eo, "dw_out", H)
        if bias:
            n = (rows + 300) * U
            _within(out["db_in"], dbi, np.stack([edg.sum(0) + n * np.abs(dg).sum(0),
                                                 edu.sum(0) + n * np.abs(du).sum(0)]), "db_in")
            _within(out["db_out"], dbo, (2 * rows + 300) * U * D.sum(0), "db_out")


@pytest.mark.parametrize("rows,C,Hd", [(6, 64, 96), (800, 96, 64), (300, 192, 384)])
def test_gated_ffn_non_finite_rows_stay_apart(rows, C, Hd):
    x, wi, bi, wo, bo, r = _ffn_case(rows, C, Hd)
    ffn = _ffn_dev(wi, bi, wo, bo)
    clean = R.rib_gated_ffn_fwd(x.cuda(), ffn, residual=r.cuda())
    x[2, 7], x[rows - 1, 0], r[1, 3] = float("nan"), float("inf"), float("inf")
    y = R.rib_gated_ffn_fwd(x.cuda(), ffn, residual=r.cuda())
    _done()
    rest = [i for i in range(rows) if i not in (1, 2, rows - 1)]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[2]).all()
    assert not torch.isfinite(y[rows - 1]).any() and torch.isinf(y[1, 3])
    cols = [c for c in range(C) if c != 3]
    assert torch.equal(y[1, cols], clean[1, cols])


@pytest.mark.parametrize("Hd", [192, 64])
def test_gated_ffn_outputs_may_take_their_residuals_place(Hd):
    x, wi, bi, wo, bo, r = _ffn_case(700 if Hd > 64 else 800, 96, Hd)
    ffn = _ffn_dev(wi, bi, wo, bo)
    x, r = x.cuda(), r.cuda()
    y = R.rib_gated_ffn_fwd(x, ffn, residual=r)
    g = R.rib_gated_ffn_bwd(x, ffn, r, dx_add=r)
    y2, d2 = r.clone(), r.clone()
    R.rib_gated_ffn_fwd(x, ffn, residual=y2, y=y2)
    R.rib_gated_ffn_bwd(x, ffn, r, dx_add=d2, dx=d2)
    _done()
    assert torch.equal(y, y2) and torch.equal(g["dx"], d2)


# ------------------------------------------------------------------ all of them

def _calls(rows=600, C=96, Hd=200, seed=61):
    """name -> (function of outputs' buffers, the outputs' shapes and types)."""
    x, dy = _rand((rows, C), seed).cuda(), _rand((rows, C), seed + 1).cuda()
    g = (1 + _rand((C,), seed + 2, 0.2, f32)).cuda()
    w, b = _rand((Hd, C), seed + 3, C ** -0.5).cuda(), _rand((Hd,), seed + 4, 0.2, f32).cuda()
    dw_, pre = _rand((rows, Hd), seed + 5).cuda(), _rand((rows, Hd), seed + 6).cuda()
    _, wi, bi, wo, bo, _ = _ffn_case(1, C, Hd, seed + 7)
    ffn = _ffn_dev(wi, bi, wo, bo)
    _, wi, bi, wo, bo, _ = _ffn_case(1, C, 64, seed + 8)
    thin = _ffn_dev(wi, bi, wo, bo)
    _, mean, rstd = R.rib_layer_norm_fwd(x)
    rc, rh, cc, hh = ((rows, C), bf), ((rows, Hd), bf), ((C,), f32), ((Hd,), f32)
    return {
        "norm_fwd": (lambda o, **k: R.rib_layer_norm_fwd(x, g, g, y=o[0], mean=o[1], rstd=o[2], **k),
                     [rc, ((rows,), f32), ((rows,), f32)]),
        "norm_bwd": (lambda o, **k: R.rib_layer_norm_bwd(x, dy, mean, rstd, g, dres=dy, dx=o[0], dgamma=o[1],
                                                         dbeta=o[2], **k), [rc, cc, cc]),
        "linear_fwd": (lambda o, **k: R.rib_linear_fwd(x, w, b, act="gelu", residual=dw_, y=o[0], pre=o[1], **k),
                       [rh, rh]),
        "linear_bwd": (lambda o, **k: R.rib_linear_bwd(x, w, dw_, act="gelu", pre=pre, dx_add=dy, dx=o[0], dw=o[1],
                                                       db=o[2], **k), [rc, ((Hd, C), f32), hh]),
        "linear_bwd_plain": (lambda o, **k: R.rib_linear_bwd(x, w, dw_, dx=o[0], dw=o[1], db=o[2], **k),
                             [rc, ((Hd, C), f32), hh]),
        "ffn_fwd": (lambda o, **k: R.rib_gated_ffn_fwd(x, ffn, residual=dy, y=o[0], **k), [rc]),
        "ffn_fwd_one_kernel": (lambda o, **k: R.rib_gated_ffn_fwd(x, thin, residual=dy, y=o[0], **k), [rc]),
        "ffn_bwd": (lambda o, **k: R.rib_gated_ffn_bwd(x, ffn, dy, dx=o[0], dw_in=o[1], db_in=o[2], dw_out=o[3],
                                                       db_out=o[4], **k),
                    [rc, ((2, Hd, C), f32), ((2, Hd), f32), ((C, Hd), f32), cc]),
    }


NAMES = ["norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd", "linear_bwd_plain", "ffn_fwd",
         "ffn_fwd_one_kernel", "ffn_bwd"]


def _fresh(spec):
    return [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in spec]


@pytest.mark.parametrize("name", NAMES)
def test_nothing_is_written_behind_the_outputs(name):
    fn, spec = _calls()[name]
    pads, outs = [], []
    for s, t in spec:
        n = int(np.prod(s))
        buf = torch.full((n + 4096,), 7.0, dtype=t, device="cuda")
        pads.append(buf[n:])
        outs.append(buf[:n].view(s))
    fn(outs)
    _done()
    ref = _fresh(spec)
    fn(ref)
    _done()
    for p, o, r in zip(pads, outs, ref):
        assert (p == 7.0).all() and torch.equal(o, r)


@pytest.mark.parametrize("name", NAMES)
def test_repeated_captured_and_side_stream_calls_agree(name):
    fn, spec = _calls()[name]
    ref = _fresh(spec)
    fn(ref)
    _done()
    again = _fresh(spec)
    fn(again)
    # on another stream, its outputs and workspace allocated by the call
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = _fresh(spec)
    side.wait_stream(torch.cuda.current_stream())
    fn(third, stream=side)
    raw = _fresh(spec)
    side.wait_stream(torch.cuda.current_stream())
    fn(raw, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    _done()
    # captured and replayed twice
    cap = _fresh(spec)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(cap)
    for t in cap:
        t.fill_(3.0)
    graph.replay()
    graph.replay()
    _done()
    for r, *rest in zip(ref, again, third, raw, cap):
        for t in rest:
            assert torch.equal(r, t)


def test_two_calls_at_once_on_two_streams():
    calls = _calls(rows=3000)
    refs, outs = {}, {}
    for n, (fn, spec) in calls.items():
        refs[n], outs[n] = _fresh(spec), _fresh(spec)
        fn(refs[n])
    _done()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, (n, (fn, _)) in enumerate(calls.items()):
        fn(outs[n], stream=streams[i % 2])
    _done()
    for n in calls:
        assert all(torch.equal(a, b) for a, b in zip(refs[n], outs[n])), n


def test_no_rows():
    C, Hd = 96, 200
    x, g = torch.empty((0, C), dtype=bf, device="cuda"), torch.ones(C, device="cuda")
    w = _rand((Hd, C), 1).cuda()
    dy = torch.empty((0, Hd), dtype=bf, device="cuda")
    _, wi, bi, wo, bo, _ = _ffn_case(1, C, Hd)
    ffn = _ffn_dev(wi, bi, wo, bo)
    y, mean, rstd = R.rib_layer_norm_fwd(x, g)
    n = R.rib_layer_norm_bwd(x, x, mean, rstd, g)
    z, _ = R.rib_linear_fwd(x, w)
    grads = [n["dgamma"], n["dbeta"]]
    for dt in (bf, f32):
        b = R.rib_linear_bwd(x, w, dy, dw=torch.full((Hd, C), 7.0, dtype=dt, device="cuda"))
        f = R.rib_gated_ffn_bwd(x, ffn, x, dw_dtype=dt, dw_in=torch.full((2, Hd, C), 7.0, dtype=dt, device="cuda"))
        grads += [b["dw"], b["db"], f["dw_in"], f["db_in"], f["dw_out"], f["db_out"]]
    _done()
    assert y.shape == (0, C) and z.shape == (0, Hd) and R.rib_gated_ffn_fwd(x, ffn).shape == (0, C)
    assert all((t == 0).all() for t in grads)


def test_offsets_beyond_31_bits():
    """More than 2^31 elements: the last rows come out as they do alone."""
    rows, C = (1 << 31) // 1024 + 130, 1024
    x = torch.zeros((rows, C), dtype=bf, device="cuda")
    tail = _rand((200, C), 71).cuda()
    x[-200:] = tail
    g = (1 + _rand((C,), 72, 0.2, f32)).cuda()
    y, mean, rstd = R.rib_layer_norm_fwd(x, g)
    want, m1, r1 = R.rib_layer_norm_fwd(tail, g)
    _done()
    assert torch.equal(y[-200:], want) and torch.equal(mean[-200:], m1)
    w = _rand((C, 64), 73, 0.1).cuda()
    xs = torch.zeros((rows, 64), dtype=bf, device="cuda")
    xs[-200:] = tail[:, :64]
    R.rib_linear_fwd(xs, w, act="silu", residual=x, y=y)
    alone, _ = R.rib_linear_fwd(tail[:, :64].contiguous(), w, act="silu", residual=tail)
    _done()
    assert torch.equal(y[-200:], alone)
    d = R.rib_linear_bwd(xs, w, x, dw_dtype=bf)
    small = R.rib_linear_bwd(tail[:, :64].contiguous(), w, tail)
    _done()
    assert torch.equal(d["dx"][-200:], small["dx"])
    assert (_np(d["dw"]) - _np(small["dw"])).__abs__().max() <= 2 * H * np.abs(_np(small["dw"])).max()
