"""The block's fp64 oracle: its backward against central differences of its
forward, in the input, the position tokens and every weight."""
import numpy as np
import pytest

from oracle.block_oracle import block_bwd, block_fwd

HEADS, M, RANK, C, HIDDEN = 2, 4, 3, 8, 5


def _weights(cla, seed=3):
    r = np.random.default_rng(seed)
    n = lambda *s, std=1.0: r.standard_normal(s) * std
    w = dict(norm1_gamma=1 + n(C, std=0.2), norm1_beta=n(C, std=0.2),
             w_qkv=n(3 * C, C, std=C ** -0.5), b_qkv=n(3 * C, std=0.2),
             w_proj=n(C, C, std=C ** -0.5), b_proj=n(C, std=0.2),
             norm2_gamma=1 + n(C, std=0.2), norm2_beta=n(C, std=0.2),
             w_in=n(2, HIDDEN, C, std=C ** -0.5), b_in=n(2, HIDDEN, std=0.2),
             w_out=n(C, HIDDEN, std=HIDDEN ** -0.5), b_out=n(C, std=0.2), cla=None)
    if cla:
        w["cla"] = (n(C, 3, 3, std=0.3), n(C, std=0.1), n(C, C, std=C ** -0.5), n(C, std=0.1))
    return w, n(1, 8, 4, C), n(1, 8, 4, C), n(HEADS, M, M, RANK), n(HEADS, M, M, RANK)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("cla", [False, True])
def test_block_gradients_are_those_of_central_differences(cla, act):
    w, x, dy, qp, kp = _weights(cla)
    geo = (HEADS, M, 2)
    g = block_bwd(x, dy, w, *geo, qp, kp, act=act)
    loss = lambda x, w, qp, kp: float((block_fwd(x, w, *geo, qp, kp, act=act) * dy).sum())
    r = np.random.default_rng(8)

    def slope(name, value, put):
        # along one random direction; the difference's own error is h^2 times a
        # third derivative (of order 1e2 at these sizes) plus 1e-15 |L| / h
        d, h = r.standard_normal(np.shape(value)), 1e-5
        num = (loss(*put(value + h * d)) - loss(*put(value - h * d))) / (2 * h)
        got = float((g[name] * d).sum())
        assert abs(num - got) <= 1e-6 * (1 + abs(got)), (name, num, got)

    slope("dx", x, lambda v: (v, w, qp, kp))
    slope("dqp", qp, lambda v: (x, w, v, kp))
    slope("dkp", kp, lambda v: (x, w, qp, v))
    for n, v in w.items():
        if n != "cla":
            slope(n, v, lambda u, n=n: (x, {**w, n: u}, qp, kp))
    if cla:
        for i, n in enumerate(("dw_dw", "db_dw", "dw_pw", "db_pw")):
            slope(f"cla_{n}", w["cla"][i], lambda u, i=i: (
                x, {**w, "cla": w["cla"][:i] + (u,) + w["cla"][i + 1:]}, qp, kp))
