"""Plain fp64 CPU oracle of one pre-norm block around the RIB attention
(TEST INFRASTRUCTURE ONLY): layer norm, qkv projection, window attention with
or without the convolutional local attention gate, output projection and
residual, layer norm, gated feed-forward block and residual.

Pins (tests/test_block_oracle.py): the backward against central differences of
the forward in every input and weight.
"""
from __future__ import annotations

from typing import Dict

import numpy as np

from . import layer_oracle as L
from .cla_oracle import _f64, cla_apply, cla_backward, cla_gate
from .rib_oracle import attn_bwd, attn_fwd

__all__ = ["block_fwd", "block_bwd"]


def _forward(x, w: Dict, heads, M, s, qp, kp, eps, act):
    x = _f64(x)
    B, H, W, C = x.shape
    rows = x.reshape(-1, C)
    t = {"x": rows}
    t["n1"], t["mean1"], t["rstd1"] = L.layer_norm_fwd(rows, w["norm1_gamma"], w["norm1_beta"], eps)
    qkv = L.linear_fwd(t["n1"], w["w_qkv"], w["b_qkv"])[0].reshape(B, H, W, 3, heads, C // heads)
    t["qkv"] = qkv
    t["attn"] = attn_fwd(qkv, M, s, qp, kp)[0]
    out = t["attn"]
    if w.get("cla") is not None:
        out = cla_apply(out, cla_gate(t["n1"].reshape(B, H, W, C), *w["cla"]))
    t["gated"] = out.reshape(-1, C)
    t["x1"] = L.linear_fwd(t["gated"], w["w_proj"], w["b_proj"], residual=rows)[0]
    t["n2"], t["mean2"], t["rstd2"] = L.layer_norm_fwd(t["x1"], w["norm2_gamma"], w["norm2_beta"],
                                                       eps)
    y = L.gated_ffn_fwd(t["n2"], w["w_in"], w["b_in"], w["w_out"], w["b_out"], act,
                        residual=t["x1"])
    return y.reshape(x.shape), t


def block_fwd(x, w, heads, M, s, qp, kp, eps=1e-5, act="silu"):
    """y for x [B][H][W][C].  w: the weights by name (norm1_gamma, norm1_beta,
    w_qkv, b_qkv, w_proj, b_proj, norm2_gamma, norm2_beta, w_in, b_in, w_out,
    b_out, and cla = (w_dw, b_dw, w_pw, b_pw) or None)."""
    return _forward(x, w, heads, M, s, qp, kp, eps, act)[0]


def block_bwd(x, dy, w, heads, M, s, qp, kp, eps=1e-5, act="silu"):
    """Gradients by name: dx, the weights', dqp, dkp and cla_* with the gate."""
    _, t = _forward(x, w, heads, M, s, qp, kp, eps, act)
    shape = _f64(x).shape
    C = shape[-1]
    dy = _f64(dy).reshape(-1, C)
    g = {}
    dn2, g["w_in"], g["b_in"], g["w_out"], g["b_out"] = L.gated_ffn_bwd(
        t["n2"], w["w_in"], w["b_in"], w["w_out"], dy, act)
    dx1, g["norm2_gamma"], g["norm2_beta"] = L.layer_norm_bwd(
        t["x1"], dn2, t["mean2"], t["rstd2"], w["norm2_gamma"], dres=dy)
    dout, g["w_proj"], g["b_proj"] = L.linear_bwd(t["gated"], w["w_proj"], dx1)
    dout, dn1 = dout.reshape(t["attn"].shape), None
    if w.get("cla") is not None:
        c = cla_backward(t["n1"].reshape(shape), *w["cla"], t["attn"], dout)
        dout, dn1 = c["d_o"].reshape(t["attn"].shape), c["dx"].reshape(-1, C)
        g.update({f"cla_{k}": c[k] for k in ("dw_dw", "db_dw", "dw_pw", "db_pw")})
    dqkv, g["dqp"], g["dkp"] = attn_bwd(t["qkv"], dout, M, s, qp, kp)
    dn1, g["w_qkv"], g["b_qkv"] = L.linear_bwd(t["n1"], w["w_qkv"], dqkv.reshape(-1, 3 * C),
                                               dx_add=dn1)
    dx, g["norm1_gamma"], g["norm1_beta"] = L.layer_norm_bwd(
        t["x"], dn1, t["mean1"], t["rstd1"], w["norm1_gamma"], dres=dx1)
    g["dx"] = dx.reshape(shape)
    return g
