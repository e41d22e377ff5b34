"""Plain fp64 CPU oracle of the layer's other operators: layer norm, linear
projections with an epilogue and the gated feed-forward block, forward and
backward (TEST INFRASTRUCTURE ONLY; the CUDA library never uses it).

Feature maps are [rows][channels].  Every function takes anything numpy or
torch can hold and computes in fp64 with nothing rounded.

Pins (tests/test_layer_oracle.py): the forwards against torch's fp64
routines, the backwards against torch autograd and central differences.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

from .cla_oracle import _f64

__all__ = ["act_value", "act_slope", "layer_norm_fwd", "layer_norm_bwd", "linear_fwd",
           "linear_bwd", "gated_ffn_fwd", "gated_ffn_bwd"]


def _phi(z):
    return 0.5 * erfc(-z / np.sqrt(2.0))


def _logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act_value(z, act):
    z = _f64(z)
    if act == "gelu":
        return z * _phi(z)
    return z * _logistic(z) if act == "silu" else z


def act_slope(z, act):
    z = _f64(z)
    if act == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if act == "silu":
        s = _logistic(z)
        return s * (1.0 + z * _logistic(-z))
    return np.ones_like(z)


def layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd)."""
    x = _f64(x)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * _f64(gamma)
    if beta is not None:
        y = y + _f64(beta)
    return y, mean, rstd


def layer_norm_bwd(x, dy, mean, rstd, gamma=None, dres=None):
    """(dx, dgamma, dbeta) for the statistics given."""
    x, dy, r = _f64(x), _f64(dy), _f64(rstd)[:, None]
    xh = (x - _f64(mean)[:, None]) * r
    g = dy if gamma is None else dy * _f64(gamma)
    dx = r * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + _f64(dres)
    return dx, (dy * xh).sum(0), dy.sum(0)


def linear_fwd(x, w, bias=None, act="none", residual=None):
    """(y, z): y = act(z) + residual, z = x w^T + bias."""
    z = _f64(x) @ _f64(w).T
    if bias is not None:
        z = z + _f64(bias)
    y = act_value(z, act)
    return (y if residual is None else y + _f64(residual)), z


def linear_bwd(x, w, dy, act="none", pre=None, dx_add=None):
    """(dx, dw, db)."""
    dz = _f64(dy)
    if act != "none":
        dz = dz * act_slope(pre, act)
    dx = dz @ _f64(w)
    if dx_add is not None:
        dx = dx + _f64(dx_add)
    return dx, dz.T @ _f64(x), dz.sum(0)


def _gate_up(x, w_in, b_in):
    x, w = _f64(x), _f64(w_in)
    g, u = x @ w[0].T, x @ w[1].T
    if b_in is not None:
        b = _f64(b_in)
        g, u = g + b[0], u + b[1]
    return g, u


def gated_ffn_fwd(x, w_in, b_in, w_out, b_out, act="silu", residual=None):
    g, u = _gate_up(x, w_in, b_in)
    y = (act_value(g, act) * u) @ _f64(w_out).T
    if b_out is not None:
        y = y + _f64(b_out)
    return y if residual is None else y + _f64(residual)


def gated_ffn_bwd(x, w_in, b_in, w_out, dy, act="silu", dx_add=None):
    """(dx, dw_in, db_in, dw_out, db_out)."""
    g, u = _gate_up(x, w_in, b_in)
    x, w, dy = _f64(x), _f64(w_in), _f64(dy)
    a = act_value(g, act)
    dh = dy @ _f64(w_out)
    dg, du = dh * u * act_slope(g, act), dh * a
    dx = dg @ w[0] + du @ w[1]
    if dx_add is not None:
        dx = dx + _f64(dx_add)
    return (dx, np.stack([dg.T @ x, du.T @ x]), np.stack([dg.sum(0), du.sum(0)]), dy.T @ (a * u),
            dy.sum(0))
