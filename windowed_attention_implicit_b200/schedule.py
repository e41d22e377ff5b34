"""Host-level sequences of RIB attention layers and of whole blocks around them.

"Rank-Factorized Implicit Neural Bias" (gist.science English summary,
Technical Summary §2.C): the window size cycles within a block (e.g.
16 -> 32 -> 64), and the positional tokens depend only on the window geometry
(Chinese summary §2.A), so one Qp/Kp set per (MLP, window size) serves every
window, batch entry and layer that shares it.  This module runs such layer
sequences through the library's entry points with a geometry cache; it adds
no arithmetic of its own.

RIBBlock is one pre-norm block of such a network, forward and backward: layer
norm, qkv projection, window attention (with or without the convolutional
local attention gate), output projection with its residual, layer norm and the
gated feed-forward block with its residual.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import torch

from . import (ClaGate, GatedFfn, PositionMLP, PositionMLPGrad, PosTokenCache, rib_cla_bwd,
               rib_cla_gate, rib_gated_ffn_bwd, rib_gated_ffn_fwd, rib_layer_norm_bwd,
               rib_layer_norm_fwd, rib_linear_bwd, rib_linear_fwd, rib_window_attn_bwd,
               rib_window_attn_fwd, rib_window_attn_fwd_cla)


@dataclass
class LayerSpec:
    window: int
    shift: int
    mlp: PositionMLP


@dataclass
class LayerState:
    out: torch.Tensor
    lse: torch.Tensor


class RIBLayerStack:
    """A sequence of RIB window-attention layers (a cyclic window schedule, or
    a stack of layers that alternate the shift) sharing one position-token
    cache."""

    def __init__(self, layers: Sequence[LayerSpec], cache: Optional[PosTokenCache] = None):
        self.layers = list(layers)
        self.cache = cache if cache is not None else PosTokenCache()

    def tokens(self, i: int):
        spec = self.layers[i]
        _, _, qp16, kp16 = self.cache.get(spec.mlp, spec.window)
        return qp16, kp16

    def forward(self, qkvs: Sequence[torch.Tensor]) -> List[LayerState]:
        """qkvs[i]: bf16 [B][H][W][3][heads][32] input of layer i."""
        states = []
        for i, (spec, qkv) in enumerate(zip(self.layers, qkvs)):
            qp16, kp16 = self.tokens(i)
            out, lse = rib_window_attn_fwd(qkv, spec.window, spec.shift, qp16, kp16,
                                           rank=spec.mlp.rank)
            states.append(LayerState(out, lse))
        return states

    def backward(self, qkvs: Sequence[torch.Tensor], states: Sequence[LayerState],
                 douts: Sequence[torch.Tensor], mlp_grads: bool = True):
        """Per-layer gradients (dqkv, dqp, dkp and, if requested, the MLP
        weight gradients) for upstream gradients douts[i]."""
        grads = []
        for i, (spec, qkv, st, dout) in enumerate(zip(self.layers, qkvs, states, douts)):
            qp16, kp16 = self.tokens(i)
            grads.append(rib_window_attn_bwd(qkv, st.out, dout, st.lse, spec.window, spec.shift,
                                             qp16, kp16, rank=spec.mlp.rank,
                                             mlp=spec.mlp if mlp_grads else None))
        return grads


@dataclass
class BlockWeights:
    """Device weights of a block over C channels: layer norms fp32 [C];
    projections bf16 [out][in] with fp32 biases or None: w_qkv [3 C][C] (its
    output read as [3][heads][head_dim]), w_proj [C][C]; the feed-forward block
    and, optionally, the gate on the attention's output."""
    norm1_gamma: torch.Tensor
    norm1_beta: torch.Tensor
    w_qkv: torch.Tensor
    b_qkv: Optional[torch.Tensor]
    w_proj: torch.Tensor
    b_proj: Optional[torch.Tensor]
    norm2_gamma: torch.Tensor
    norm2_beta: torch.Tensor
    ffn: GatedFfn
    cla: Optional[ClaGate] = None

    def grad_shapes(self) -> Dict[str, tuple]:
        """Shapes of the weights' gradients, under RIBBlock.backward's names
        (without the gate's and the position MLP's)."""
        named = {n: getattr(self, n) for n in (
            "norm1_gamma", "norm1_beta", "w_qkv", "b_qkv", "w_proj", "b_proj", "norm2_gamma",
            "norm2_beta")}
        named.update({n: getattr(self.ffn, n) for n in ("w_in", "b_in", "w_out", "b_out")})
        return {n: tuple(t.shape) for n, t in named.items() if t is not None}


@dataclass
class BlockState:
    """What a block's forward keeps for its backward."""
    x: torch.Tensor
    n1: torch.Tensor
    mean1: torch.Tensor
    rstd1: torch.Tensor
    qkv: torch.Tensor
    gate: Optional[torch.Tensor]
    attn: torch.Tensor              # attention output before the gate
    gated: torch.Tensor             # what the output projection reads
    lse: torch.Tensor
    x1: torch.Tensor                # x + output projection
    n2: torch.Tensor
    mean2: torch.Tensor
    rstd2: torch.Tensor


class RIBBlock:
    """x1 = x + proj(attn(qkv(norm1(x)))),  y = x1 + ffn(norm2(x1)), for x bf16
    [B][H][W][C].  With weights.cla the attention's output is multiplied by the
    gate of norm1(x).  The feature map never leaves its raster layout: the
    projections and norms take its pixels as rows."""

    def __init__(self, spec: LayerSpec, weights: BlockWeights,
                 cache: Optional[PosTokenCache] = None, eps: float = 1e-5, act: str = "silu"):
        self.spec, self.weights, self.eps, self.act = spec, weights, eps, act
        self.cache = cache if cache is not None else PosTokenCache()

    def forward(self, x: torch.Tensor):
        """(y, BlockState)."""
        w, spec = self.weights, self.spec
        B, H, W, C = x.shape
        heads = spec.mlp.heads
        if C % heads:
            raise ValueError(f"{C} channels do not split into {heads} heads")
        _, _, qp16, kp16 = self.cache.get(spec.mlp, spec.window)
        n1, mean1, rstd1 = rib_layer_norm_fwd(x, w.norm1_gamma, w.norm1_beta, self.eps)
        qkv = rib_linear_fwd(n1, w.w_qkv, w.b_qkv)[0]
        qkv = qkv.view(B, H, W, 3, heads, C // heads)
        if w.cla is None:
            gate = None
            attn, lse = rib_window_attn_fwd(qkv, spec.window, spec.shift, qp16, kp16,
                                            rank=spec.mlp.rank)
            gated = attn
        else:
            gate = rib_cla_gate(n1, w.cla)
            attn, gated, lse = rib_window_attn_fwd_cla(qkv, spec.window, spec.shift, gate, qp16,
                                                       kp16, rank=spec.mlp.rank)
        x1 = rib_linear_fwd(gated.view(B, H, W, C), w.w_proj, w.b_proj, residual=x)[0]
        n2, mean2, rstd2 = rib_layer_norm_fwd(x1, w.norm2_gamma, w.norm2_beta, self.eps)
        y = rib_gated_ffn_fwd(n2, w.ffn, self.act, residual=x1)
        return y, BlockState(x, n1, mean1, rstd1, qkv, gate, attn, gated, lse, x1, n2, mean2, rstd2)

    def backward(self, state: BlockState, dy: torch.Tensor, mlp_grads: bool = True,
                 grads: Optional[Dict[str, torch.Tensor]] = None,
                 dw_dtype: torch.dtype = torch.float32) -> dict:
        """Gradients for dy: dx, every weight's under its name in BlockWeights,
        dqp, dkp, dmlp (if mlp_grads) and cla (a dict, with the gate).  grads:
        buffers for weight gradients, by name (those of a FlatGrads, say);
        the others are allocated, the projections' in dw_dtype."""
        w, spec, s, o = self.weights, self.spec, state, dict(grads or {})
        unknown = set(o) - set(w.grad_shapes())
        if unknown:
            raise ValueError(f"no such gradients: {sorted(unknown)}")
        B, H, W, C = s.x.shape
        f = rib_gated_ffn_bwd(s.n2, w.ffn, dy, self.act, dw_in=o.get("w_in"), db_in=o.get("b_in"),
                              dw_out=o.get("w_out"), db_out=o.get("b_out"), dw_dtype=dw_dtype)
        n2 = rib_layer_norm_bwd(s.x1, f["dx"], s.mean2, s.rstd2, w.norm2_gamma, dres=dy,
                                dgamma=o.get("norm2_gamma"), dbeta=o.get("norm2_beta"))
        dx1 = n2["dx"]
        p = rib_linear_bwd(s.gated.view(B, H, W, C), w.w_proj, dx1, with_db=w.b_proj is not None,
                           dw=o.get("w_proj"), db=o.get("b_proj"), dw_dtype=dw_dtype)
        _, _, qp16, kp16 = self.cache.get(spec.mlp, spec.window)
        dout, dn1, cla = p["dx"].view(s.attn.shape), None, None
        if w.cla is not None:
            cla = rib_cla_bwd(s.n1, w.cla, s.gate, s.attn, dout)
            dout, dn1 = cla.pop("dout"), cla.pop("dx")
        a = rib_window_attn_bwd(s.qkv, s.attn, dout, s.lse, spec.window, spec.shift, qp16, kp16,
                                rank=spec.mlp.rank, mlp=spec.mlp if mlp_grads else None)
        q = rib_linear_bwd(s.n1, w.w_qkv, a["dqkv"].view(B, H, W, 3 * C), dx_add=dn1,
                           with_db=w.b_qkv is not None, dw=o.get("w_qkv"), db=o.get("b_qkv"),
                           dw_dtype=dw_dtype)
        n1 = rib_layer_norm_bwd(s.x, q["dx"], s.mean1, s.rstd1, w.norm1_gamma, dres=dx1,
                                dgamma=o.get("norm1_gamma"), dbeta=o.get("norm1_beta"))
        return {"dx": n1["dx"], "norm1_gamma": n1["dgamma"], "norm1_beta": n1["dbeta"],
                "w_qkv": q["dw"], "b_qkv": q["db"], "w_proj": p["dw"], "b_proj": p["db"],
                "norm2_gamma": n2["dgamma"], "norm2_beta": n2["dbeta"], "w_in": f["dw_in"],
                "b_in": f["db_in"], "w_out": f["dw_out"], "b_out": f["db_out"],
                "dqp": a["dqp"], "dkp": a["dkp"], "dmlp": a["dmlp"], "cla": cla}
