"""A whole block -- norm, qkv projection, window attention (gated or not), output
projection and residual, norm, gated feed-forward and residual -- forward and
backward through schedule.RIBBlock, against the fp64 oracle of the block.

Bounds: the forward stores eight tensors in bf16 on its way to y (n1, qkv, the
softmax's weights, attention, its gated form, x1, n2, h) and rounds y; a
gradient passes at most eight more (dg and du, the norms' and projections'
inputs, the attention's two, its own).  Each rounding is at most H = 2^-8 of the
value.  With weights of unit gain (rows of variance 1 / fan-in, norms about one)
none grows on its way, so the 2-norm error stays below the number of roundings
times H even if all of them lay the same way: 9 H for y, 17 H for gradients.
"""
import numpy as np
import pytest
import torch

import oracle as O
import rib_inputs as I
import windowed_attention_implicit_b200 as R
from oracle.block_oracle import block_bwd, block_fwd
from tests.rib_testlib import bf16_round
from windowed_attention_implicit_b200.parallel import FlatGrads
from windowed_attention_implicit_b200.schedule import BlockWeights, LayerSpec, RIBBlock

pytestmark = pytest.mark.gpu

H = 2.0 ** -8
RANK, FREQ, MLP_HIDDEN = 16, 4, 16
# batch, height, width, heads, window, shift, hidden, gate: the feed-forward's
# one-kernel form (hidden 64, 4 row tiles), its two products, a ragged width
CASES = [(1, 32, 32, 2, 16, 8, 64, False), (2, 16, 32, 3, 16, 0, 200, True),
         (1, 16, 48, 4, 16, 8, 256, True), (1, 16, 16, 1, 16, 0, 32, False)]


def _params(heads, hidden, cla, seed=5):
    C = 32 * heads
    r = lambda i, *s, std=1.0: I.randn(s, seed=seed + i, std=std)
    bf = lambda t: t.to(torch.bfloat16).float()
    w = dict(norm1_gamma=1 + r(1, C, std=0.2), norm1_beta=r(2, C, std=0.2),
             w_qkv=bf(r(3, 3 * C, C, std=C ** -0.5)), b_qkv=r(4, 3 * C, std=0.2),
             w_proj=bf(r(5, C, C, std=C ** -0.5)), b_proj=r(6, C, std=0.2),
             norm2_gamma=1 + r(7, C, std=0.2), norm2_beta=r(8, C, std=0.2),
             w_in=bf(r(9, 2, hidden, C, std=C ** -0.5)), b_in=r(10, 2, hidden, std=0.2),
             w_out=bf(r(11, C, hidden, std=hidden ** -0.5)), b_out=r(12, C, std=0.2), cla=None)
    if cla:
        c = I.make_cla(C, seed)
        w["cla"] = tuple(c[k] if isinstance(c, dict) else getattr(c, k)
                         for k in ("w_dw", "b_dw", "w_pw", "b_pw"))
    return w


def _block(w, heads, window, shift, act="silu"):
    freqs = I.default_freqs(FREQ)
    mq = I.make_mlp(FREQ, MLP_HIDDEN, heads, RANK, 5, 0, strong=True)
    mk = I.make_mlp(FREQ, MLP_HIDDEN, heads, RANK, 5, 1, strong=True)
    mlp = R.PositionMLP.from_params(freqs, mq, mk, heads, RANK)
    d = {n: t.cuda() for n, t in w.items() if n != "cla"}
    ffn = R.GatedFfn.from_params(d.pop("w_in"), d.pop("b_in"), d.pop("w_out"), d.pop("b_out"))
    for n in ("w_qkv", "w_proj"):
        d[n] = d[n].to(torch.bfloat16)
    cla = None if w["cla"] is None else R.ClaGate.from_params(*w["cla"])
    block = RIBBlock(LayerSpec(window, shift, mlp), BlockWeights(**d, ffn=ffn, cla=cla), act=act)
    qp, kp = (bf16_round(t) for t in O.pos_tokens(freqs, mq, mk, window, heads, RANK))
    return block, qp, kp


def _done():
    torch.cuda.synchronize()
    code, site = R.rib_last_status()
    assert code == 0, f"{R.rib_status_string(code)} at site {site}"


def _rel(got, ref):
    got = got.detach().double().cpu().numpy().reshape(ref.shape)
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def _setup(case, act="silu"):
    B, Hh, W, heads, M, s, hidden, cla = case
    w = _params(heads, hidden, cla)
    block, qp, kp = _block(w, heads, M, s, act)
    x, dy = (I.randn((B, Hh, W, 32 * heads), seed=i, dtype=torch.bfloat16) for i in (31, 32))
    return w, block, (heads, M, s, qp, kp), x, dy


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("case", CASES)
def test_block_forward_and_backward(case, act):
    w, block, geo, x, dy = _setup(case, act)
    y, state = block.forward(x.cuda())
    g = block.backward(state, dy.cuda())
    _done()
    assert _rel(y, block_fwd(x, w, *geo, act=act)) <= 9 * H
    ref = block_bwd(x, dy, w, *geo, act=act)
    for name, r in ref.items():
        got = g["cla"][name[4:]] if name.startswith("cla_") else g[name]
        assert _rel(got, r) <= 17 * H, (name, _rel(got, r))
    assert (g["cla"] is None) == (w["cla"] is None)


def test_block_gradients_into_a_flat_buffer():
    w, block, geo, x, dy = _setup(CASES[1])
    _, state = block.forward(x.cuda())
    ref = block.backward(state, dy.cuda(), mlp_grads=False)
    flat = FlatGrads.for_block(block.weights)
    flat.flat.fill_(7.0)
    got = block.backward(state, dy.cuda(), mlp_grads=False, grads=flat.named())
    _done()
    for n, t in flat.named().items():
        assert got[n].data_ptr() == t.data_ptr() and torch.equal(t, ref[n]), n
    with pytest.raises(ValueError):
        block.backward(state, dy.cuda(), grads={"w_q": flat.flat})


def test_block_step_captured_and_replayed():
    w, block, geo, x, dy = _setup(CASES[2])
    x, dy = x.cuda(), dy.cuda()
    y, state = block.forward(x)
    ref = block.backward(state, dy)
    _done()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2 = block.forward(x)
        g2 = block.backward(s2, dy)
    names = [n for n in ref if isinstance(ref[n], torch.Tensor)]
    for _ in range(2):
        y2.fill_(3.0)
        for n in names:
            g2[n].fill_(3.0)
        graph.replay()
        _done()
        assert torch.equal(y, y2)
        for n in names:
            assert torch.equal(ref[n], g2[n]), n


def test_two_blocks_share_one_token_cache():
    """Two blocks in a row share one token cache; their result is the second
    block's on the first's output."""
    w, block, geo, x, _ = _setup(CASES[0])
    second = RIBBlock(block.spec, block.weights, cache=block.cache)
    mid, _ = block.forward(x.cuda())
    out, _ = second.forward(mid)
    _done()
    assert len(block.cache) == 1
    assert _rel(out, block_fwd(mid.cpu(), w, *geo)) <= 9 * H
