"""A whole block on maps of thousands of pixels, where its persistent kernels take
several tiles each, against the fp64 oracle: the checks and bounds of
test_gpu_block."""
import pytest
import torch

from oracle.block_oracle import block_bwd, block_fwd
from tests.test_gpu_block import H, _done, _rel, _setup

pytestmark = pytest.mark.gpu

# batch, height, width, heads, window, shift, hidden, gate
CASES = [(1, 128, 128, 3, 16, 8, 192, False), (2, 64, 96, 6, 16, 0, 384, True)]


@pytest.mark.parametrize("case", CASES)
def test_block_on_a_large_map(case):
    w, block, geo, x, dy = _setup(case)
    y, state = block.forward(x.cuda())
    g = block.backward(state, dy.cuda())
    _done()
    assert _rel(y, block_fwd(x, w, *geo, act="silu")) <= 9 * H
    for name, r in block_bwd(x, dy, w, *geo, act="silu").items():
        got = g["cla"][name[4:]] if name.startswith("cla_") else g[name]
        assert _rel(got, r) <= 17 * H, (name, _rel(got, r))


def test_block_on_a_large_map_on_another_stream_and_captured():
    w, block, geo, x, dy = _setup(CASES[0])
    x, dy = x.cuda(), dy.cuda()
    y, state = block.forward(x)
    ref = block.backward(state, dy)
    _done()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, s1 = block.forward(x)
        g1 = block.backward(s1, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2 = block.forward(x)
        g2 = block.backward(s2, dy)
    graph.replay()
    graph.replay()
    _done()
    assert torch.equal(y, y1) and torch.equal(y, y2)
    for n, t in ref.items():
        # the attention's own position gradients are sums of atomics
        if isinstance(t, torch.Tensor) and n not in ("dqp", "dkp"):
            assert torch.equal(t, g1[n]) and torch.equal(t, g2[n]), n
