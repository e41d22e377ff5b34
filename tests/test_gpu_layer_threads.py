"""Calls from host threads other than the one that set everything up, one at a
time and two at once."""
import sys
import threading

import pytest
import torch

import rib_inputs as I
import windowed_attention_implicit_b200 as R

pytestmark = pytest.mark.gpu

bf, f32 = torch.bfloat16, torch.float32
CALLS = 20000


def _rand(shape, seed, std=1.0, dtype=bf):
    return I.randn(shape, seed=seed, std=std).to(dtype).cuda()


def _p(t):
    return t.data_ptr()


def _norm(rows, C, seed):
    x, y = _rand((rows, C), seed), torch.empty((rows, C), dtype=bf, device="cuda")
    return R.library().rib_layer_norm_fwd, (_p(x), 0, rows, C, None, None, 1e-5, _p(y), None, None), [x, y], y


def _linear(rows, K, N, seed):
    x, w = _rand((rows, K), seed), _rand((N, K), seed + 1, K ** -0.5)
    y = torch.empty((rows, N), dtype=bf, device="cuda")
    return R.library().rib_linear_fwd, (_p(x), rows, K, _p(w), N, None, 0, None, None, _p(y)), [x, w, y], y


def _ffn(rows, C, H, seed):
    x = _rand((rows, C), seed)
    wi, wo = _rand((2, H, C), seed + 1, C ** -0.5), _rand((C, H), seed + 2, H ** -0.5)
    y = torch.empty((rows, C), dtype=bf, device="cuda")
    n = R.rib_gated_ffn_fwd_workspace(rows, C, H)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    return (R.library().rib_gated_ffn_fwd,
            (_p(x), rows, C, H, _p(wi), None, _p(wo), None, 2, None, _p(y), _p(ws) if n else None, n),
            [x, wi, wo, y, ws], y)


MAKERS = {"norm": (_norm, (20, 192)), "linear": (_linear, (100, 64, 64)), "few rows": (_linear, (2, 64, 64)),
          "feed-forward": (_ffn, (800, 64, 64)), "feed-forward, two products": (_ffn, (300, 264, 520))}


@pytest.mark.parametrize("name", MAKERS)
def test_first_cuda_work_of_a_thread(name):
    """A thread that has made no CUDA call has no current context yet."""
    make, shape = MAKERS[name]
    fn, args, _, y = make(*shape, seed=5)
    st = torch.cuda.current_stream().cuda_stream
    assert fn(*args, st) == 0
    want = y.clone()
    y.zero_()
    torch.cuda.synchronize()
    codes = []
    t = threading.Thread(target=lambda: codes.append(fn(*args, st)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [0] and torch.equal(y, want)


def test_first_cuda_work_of_a_thread_through_the_binding():
    x, w = _rand((100, 64), 1), _rand((64, 64), 2)
    qkv, y = _rand((1, 16, 16, 3, 2, 32), 4), torch.empty((100, 64), dtype=bf, device="cuda")
    got = []

    def work():
        try:
            R.rib_linear_fwd(x, w, y=y)
            got.append(R.rib_window_attn_fwd(qkv, 16, 0, rank=0)[0])
        except Exception as e:   # shown by the test
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.equal(y, R.rib_linear_fwd(x, w)[0])
    assert torch.equal(got[0], R.rib_window_attn_fwd(qkv, 16, 0, rank=0)[0])


# pairs of shapes that run as one instance of a kernel: one and sixteen warps of
# the norm's pipelines, column tiles of 64 and 256, rings of two and four chunks
PAIRS = {"norm": (_norm, (4, 192), (20000, 192)), "linear": (_linear, (100, 64, 64), (100, 64, 2048)),
         "feed-forward": (_ffn, (800, 64, 64), (800, 256, 64))}


@pytest.mark.parametrize("name", PAIRS)
def test_two_threads_at_once(name):
    """At shapes whose kernels take different amounts of shared memory: every call
    succeeds and gives what it gives alone."""
    make, *shapes = PAIRS[name]
    calls = [make(*s, seed=11 + 7 * i) for i, s in enumerate(shapes)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for fn, args, _, y in calls:
        assert fn(*args, torch.cuda.current_stream().cuda_stream) == 0
        alone.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    codes = [set(), set()]
    gate = threading.Barrier(2)

    def run(i):
        fn, args, _, _ = calls[i]
        st = streams[i].cuda_stream
        gate.wait()
        for k in range(CALLS):
            codes[i].add(fn(*args, st))
            if k % 500 == 499:   # bounds what is queued
                streams[i].synchronize()

    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]
    assert R.rib_last_status()[0] == 0
    for (_, _, _, y), ref in zip(calls, alone):
        assert torch.equal(y, ref)
