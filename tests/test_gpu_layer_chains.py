"""Calls in a row on one stream that write what the next reads, and over and over
into the same buffers, without a synchronisation between them: each kernel is
there before the one that it waits for has finished."""
import pytest
import torch

import rib_inputs as I
import windowed_attention_implicit_b200 as R

pytestmark = pytest.mark.gpu

bf, f32 = torch.bfloat16, torch.float32


def _rand(shape, seed, std=1.0, dtype=bf):
    return I.randn(shape, seed=seed, std=std).to(dtype).cuda()


def _done():
    torch.cuda.synchronize()
    code, site = R.rib_last_status()
    assert code == 0, f"{R.rib_status_string(code)} at site {site}"


@pytest.mark.parametrize("rows", [1, 2, 8, 40])
def test_tokens_through_one_workspace(rows):
    """A decoder's loop: norm, feed-forward, norm, projection for a few rows, its
    buffers and workspace the same in every step, against the same steps with a
    synchronisation after each call."""
    C, H, steps = 192, 512, 200
    ffn = R.GatedFfn(_rand((2, H, C), 1, C ** -0.5), _rand((2, H), 2, 0.2, f32), _rand((C, H), 3, H ** -0.5),
                     _rand((C,), 4, 0.2, f32))
    w, g = _rand((C, C), 5, C ** -0.5), 1 + _rand((C,), 6, 0.2, f32)
    n = R.rib_gated_ffn_fwd_workspace(rows, C, H)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    buf = [torch.empty((rows, C), dtype=bf, device="cuda") for _ in range(3)]
    stats = [torch.empty((rows,), device="cuda") for _ in range(2)]
    start = _rand((rows, C), 7)

    def run(wait):
        x, seen = start.clone(), []
        for _ in range(steps):
            for call in (lambda: R.rib_layer_norm_fwd(x, g, y=buf[0], mean=stats[0], rstd=stats[1]),
                         lambda: R.rib_gated_ffn_fwd(buf[0], ffn, residual=x, y=buf[1], workspace=ws),
                         lambda: R.rib_layer_norm_fwd(buf[1], g, y=buf[2], mean=stats[0], rstd=stats[1]),
                         lambda: R.rib_linear_fwd(buf[2], w, act="gelu", y=x)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen.append(x.clone())
        _done()
        return torch.stack(seen)

    assert torch.equal(run(False), run(True))


def test_backward_steps_through_one_workspace():
    """Norm and projection, forward and backward through an activation, each step
    reading the gradients that the one before has written."""
    rows, C, steps = 1000, 96, 60
    w, g = _rand((C, C), 1, C ** -0.5), 1 + _rand((C,), 2, 0.2, f32)
    ws = torch.empty(max(R.rib_linear_bwd_workspace(rows, C, C, "silu"), R.rib_layer_norm_bwd_workspace(rows, C)),
                     dtype=torch.uint8, device="cuda")
    x, start = _rand((rows, C), 3), _rand((rows, C), 4)
    y, pre, dz, dn = (torch.empty_like(x) for _ in range(4))
    out = [torch.empty((C,), device="cuda") for _ in range(3)]
    dw = torch.empty((C, C), device="cuda")
    _, mean, rstd = R.rib_layer_norm_fwd(x, g)

    def run(wait):
        d, seen = start.clone(), []
        for _ in range(steps):
            for call in (lambda: R.rib_linear_fwd(d, w, act="silu", y=y, pre=pre),
                         lambda: R.rib_linear_bwd(d, w, y, act="silu", pre=pre, dx=dz, dw=dw, db=out[0],
                                                  workspace=ws),
                         lambda: R.rib_layer_norm_bwd(x, dz, mean, rstd, g, dx=dn, dgamma=out[1], dbeta=out[2],
                                                      workspace=ws),
                         lambda: R.rib_layer_norm_fwd(dn, g, y=d, mean=rows_stat, rstd=rows_stat2)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen.append(torch.cat([d.float().flatten(), dw.flatten(), *out]))
        _done()
        return torch.stack(seen)

    rows_stat, rows_stat2 = torch.empty((rows,), device="cuda"), torch.empty((rows,), device="cuda")
    a, b = run(False), run(True)
    assert torch.isfinite(a).all() and torch.equal(a, b)
