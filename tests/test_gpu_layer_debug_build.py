"""The layer operators in the bounds-checked debug build: every entry point
runs once in each build, in a process of its own; no guarded access may fall
outside its buffer and every output must equal the release build's, bit for
bit (all their sums run in a fixed order)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from windowed_attention_implicit_b200 import build as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_RUN = r"""
import ctypes, sys
import numpy as np, torch
import rib_inputs as I
import windowed_attention_implicit_b200 as R
out = {}
def rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    return I.randn(shape, seed=seed, std=std).to(dtype).cuda()
def keep(name, got):
    torch.cuda.synchronize()
    code, site = R.rib_last_status()
    if code:
        info = (ctypes.c_ulonglong * 2)()
        R.library().rib_debug_guard_info(info)
        raise SystemExit(f"{name}: status {code} at site {site}, index {info[0]} of {info[1]}")
    got = got if isinstance(got, dict) else dict(enumerate(got if isinstance(got, tuple) else (got,)))
    for k, v in got.items():
        if v is not None:
            out[f"{name}_{k}"] = v.float().cpu().numpy()
f32 = torch.float32
for rows, C in ((1, 1), (77, 96), (33, 250), (9, 520), (5, 1000), (3, 2048), (3, 4104), (2, 8191)):
    for dt in (torch.bfloat16, f32):
        x, g = rand((rows, C), 1, dtype=dt), rand((C,), 2, dtype=f32)
        y, m, r = R.rib_layer_norm_fwd(x, g, g)
        keep(f"ln_{rows}_{C}_{dt}", (y, m, r))
        keep(f"lnb_{rows}_{C}_{dt}", R.rib_layer_norm_bwd(x, y, m, r, g, dres=x))
for rows, K, N in ((1, 8, 8), (300, 200, 264), (700, 1032, 72), (38401, 72, 72)):
    x, w, b = rand((rows, K), 3), rand((N, K), 4, K ** -0.5), rand((N,), 5, dtype=f32)
    r = rand((rows, N), 6)
    for act in ("none", "gelu", "silu"):
        y, pre = R.rib_linear_fwd(x, w, b, act=act, residual=r, save_pre=True)
        keep(f"lin_{rows}_{act}", (y, pre))
        keep(f"linb_{rows}_{act}", R.rib_linear_bwd(x, w, r, act=act, pre=pre, dx_add=x))
    keep(f"linb_{rows}_db", R.rib_linear_bwd(x, w, r, with_dx=False, with_dw=False))
for rows, C, H in ((1, 8, 8), (300, 200, 264), (20000, 64, 72), (700, 1032, 72), (5000, 192, 384)):
    x, dy = rand((rows, C), 7), rand((rows, C), 8)
    ffn = R.GatedFfn(rand((2, H, C), 9, C ** -0.5), rand((2, H), 10, dtype=f32),
                     rand((C, H), 11, H ** -0.5), rand((C,), 12, dtype=f32))
    for act in ("gelu", "silu"):
        keep(f"ffn_{rows}_{act}", R.rib_gated_ffn_fwd(x, ffn, act=act, residual=dy))
        keep(f"ffnb_{rows}_{act}", R.rib_gated_ffn_bwd(x, ffn, dy, act=act, dx_add=dy))
out["debug"] = np.array([R.library().rib_debug_build()])
np.savez(sys.argv[1], **out)
"""


def _run(tmp_path, debug):
    env = dict(os.environ)
    env.pop("RIB_DEBUG_LIBRARY", None)
    if debug:
        env["RIB_DEBUG_LIBRARY"] = "1"
    path = tmp_path / f"{debug}.npz"
    r = subprocess.run([sys.executable, "-c", _RUN, str(path)], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return np.load(path)


def test_layer_operators_in_bounds_and_equal_to_release(tmp_path):
    B.build(debug=True)
    rel, dbg = _run(tmp_path, False), _run(tmp_path, True)
    assert rel["debug"][0] == 0 and dbg["debug"][0] == 1
    assert sorted(rel.files) == sorted(dbg.files) and len(rel.files) > 100
    bad = [k for k in rel.files if k != "debug" and not np.array_equal(rel[k], dbg[k])]
    assert not bad, bad
