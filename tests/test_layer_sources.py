"""What the layer operators' kernels owe the memory model, where no run can show
its absence: read from the sources."""
import os
import re

import windowed_attention_implicit_b200 as R

CSRC = os.path.join(os.path.dirname(R.__file__), "csrc")


def _code(name):
    """A source file without its comments and line breaks."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    return " ".join(text.split())


def test_the_pairs_hand_over_tensor_memory_only():
    """CTA 0 issues a pair's MMAs, which read both CTAs' memories.  The remote
    arrival is released at CTA scope: it orders tensor memory, by the tcgen05
    fences around it, but no shared memory that CTA 1's threads have written.  So
    the one-kernel feed-forward hands h over in tensor memory."""
    fused = _code("ffn_fused.cuh")
    # what the epilogue warps send to CTA 0, each behind a fence
    assert set(re.findall(r"to_leader\(&bb\.(\w+)", fused)) == {"h_full", "y_free"}
    assert len(re.findall(r"mbar_arrive_remote\(", fused)) == 1    # in to_leader
    # h: stored to tensor memory, complete, fenced, handed over, with nothing between
    assert re.search(r"tmem_st_x8\(acc, out\); tmem_wait_st\(\); tc_fence_before\(\); "
                     r"to_leader\(&bb\.h_full", fused)
    # its MMA waits, fences and takes A from tensor memory
    y = fused[fused.index("auto issue_y"):fused.index("pair_commit<2>(&bb.y_done")]
    assert re.search(r"warp_wait\(&bb\.h_full.*tc_fence_after\(\); pair_umma_ts_steps\(", y)
    assert "pair_umma_steps" not in y and "pair_umma4" not in y


def test_columns_of_h_are_not_overwritten_before_they_are_read():
    """The next GU in h's columns has another shape than the Y that reads them:
    the tensor core orders only MMAs of one shape and accumulator, so GU waits
    for Y's completion."""
    fused = _code("ffn_fused.cuh")
    gu = fused[fused.index("for (int g = 0; ok && g <= total"):fused.index("pair_commit<2>(&bb.gu_full")]
    assert re.search(r"if \(g >= 2 && !\(ok = warp_wait\(&bb\.y_done\[g & 1\], \(\(g >> 1\) - 1\) & 1,", gu)
    assert re.search(r"pair_umma_ts_steps\(.*?pair_commit<2>\(&bb\.y_done\[g & 1\]\)", fused)


def test_dependent_kernels_read_by_coherent_loads():
    """The layer's kernels are launched before the one they wait for has finished,
    so what they read is written during their life.  The non-coherent load path
    (the __ldg intrinsic, the nc loads, const restrict pointers) is for data that
    is not."""
    for name in ("layer_norm.cuh", "gemm.cuh", "ffn.cuh", "ffn_fused.cuh", "few_rows.cuh"):
        code = _code(name)
        assert "pdl_wait()" in code, name
        for path in ("__ldg", "ld.global.nc", "__restrict__", "__ldcs", "tex1D"):
            assert path not in code, (name, path)
    # the wait orders: loads cannot be moved before it
    wait = _code("layer_norm.cuh")
    assert re.search(r'asm volatile\("griddepcontrol\.launch_dependents;\\n\\tgriddepcontrol\.wait;" ::: "memory"\)',
                     wait)
