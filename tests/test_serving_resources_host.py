"""Registers and spills of the serving kernels, from ptxas (no GPU): what they run with is decided by
their budgets, and the spills that the tensor-core kernel has are bounded here."""
import functools
import os
import re
import subprocess

import pytest


@functools.lru_cache(maxsize=None)
def report(src, tmp):
    """{entry: (registers, bytes of spill stores, of loads)}; a kernel's helper functions that were
    not inlined have lines of their own, which are left out."""
    from compressed_attention_cvq_b200 import build as B

    try:
        nvcc = B.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    r = subprocess.run([nvcc, *B.ARCH, *B.FLAGS, "-Xptxas", "-v", "-c", os.path.join(B.CSRC, src), "-o",
                        os.path.join(tmp, src + ".o")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    spills, regs, of, entry = {}, {}, None, None
    for line in r.stderr.splitlines():
        if m := re.search(r"Compiling entry function '([^']+)'", line):
            entry = m.group(1)
        elif m := re.search(r"Function properties for (\S+)", line):
            of = m.group(1)
        elif m := re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line):
            spills[of] = int(m.group(1)), int(m.group(2))
        elif m := re.search(r"Used (\d+) registers", line):
            regs[entry] = int(m.group(1))
    return {k: (n, *spills[k]) for k, n in regs.items()}


@pytest.mark.parametrize("src,kernel,max_regs,max_spill", [
    # 27 warps on an SM: 72 registers a thread.  Its softmax holds 64 scores at once (8-scalar groups), which
    # measured faster with the spills than reading them twice without (271 and 293 us)
    ("prefix_mma.cu", "prefix_mma_kernelILi2ELb0ELi1E", 72, 512),
    ("prefix_mma.cu", "prefix_mma_kernelILi4ELb0ELi2E", 72, 512),
    ("prefix_mma.cu", "prefix_mma_kernelILi4ELb1E", 72, 160),
    ("prefix_mma.cu", "prefix_book_kernel", 64, 0),
    ("attend_f32.cu", "attend_f32_kernelILi16E", 128, 0),      # two CTAs of 256 threads an SM
    ("attend_f32.cu", "attend_f32_kernelILi64E", 255, 0),
    ("attend_f32.cu", "merge_kernel", 64, 0),
    ("paged_attend.cu", "paged_attend_kernel", 255, 0),        # two CTAs of 128 threads an SM
    ("paged_append.cu", "paged_append_kernel", 40, 0),         # twelve CTAs of 128 threads an SM
])
def test_serving_kernels_fit_their_budget(src, kernel, max_regs, max_spill, tmp_path_factory):
    res = report(src, str(tmp_path_factory.getbasetemp()))
    hits = {k: v for k, v in res.items() if kernel in k}
    assert hits, f"no {kernel} entry in the ptxas report of {src}"
    for name, (regs, stores, loads) in hits.items():
        assert regs <= max_regs, (name, regs)
        assert stores <= max_spill and loads <= max_spill, (name, stores, loads)
