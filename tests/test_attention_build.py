"""Register, spill and stack budgets of the attention layer's kernels, from
ptxas's resource report (no GPU: nvcc cross-compiles for sm_100a).

The limits are the current figures: a change that begins to spill, or that
costs a kernel a block of its occupancy, fails here before it reaches a GPU."""
import os
import re
import shutil
import subprocess

import pytest

from nvfp4_w4a4_quantized_act_b200 import build as nbuild

# kernel -> (max registers, max stack bytes, max spill-store bytes)
BUDGET = {
    "qk_norm_rope_kernel<128>": (48, 0, 0),   # 40 warps an SM
    "qk_norm_rope_kernel<256>": (48, 0, 0),
    "kv_append_kernel<128>": (64, 0, 0),      # 32 warps an SM
    "kv_append_kernel<256>": (64, 0, 0),
    "paged_attention_kernel<128>": (128, 8, 8),
    "paged_attention_kernel<256>": (128, 8, 8),
    "paged_decode_kernel<128>": (168, 0, 0),
    "paged_decode_kernel<256>": (168, 40, 40),
    "paged_attention_join_kernel<128, 4>": (64, 0, 0),
    "paged_attention_join_kernel<256, 4>": (64, 0, 0),
    "paged_attention_join_kernel<128, 8>": (128, 0, 0),
    "paged_attention_join_kernel<256, 8>": (128, 0, 0),
}


@pytest.fixture(scope="module")
def report():
    if not os.path.exists(nbuild.NVCC):
        pytest.skip("nvcc not available")
    entries = {}
    for source in nbuild.attention_sources():
        flags = [f for f in nbuild.NVCC_FLAGS if f != "-shared"]
        r = subprocess.run([nbuild.NVCC, *flags, "-Xptxas", "-v", "-c", "-o", os.devnull, source], capture_output=True, text=True,
                           timeout=900)
        assert r.returncode == 0, r.stderr[-3000:]
        cur = None
        for line in r.stderr.splitlines():
            m = re.search(r"Compiling entry function '([^']+)' for 'sm_100a'", line)
            if m:
                cur = entries.setdefault(m.group(1), {})
            m = re.search(r"(\d+) bytes stack frame, (\d+) bytes spill stores", line)
            if m and cur is not None and "stack" not in cur:
                cur["stack"], cur["spill"] = map(int, m.groups())
            m = re.search(r"Used (\d+) registers", line)
            if m and cur is not None:
                cur["regs"] = int(m.group(1))
    names = subprocess.run([shutil.which("c++filt") or "/usr/bin/c++filt"], input="\n".join(entries), capture_output=True, text=True,
                           check=True).stdout.splitlines()
    return dict(zip(names, entries.values()))


def test_every_kernel_has_a_budget(report):
    assert report
    for name in report:
        assert sum(k in name for k in BUDGET) == 1, name


@pytest.mark.parametrize("kernel", sorted(BUDGET))
def test_kernel_within_budget(report, kernel):
    hits = [e for name, e in report.items() if kernel in name]
    assert len(hits) == 1
    regs, stack, spill = BUDGET[kernel]
    assert hits[0]["regs"] <= regs and hits[0]["stack"] <= stack and hits[0]["spill"] <= spill, hits[0]
