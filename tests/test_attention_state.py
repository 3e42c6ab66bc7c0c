"""What the attention kernels' warps hand one another from item to item, from
the headers alone (no GPU: nvcc compiles a few assertions)."""
import os
import subprocess

import pytest

from nvfp4_w4a4_quantized_act_b200 import build as nbuild

SOURCE = r"""
#include <type_traits>
#include "attention/paged_attention_kernel.cuh"
using namespace nvfp4::attn;
template <int D> void check() {
    using S = AttnSmem<D>;
#define TWO(member) static_assert(std::rank<decltype(S::member)>::value >= 1 && std::extent<decltype(S::member)>::value == 2, #member)
%s
}
template void check<128>();
template void check<256>();
"""


@pytest.mark.parametrize("member", ["row_scale", "sum", "ref", "nan_any", "nan_key"])
def test_item_state_is_kept_by_parity(member, tmp_path):
    """Warps that have finished an item write the next one's state while others
    still read this one's: each such array has a copy for even and odd items."""
    if not os.path.exists(nbuild.NVCC):
        pytest.skip("nvcc not available")
    source = tmp_path / "state.cu"
    source.write_text(SOURCE % f"    TWO({member});")
    flags = [f for f in nbuild.NVCC_FLAGS if f != "-shared"]
    r = subprocess.run([nbuild.NVCC, *flags, "-c", "-o", os.devnull, str(source)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
