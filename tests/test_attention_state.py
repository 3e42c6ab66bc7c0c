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


UNWIND = r"""
#include <cstdio>
#include <cstring>
#include <new>
#include "attention/attention_schedule.cuh"
using namespace nvfp4::attn;
int main()
{
    alignas(Item) unsigned char raw[sizeof(Item)];
    std::memset(raw, 0x5A, sizeof(raw));  // what lies in a register that nothing has set
    const Item it = *new (raw) Item(Item::none());
    const bool ok = it.blocks == 0 && it.t0 == 0 && it.keys == 0 && it.seen_first == 0 && it.rows == 0 && it.past0 == 0 &&
                    it.token0 == 0 && it.head == 0 && it.seq == 0 && it.part == 1;
    std::puts(ok ? "ok" : "undefined fields");
    return ok ? 0 : 1;
}
"""


def test_an_item_that_never_came_addresses_nothing(tmp_path):
    """When a warp's wait for an item runs out it goes on with Item::none() to
    the vote that ends the kernel: no rows to read, no result or gate (part 1),
    no sequence but the first."""
    if not os.path.exists(nbuild.NVCC):
        pytest.skip("nvcc not available")
    source, program = tmp_path / "unwind.cu", tmp_path / "unwind"
    source.write_text(UNWIND)
    flags = [f for f in nbuild.NVCC_FLAGS if f not in ("-shared", "-Xcompiler", "-fPIC")]
    r = subprocess.run([nbuild.NVCC, *flags, "-o", str(program), str(source)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
