"""The traffic figure of bench.py's roofline comes from a committed Nsight Compute
summary, keyed by the sources of the kernel that it was captured on."""
import os
import re
import shutil

import pytest

import bench

PKG = "quantized_moe_expert_router_gb300"


@pytest.mark.parametrize("kernel,tag", [("expert_gemv.cu", "expert_gemv_gu_k3b1"), ("grouped.cu", "group_tc_gu_prefill512"),
                                        ("grouped.cu", "group_tc_gu_prefill512w4a4")])
def test_the_committed_summary_is_of_the_committed_kernel(kernel, tag):
    got, source = bench.ncu_traffic(kernel, tag)
    assert got is not None and got > 0, source


@pytest.fixture
def copy(tmp_path):
    shutil.copytree(os.path.join(bench.ROOT, PKG, "csrc"), tmp_path / PKG / "csrc")
    shutil.copytree(os.path.join(bench.ROOT, "include"), tmp_path / "include")
    return tmp_path


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_the_key_is_of_what_goes_into_the_kernel(copy, kernel):
    def edited(path, old, new):
        text = path.read_text()
        assert old in text
        path.write_text(text.replace(old, new))
        key = bench.kernel_sources_sha256(kernel, str(copy))
        path.write_text(text)
        return key
    header, core = copy / "include" / "moe.h", copy / PKG / "csrc" / "gemv_core.cuh"
    key = bench.kernel_sources_sha256(kernel)
    assert bench.kernel_sources_sha256(kernel, str(copy)) == key
    same = "const char *moe_status_string(moe_status status);"
    assert edited(header, same, same + "\nmoe_status moe_other(int x);\n#define MOE_OTHER 3\n") == key
    assert edited(header, "#define MOE_FLAG_TIMEOUT 0x4", "#define MOE_FLAG_TIMEOUT 0x8") != key
    assert edited(core, "kSliceSteps = 32", "kSliceSteps = 16") != key


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_every_included_file_is_in_the_key(kernel):
    """Followed from the .cu, but for the public header."""
    todo, seen = [kernel], set()
    while todo:
        name = todo.pop()
        if name in seen:
            continue
        seen.add(name)
        with open(os.path.join(bench.ROOT, PKG, "csrc", name)) as f:
            todo += [n for n in re.findall(r'#include "(.*?)"', f.read()) if n != "moe.h"]
    assert seen == set(bench.KERNEL_SOURCES[kernel])
