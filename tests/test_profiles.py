"""The recorded DRAM traffic of a kernel belongs to what it compiles from, not to the other calls that the library declares."""
import os
import re
import shutil

import pytest

import bench

CALL = "\nOKV_API okv_status okv_of_another_kind(int32_t n, void* stream);\n"


@pytest.mark.parametrize("profile", ["attend_mma_qwen3_8b_16k.md", "stage_kernel_qwen3_8b_16k.md"])
def test_traffic_outlives_declarations_of_other_calls(tmp_path, monkeypatch, profile):
    text = open(os.path.join(bench.ROOT, "profiles", profile)).read()
    sources = re.search(r"bench: traffic_bytes_per_launch=\d+ source=(\S+)", text).group(1).split(",")
    for path in ["include/okv.h", "profiles/" + profile] + sources:
        to = tmp_path / path
        to.parent.mkdir(parents=True, exist_ok=True)
        shutil.copy(os.path.join(bench.ROOT, path), to)
    with open(tmp_path / "include" / "okv.h", "a") as f:
        f.write(CALL)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    traffic = bench.profiled_traffic(profile)
    assert traffic is not None
    with open(tmp_path / sources[0], "a") as f:  # a change of the kernel still ends it
        f.write("\n")
    assert bench.profiled_traffic(profile) is None
