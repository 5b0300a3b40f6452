"""The guard of the committed traffic counters: the hash of the routed call's
sources changes with every file its kernels are built from, and with no other."""

import os
import shutil

import bench

CSRC = os.path.join("quantized_moe_expert_route_amd", "csrc")


def test_kernel_source_hash_covers_the_calls_files_only(tmp_path):
    d = tmp_path / CSRC
    shutil.copytree(os.path.join(bench.ROOT, CSRC), d)
    before = bench.kernel_source_hash(str(tmp_path))
    assert before == bench.kernel_source_hash()
    assert set(bench.CALL_SOURCES) <= set(os.listdir(d))
    counted = set()
    for f in sorted(os.listdir(d)):
        text = (d / f).read_text()
        (d / f).write_text(text + "// more\n")
        if bench.kernel_source_hash(str(tmp_path)) != before:
            counted.add(f)
        (d / f).write_text(text)
    assert counted == set(bench.CALL_SOURCES) | {"common.h", "internal.h", "route_common.h", "shared_small.h"}
