"""What the benchmark derives without a GPU."""
import shutil

import pytest

import bench


@pytest.mark.parametrize("stage,parts", [("fwd_bf16", []), ("bwd_bf16", ["bwd_parts.cuh"]), ("fwd_fp8", ["fp8_row.cuh"]),
                                         ("fp8_prepass", ["fp8_row.cuh"])])
def test_traffic_digests_cover_included_files(stage, parts, tmp_path):
    """A change in any file that the stage's kernel is compiled from makes its traffic figure old."""
    names = bench.kernel_sources(stage)
    assert names[0] == bench.KERNEL_SOURCES[stage] and len(names) == len(set(names))
    assert {"sm103_prims.cuh", "common.h", *parts} <= set(names)
    csrc = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, csrc)
    digest = bench.kernel_source_digest(stage)
    assert len(digest) == 16 and digest == bench.kernel_source_digest(stage, str(csrc))
    for name in names:
        with open(csrc / name, "a") as f:
            f.write("// changed\n")
        changed = bench.kernel_source_digest(stage, str(csrc))
        assert changed != digest
        digest = changed
