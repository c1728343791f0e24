"""Recorded traffic is tied to the MLP kernels' sources and to what chooses
among them, and to nothing else."""
import os
import shutil

import bench

CSRC = os.path.join("nvfp4_quantized_dense_amd", "csrc")


def test_every_source_counts_but_the_attention_half(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    here = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == here
    same = set()
    for name in sorted(os.listdir(tmp_path / CSRC)):
        path = tmp_path / CSRC / name
        text = path.read_text()
        path.write_text(text + "\n// changed\n")
        if bench.kernel_source_hash() == here:
            same.add(name)
        path.write_text(text)
    assert "api.cpp" not in same and "device_common.h" not in same and "tiled.hip" not in same
    assert same == {"attention.h", "attention_api.cpp", "norm_quant.hip", "kv_attention.hip", "kv_attention_common.h",
                    "kv_attention_plan.h", "kv_attention_tile.hip", "kv_cache.hip", "kv_layout.h"}
    assert "attention" not in (tmp_path / CSRC / "api.cpp").read_text()  # the half left out is not in there
