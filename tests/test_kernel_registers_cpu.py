"""Registers of built kernels that decide how many workgroups a CU holds, from
the metadata of the library's code objects."""
import os
import re
import struct
import subprocess

import pytest

import nvfp4_quantized_dense_amd as nv

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Registers of each kernel by its mangled name."""
    if not os.path.exists(READELF):
        pytest.skip("no llvm-readelf")
    lib, out = nv.lib()._name, {}
    with open(lib, "rb") as f:
        data = f.read()
    at = data.find(MAGIC)
    while at >= 0:
        entry = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, entry - 8)[0]):
            start, size, n = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + n].decode()
            entry += 24 + n
            if "gfx950" in target and size:
                path = str(tmp_path_factory.mktemp("code") / "object")
                with open(path, "wb") as f:
                    f.write(data[at + start:at + start + size])
                notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True, check=True).stdout
                for kernel in notes.split("- .agpr_count:")[1:]:
                    found = {k: re.search(r"\." + k + r":\s+(\S+)", kernel) for k in ("name", "vgpr_count", "private_segment_fixed_size")}
                    out[found["name"][1]] = (int(found["vgpr_count"][1]), int(found["private_segment_fixed_size"][1]))
        at = data.find(MAGIC, at + 1)
    assert out
    return out


def test_single_tokens_of_64_channels_run_five_workgroups_a_cu(kernels):
    """512 registers a lane of a SIMD, in eights: 96 for five waves. 1280 (sequence, kv head) pairs of up to 2048 keys are
    one round so, 31.5 us; with four, two rounds, 35.3."""
    names = [k for k in kernels if re.search(r"k_kv_attentionILi64ELi1ELi[12]ELb0EE", k)]
    assert len(names) == 2 and all(kernels[k][0] <= 96 and kernels[k][1] == 0 for k in names), {k: kernels[k] for k in names}
