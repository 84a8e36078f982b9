"""What the compiler gave the attention's kernels, from the metadata of the
library as it was built.  Accumulator registers are asked for to be none:
variants of these kernels that used them heavily have given wrong values."""
import os
import re
import struct
import subprocess

import pytest

import gguf_quantized_matvec_amd as g

READELF = "/opt/rocm/llvm/bin/llvm-readelf"

pytestmark = [pytest.mark.skipif(not os.path.exists(g.LIB_PATH), reason="libqmv.so not built"),
              pytest.mark.skipif(not os.path.exists(READELF), reason="no llvm-readelf")]


def code_objects(lib):
    """The device code objects of a library: entries of its offload bundles."""
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = lib.find(magic)
    while at >= 0:
        count, = struct.unpack_from("<Q", lib, at + len(magic))
        entry = at + len(magic) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", lib, entry)
            target = lib[entry + 24:entry + 24 + length]
            entry += 24 + length
            if size and b"amdgcn" in target:
                yield lib[at + offset:at + offset + size]
        at = lib.find(magic, at + 1)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> its numbers."""
    found = {}
    with open(g.LIB_PATH, "rb") as f:
        lib = f.read()
    for i, code in enumerate(code_objects(lib)):
        path = tmp_path_factory.mktemp("code") / f"{i}.elf"
        path.write_bytes(code)
        text = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        for part in re.split(r"\n  - \.", text)[1:]:
            name = re.search(r"\.name:\s+(\S*k_\S+)", part)
            if name:
                found[name.group(1)] = {k: int(v) for k, v in re.findall(r"\.?(\w+):\s+(\d+)\n", part)}
    return found


def test_attention_kernels(kernels):
    attention = {n: k for n, k in kernels.items() if "k_attn" in n}
    # heads of 1..4 blocks in three kernels, of 5..8 in one, and the join's seven widths
    assert len(attention) == 4 * 3 + 4 + 7
    for name, k in attention.items():
        assert k["agpr_count"] == 0, name
        assert k["vgpr_spill_count"] <= 16, (name, k["vgpr_spill_count"])


def test_waves_a_simd(kernels):
    """512 registers a SIMD: three waves of k_attn for heads of up to 128 elements, two of the others."""
    for name, k in kernels.items():
        if "k_attnI" in name or "k_attn_wide" in name:
            few = "k_attnI" in name and re.search(r"ILi[1-4]E", name)
            assert k["vgpr_count"] <= (168 if few else 256), name
