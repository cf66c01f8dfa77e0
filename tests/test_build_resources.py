"""What the compiler says of the built kernels (code-object metadata of libmoe.so), without
a GPU."""
import os
import re
import struct
import subprocess

import pytest

import mixture_experts_layer_06_amd as moe

READELF = "/opt/rocm/llvm/bin/llvm-readelf"


def code_objects():
    """The gfx950 code objects in the library's offload bundles."""
    data = open(moe.LIB_PATH, "rb").read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        at = m.end()
        (count,) = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length]
            at += 24 + length
            if b"gfx950" in name and size:
                yield data[m.start() + offset:m.start() + offset + size]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> (registers spilled, scratch bytes) of every kernel."""
    if not os.path.exists(READELF):
        pytest.skip("no llvm-readelf")
    path = tmp_path_factory.mktemp("objects") / "object"
    found = {}
    for obj in code_objects():
        path.write_bytes(obj)
        notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        for one in notes.split(".agpr_count")[1:]:
            get = lambda k: int(re.search(rf"\.{k}:\s+(\d+)", one).group(1))  # noqa: E731
            name = re.search(r"\.name:\s+(_Z\S+)", one).group(1)
            found[name] = (get("vgpr_spill_count"), get("private_segment_fixed_size"))
    return found


def test_every_kernel_is_found(kernels):
    for part in ("down_kernel", "up_kernel", "grad_kernel", "gmm_pp_kernel", "norm_kernel", "loss_kernel"):
        assert any(part in k for k in kernels), part


@pytest.mark.parametrize("part", ["down_kernel", "up_kernel", "grad_kernel"])
def test_adapter_kernels_keep_their_sums_in_registers(kernels, part):
    """This compiler has stored a spilled accumulator partly to memory and partly to
    another register, and read back only the former."""
    spilled = {k: v for k, v in kernels.items() if part in k and any(v)}
    assert not spilled
