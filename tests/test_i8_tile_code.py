"""The built code of the tiled 8-bit products: the order of its last steps.

The loop requests parts behind the last step, whose offsets lie past the
descriptor: they write zeros to LDS and are in flight when the loop ends.  A wave
waits for its own; the tile's scales, which take the place of the first part, may
be stored only when every wave has."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from conftest import ROOT

LIBPATH = os.path.join(ROOT, "online_activation_aware_amd", "libttq.so")
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"

pytestmark = pytest.mark.skipif(not (os.path.exists(LIBPATH) and os.path.exists(OBJDUMP)), reason="libttq.so or llvm-objdump is not there")


def device_code(lib, kernel):
    """The gfx950 code object of a library that holds a kernel of this name."""
    at = lib.find(BUNDLE)
    while at >= 0:
        p = at + len(BUNDLE)
        count, p = struct.unpack_from("<Q", lib, p)[0], p + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", lib, p)
            target = lib[p + 24:p + 24 + n]
            p += 24 + n
            code = lib[at + offset:at + offset + size]
            if b"gfx950" in target and kernel in code:
                return code
        at = lib.find(BUNDLE, at + 1)
    raise AssertionError("no code of that kernel")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: instructions} of k_i8_tile's instances."""
    path = tmp_path_factory.mktemp("code") / "i8.co"
    with open(LIBPATH, "rb") as f:
        path.write_bytes(device_code(f.read(), b"k_i8_tile"))
    text = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
    found, lines = {}, None
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(\w+)>:", line)
        if head:
            lines = found.setdefault(head.group(1), []) if "k_i8_tile" in head.group(1) else None
        elif lines is not None and line.strip():
            lines.append(line.split("//")[0].strip())
    return found


def test_scales_are_stored_behind_every_wave_s_dma(kernels):
    assert len(kernels) == 16                            # four tiles: bf16, fp32, gate and up, parts
    stores = 0
    for name, lines in kernels.items():
        first = next((i for i, l in enumerate(lines) if l.startswith("ds_write")), None)
        if first is None:                                # parts: their sums leave without scales
            continue
        stores += 1
        steps = [l for l in lines[:first] if l.startswith("s_barrier") or "vmcnt(0)" in l or l.endswith(" lds")]
        assert steps[-1].startswith("s_barrier") and "vmcnt(0)" in steps[-2], (name, steps[-3:])
    assert stores == 12
