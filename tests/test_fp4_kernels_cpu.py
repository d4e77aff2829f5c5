"""The registers that the kernels of the 4-bit experts take, as the library holds them."""

import os
import re
import struct
import subprocess

import pytest

import combine_expert_ffn_amd._lib as L

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _kernels(tmp_path):
    """{mangled name: (registers per lane, spilled ones)} of the library's gfx950 kernels."""
    if not os.path.exists(READELF):
        pytest.skip("no llvm-readelf")
    data, found = open(L.LIB_PATH, "rb").read(), {}
    for m in re.finditer(re.escape(MAGIC), data):
        at, p = m.start(), m.start() + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, p - 8)[0]):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            target, p = data[p + 24: p + 24 + n], p + 24 + n
            if b"gfx950" not in target or not size:
                continue
            path = tmp_path / "code"
            path.write_bytes(data[at + off: at + off + size])
            notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True,
                                   check=True).stdout
            for k in notes.split("\n  - ")[1:]:
                name, regs, spill = (re.search(rf"\.{f}:\s+(\S+)", k) for f in (
                    "name", "vgpr_count", "vgpr_spill_count"))
                if name and regs:
                    found[name[1]] = int(regs[1]), int(spill[1])
    return found


def test_few_row_kernels_leave_two_waves_to_a_simd(tmp_path):
    """512 registers per lane and SIMD; vgpr_count holds both kinds."""
    small = {n: v for n, v in _kernels(tmp_path).items() if "fp4_small_kernel" in n}
    assert small
    over = {n: v for n, v in small.items() if v[0] > 256 or v[1]}
    assert not over, over
