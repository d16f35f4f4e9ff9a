"""What the compiler made of the block operators' kernels (gfx950 assembly, no
GPU): the matrix tiles read LDS without waiting for the loads of later stages,
and the norms' gradients keep their row in registers, without spilling any."""
import re
import shutil

import pytest

from test_kernel_waits import _asm, _waits_before_lds_reads

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")


def kernel(lines, name):
    """The lines of each kernel whose name holds `name`."""
    out, cur = {}, None
    for line in lines:
        m = re.match(r"(_Z\w*):", line)
        if m:
            cur = m.group(1) if name in m.group(1) else None
        if cur:
            out.setdefault(cur, []).append(line)
    return out


def test_tiles_read_lds_beside_loads_in_flight(tmp_path):
    kernels = kernel(_asm("fp8_gemm.hip", str(tmp_path / "g.s")), "tile_kernel")
    assert len(kernels) == 10
    for name, lines in kernels.items():
        assert not _waits_before_lds_reads(lines), name


def test_norm_gradients_spill_no_register(tmp_path):
    text = "\n".join(_asm("norms.hip", str(tmp_path / "n.s")))
    found = 0
    for block in text.split("  - .agpr_count")[1:]:
        name, spilled = re.search(r"\.name:\s+(\S+)", block), re.search(r"\.vgpr_spill_count:\s+(\d+)", block)
        if name and "norm_bwd_kernel" in name.group(1):
            assert int(spilled.group(1)) == 0, name.group(1)
            found += 1
    assert found == 50                                          # 5 pairs of types, 5 widths, 2 ends
