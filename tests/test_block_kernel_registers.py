"""No kernel of the 8-bit operators and norms keeps a vector register in memory
(gfx950 assembly, no GPU): none spills one and none has scratch memory."""
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_waits import _asm

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")

KERNELS = {"fp8.hip": 18 + 3 + 3, "fp8_gemm.hip": 7 + 3 + 3 + 1, "fp8_layer.hip": 4, "norms.hip": 60 + 50 + 1}


def test_no_kernel_keeps_registers_in_memory(tmp_path):
    with ThreadPoolExecutor(len(KERNELS)) as ex:
        asm = list(ex.map(lambda src: _asm(src, str(tmp_path / (src + ".s"))), KERNELS))
    for src, lines in zip(KERNELS, asm):
        blocks = "\n".join(lines).split("  - .agpr_count")[1:]
        assert len(blocks) == KERNELS[src], (src, len(blocks))
        for block in blocks:
            name = re.search(r"\.name:\s+(\S+)", block).group(1)
            for key in ("vgpr_spill_count", "private_segment_fixed_size"):
                assert int(re.search(rf"\.{key}:\s+(\d+)", block).group(1)) == 0, (name, key)
