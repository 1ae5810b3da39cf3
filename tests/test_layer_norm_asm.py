"""The layer norm's kernels that keep a row in registers without spilling, as
layer_norm.hip says of them: the listings hold no scratch accesses.

CPU only (hipcc cross-compiles); skipped where hipcc is missing."""
import os
import re
import shutil

import pytest

from test_epilogue_asm import _build_module, _device_asm, _kernels

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


def in_registers(name):
    m = re.search(r"layer_norm_kernelILi\dELi\dELi(\d)ELi\dELi\d+E", name)
    if m:                                                # forward: up to two pieces to a lane
        return int(m.group(1)) <= 2
    m = re.search(r"layer_norm_backward_kernelILi\dELb(\d)ELi(\d)ELi(\d)ELi\d+E", name)
    if m:                                                # one piece, or two from the stream on aligned rows
        kept, pieces, access = (int(g) for g in m.groups())
        return pieces == 1 or (pieces == 2 and not kept and access != 0)
    return "layer_norm_columns_kernel" in name or "layer_norm_dweight_kernel" in name


def test_rows_in_registers(tmp_path):
    kernels = _kernels(_device_asm(_build_module(), "layer_norm.hip", str(tmp_path / "layer_norm.s")))
    checked = [n for n in kernels if in_registers(n)]
    # forward: outputs by accesses of both types by row lanes, of one piece and two; gradient: 2 types' sources, accesses
    # and lanes of one piece, and of two from the stream; the columns' kernels; the one that adds them
    assert len(checked) == 3 * 5 * (3 + 1) + 2 * 5 * 3 + (1 + 2) + 2 * 2 * 2 + 1, len(checked)
    for n in checked:
        assert not any(line.split() and line.split()[0].startswith("scratch_") for line in kernels[n]), n
