"""The F8 product kernels count their own loads and stores in s_waitcnt vmcnt
immediates, as the MX product kernels do (test_mx_waits_asm.py says how and
has the checks); here the F8 kernels' listings.

CPU only (hipcc cross-compiles); skipped where hipcc is missing."""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_epilogue_asm import _build_module, _device_asm, _kernels
from test_mx_waits_asm import events, rows_ok, tile_ok

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    B, tmp = _build_module(), tmp_path_factory.mktemp("asm")
    srcs = ["f8_gemm_rows.hip", "f8_gemm_tile.hip"]
    with ThreadPoolExecutor(2) as ex:
        return [_kernels(t) for t in ex.map(lambda s: _device_asm(B, s, str(tmp / (s + ".s"))), srcs)]


def geometry(bf16, nbm, nbn):
    """128 bytes per row of both operands in a slab, two stages (four of 64 x 128); a chunk of 16 scale bytes per row."""
    rows = 64 * (nbm + nbn)
    return dict(loads=rows * 128 // 4096, stages=4 if nbm == 1 else 2, scales=-(-rows * 16 // 4096), stores=2 * nbm * nbn if bf16 else 0)


def test_few_rows(listings):
    checked = 0
    for name, body in listings[0].items():
        m = re.search(r"f8_gemm_rows_kernelILi(\d)ELi(\d)ELb(\d)ELi[1-9]\d*E", name)
        if not m:
            continue
        assert m.group(2) == "1", name      # the wait counts one column block
        assert rows_ok(events(body)), (name, events(body)[:200])
        checked += 1
    assert checked == 2 * 2                  # sizes of A in LDS, outputs


def test_tiles(listings):
    checked = 0
    for name, body in listings[1].items():
        m = re.search(r"f8_gemm_tile_kernelILb(\d)ELi(\d)ELi(\d)ELi(\d)ELb(\d)E", name)
        if not m:
            continue
        nbm, nbn = int(m.group(2)), int(m.group(3))
        assert (nbm, nbn) in ((4, 4), (2, 2), (1, 2)), name
        g = geometry(m.group(1) == "1", nbm, nbn)
        ev = events(body)
        if int(m.group(4)) == 1:         # (not of two groups of waves)
            # K is whole slabs: no branch stands between the scales' loads and the first stage's
            ev.insert([i for i, e in enumerate(ev) if e == "L"][g["scales"] - 1] + 1, "|")
        assert tile_ok(ev, **g), (name, g)
        for what in "LS":                    # and every one of them counts
            for i in [k for k, e in enumerate(ev) if e == what]:
                assert not tile_ok(ev[:i] + ev[i + 1:], **g), (name, i)
        checked += 1
    assert checked == 2 * 4 + 1              # outputs, by tile sizes and two groups of waves; K in parts into fp32


def test_no_kernel_reads_spilled_registers(listings):
    """A spill's loads would count among those that the waits count."""
    for body in [b for l in listings for b in l.values()]:
        assert not any(line.split() and line.split()[0].startswith("scratch_") for line in body)
