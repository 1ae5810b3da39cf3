"""The MX product kernels load operands straight into LDS and wait for them with
s_waitcnt vmcnt immediates that count their own later loads and stores (all of
them share the counter and retire in order).  A wait vmcnt(N) covers a load
once at least N vector-memory operations were issued after it, so it is right
as long as the compiler issues all of the designed ones, in the designed
order: a missing, merged or moved one would let a wait pass early, an extra
one only makes it stricter.  These tests compile the two sources to gfx950
assembly with the library's flags and check the listings.

Few rows (rows of A in LDS): behind the last load into LDS come the first
chunks of B, ten loads without a branch, then the wait and the barrier.

Tiles: before the first barrier the scales and all stages, each stage's loads
without a branch among them, and the wait for the first stage; in the loop
the scales' loads, the wait (for the next stage, or with a whole tile's stores
and the scales behind it), the barrier, and one stage's loads without a
branch; and a whole bf16 block's stores once each.

CPU only (hipcc cross-compiles); skipped where hipcc is missing.
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_epilogue_asm import _build_module, _device_asm, _kernels

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    B, tmp = _build_module(), tmp_path_factory.mktemp("asm")
    srcs = ["mx_gemm_rows.hip", "mx_gemm_tile.hip"]
    with ThreadPoolExecutor(2) as ex:
        return [_kernels(t) for t in ex.map(lambda s: _device_asm(B, s, str(tmp / (s + ".s"))), srcs)]


def events(body):
    """What matters, in program order: "L" a load into LDS, "S" a 16-byte buffer
    store, "x" another vector-memory operation, an integer the immediate of a
    vmcnt wait, "|" a branch or a label, "B" a barrier."""
    out = []
    for line in body:
        line = line.split(";")[0].rstrip()
        tok = line.split()
        if not tok:
            continue
        if tok[0].startswith("s_cbranch") or tok[0] == "s_branch" or re.match(r"\.LBB\S+:", tok[0]):
            out.append("|")
        elif tok[0].startswith(("buffer_", "global_", "flat_", "scratch_")):
            out.append("L" if line.endswith(" lds") else "S" if tok[0] == "buffer_store_dwordx4" else "x")
        elif tok[0] == "s_waitcnt":
            m = re.search(r"vmcnt\((\d+)\)", line)
            if m:
                out.append(int(m.group(1)))
        elif tok[0] == "s_barrier":
            out.append("B")
    return out


def runs(ev, what="L"):
    """Lengths of the runs of `what` that no branch or label interrupts."""
    out, n = [], 0
    for e in ev + ["|"]:
        if e == what:
            n += 1
        elif e == "|" and n:
            out.append(n)
            n = 0
    return out


def rows_ok(ev):
    """A kernel for few rows with A in LDS: 2 chunks of B ahead, 4 pieces and a scale each."""
    first = ev.index("B")
    last = max(i for i, e in enumerate(ev[:first]) if e == "L")
    behind = ev[last + 1:first]
    while behind and behind[0] == "|":     # the end of the loop that loads
        behind = behind[1:]
    waits = [e for e in behind if isinstance(e, int)]
    return (len(waits) == 1 and behind[-1] == waits[0] and behind[:-1].count("x") >= waits[0]
            and set(behind[:-1]) == {"x"} and waits[0] <= 10)


def tile_geometry(a8, bf16, nb):
    la, lb = 64 * nb * 128 // 4096, 64 * nb * (64 if a8 else 128) // 4096
    return dict(loads=la + lb, stages=3 if a8 else 2, scales=2 * 64 * nb * 16 // 4096, stores=2 * nb * nb if bf16 else 0)


def tile_ok(ev, loads, stages, scales, stores):
    first = ev.index("B")
    second = ev.index("B", first + 1)
    before, loop, behind = ev[:first], ev[first + 1:second], ev[second + 1:]
    last = max(i for i, e in enumerate(before) if e == "L")
    first_wait = [e for e in before[last:] if isinstance(e, int)]
    ahead = (stages - 2) * loads            # of the stages behind the next one
    allowed = {0, ahead} | ({ahead + stores + scales} if stores else set())
    # the three forms of the wait stand behind branches; what else waits (for a bias) waits for all
    waits = {e for i, e in enumerate(loop) if isinstance(e, int) and loop[i - 1] == "|"}
    others = [e for e in loop if isinstance(e, int) and e > max(allowed)]
    return (runs(before) == [scales] + [loads] * stages and first_wait[-1] <= (stages - 1) * loads
            and sum(runs(loop)) == scales and waits and waits <= allowed and not others
            and runs(behind) == [loads] and ev.count("S") == stores)


def test_few_rows(listings):
    checked = 0
    for name, body in listings[0].items():
        m = re.search(r"mx_gemm_rows_kernelILi(\d)ELi(\d)ELb(\d)ELb(\d)ELb1ELi(\d)E", name)
        if not m:
            continue
        assert m.group(2) == "1", name      # the wait above counts one column block
        assert rows_ok(events(body)), (name, events(body)[:200])
        checked += 1
    assert checked == 3 * 2 * 2 * 2          # row blocks, formats, outputs, numbers of waves


def test_tiles(listings):
    checked = 0
    for name, body in listings[1].items():
        m = re.search(r"mx_gemm_tile_kernelILb(\d)ELb(\d)ELi(\d)ELi(\d)ELi(\d)E", name)
        if not m:
            continue
        assert m.group(3) == m.group(4), name
        g = tile_geometry(m.group(1) == "1", m.group(2) == "1", int(m.group(3)))
        assert tile_ok(events(body), **g), (name, g)
        checked += 1
    assert checked == 2 * 2 * 3              # formats, outputs, tile sizes and split K


def test_the_checks_see_what_is_missing(listings):
    """A load or store taken out of a listing, or a branch put before one, is found."""
    name, body = next((n, b) for n, b in listings[0].items() if "ILi1ELi1ELb1ELb1ELb1ELi8E" in n)
    ev = events(body)
    first = ev.index("B")
    x = max(i for i, e in enumerate(ev[:first]) if e == "x")
    assert rows_ok(ev) and not rows_ok(ev[:x] + ev[x + 1:]) and not rows_ok(ev[:x] + ["|"] + ev[x:])
    name, body = next((n, b) for n, b in listings[1].items() if "ILb1ELb1ELi4ELi4ELi1E" in n)
    ev, g = events(body), tile_geometry(True, True, 4)
    assert tile_ok(ev, **g)
    for what in "LS":
        for i in [k for k, e in enumerate(ev) if e == what]:
            assert not tile_ok(ev[:i] + ev[i + 1:], **g)
    i = max(k for k, e in enumerate(ev) if e == "L")
    assert not tile_ok(ev[:i] + ["|"] + ev[i:], **g)
