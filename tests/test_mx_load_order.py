"""CPU tier: the ring kernel of the MX products waits by counting the loads issued after a unit's own (an
in-order counter), which is exact only if each unit's loads all lie between its wait and the next.
This test compiles the file to gfx950 assembly and counts them in every instance's loop; and that every
read of a slot has returned before the loads that refill it are issued."""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from w4_groupwise_gemm_amd import build as B


def _asm(fmt, tmp):
    out = os.path.join(tmp, f"mx_stream_{fmt}.s")
    res = subprocess.run([B.HIPCC] + B.COMMON + B.DEVICE_FLAGS + [f"-DW4_MX_FMT={fmt}", "--cuda-device-only", "-S",
                                                                  os.path.join(B.CSRC, "mx_stream.hip"), "-o", out],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return open(out).read()


@pytest.mark.skipif(not os.path.exists(B.HIPCC) and shutil.which(B.HIPCC) is None, reason="hipcc not available")
def test_ring_loads_lie_between_their_waits():
    with tempfile.TemporaryDirectory() as tmp:
        with cf.ThreadPoolExecutor(2) as ex:
            text = "".join(ex.map(lambda f: _asm(f, tmp), (4, 8)))
    seen = 0
    for m in re.finditer(r"^_ZN2w412_GLOBAL__N_114mx_ring_kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E\S*:", text, re.M):
        fmt, rt, tt, nw, depth = map(int, m.groups())
        units = 8 // fmt
        loads = tt * 2 + rt * units
        body = text[m.end():text.index("s_endpgm", m.end())]
        lines = [l.strip() for l in body.splitlines()]
        first, second = [i for i, l in enumerate(lines) if l.startswith("s_barrier")][:2]
        # before the first barrier: the scale bytes' loads, then every unit in flight, then the wait that
        # leaves exactly those
        ahead = lines[:first]
        last = max(i for i, l in enumerate(ahead) if re.match(rf"s_waitcnt vmcnt\({depth * loads}\)", l))
        copies = max(i for i, l in enumerate(ahead) if "Inner Loop Header" in l)
        after_copies = next(i for i in range(copies, last) if ahead[i].startswith("s_cbranch"))
        assert sum(l.startswith("buffer_load") for l in ahead[after_copies:last]) == depth * loads, m.group(0)[:60]
        # the loop, from its header round to the header again
        head = next(i for i in range(first, second) if "Inner Loop Header" in lines[i])
        loop = lines[head:second] + lines[first:head]
        runs = [0]
        for l in loop:
            if re.match(rf"s_waitcnt vmcnt\({(depth - 1) * loads}\)", l):
                runs.append(0)
            elif l.startswith("buffer_load"):
                runs[-1] += 1
        assert [n for n in runs if n] == [loads] * depth, (m.group(0)[:60], runs, loads)
        # between a slot's reads and its refill every LDS operation is waited for
        pending = False
        for l in loop:
            if l.startswith("ds_read"):
                pending = True
            elif l.startswith("s_waitcnt") and "lgkmcnt(0)" in l:
                pending = False
            elif l.startswith("buffer_load") and l.endswith("lds"):
                assert not pending, (m.group(0)[:60], l)
        seen += 1
    assert seen == 48, seen
