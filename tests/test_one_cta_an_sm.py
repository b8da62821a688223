"""One CTA of a product an SM.  Each takes its tensor memory when it starts and waits for it
if need be; the CTAs of a split or paired tile wait for one another, and a kernel that starts
early (programmatic launch) holds what it has while it waits for the one before.  So two may
never share an SM's 512 columns, whatever shared memory a configuration leaves: registers
see to it.  Reads ptxas's report of the in-tree build."""

import os
import re

from grouped_gemm_epilogues_gb300 import build

REGISTERS, WARPS = 65536, 9    # of an SM; the fewest warps that a product's CTA has (a gathering one)


def test_registers_leave_room_for_one():
    build.build()
    current, seen = None, 0
    for line in open(os.path.join(build.BUILD, "ptxas.log")):
        m = re.search(r"Compiling entry function '(\S*gemm_kernel\S*)'", line)
        if m:
            current = m.group(1)
        r = re.search(r"Used (\d+) registers", line)
        if r and current:
            assert 2 * WARPS * 32 * int(r.group(1)) > REGISTERS, (current, line)
            current, seen = None, seen + 1
    assert seen >= 20
