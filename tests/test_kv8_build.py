"""What the compiler made of the extend over the 8-bit cache (host: reads its report, launches nothing)."""

import os
import re

from int2_rotated_kv_append_gb300 import build


def test_extend_kernels_have_the_launch_registers_that_their_warpgroups_divide():
    # the kernel's warpgroups exchange 512 x 128 registers among themselves; the host refuses to launch it with any other
    # number, so that a compiler that gives another is noticed here
    build.build()
    log = os.path.join(build.BUILD, "ptxas.log")
    if not os.path.exists(log):
        build.build(force=True)
    found = re.findall(r"Compiling entry function '(\S*kv8_extend_kernel\S*)'.*?Used (\d+) registers", open(log).read(), re.S)
    assert len(found) == 12 and all(int(n) == 128 for _, n in found), found
