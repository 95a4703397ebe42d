"""What the compiler makes of the tensor-core forward of attention to another sequence."""

import os
import re
import subprocess

from associative_affine_scan_gb300 import build_lib


def test_forward_has_the_registers_that_it_shares_out(tmp_path):
    """Its warpgroups hand registers to each other, shares of what the block is launched with.
    With any other number the call takes the general kernel, many times slower: so that number
    is held here."""
    src = os.path.join(build_lib.CSRC, "scan_cross_fwd.cu")
    with open(src) as f:
        want = int(re.search(r"kRegs = (\d+)", f.read()).group(1))
    r = subprocess.run([build_lib.nvcc(), *build_lib.ARCH, *build_lib.FLAGS, "-Xptxas", "-v", "-c", src, "-o",
                        str(tmp_path / "fwd.o")], capture_output=True, text=True, check=True)
    got = re.findall(r"Compiling entry function '\w*cross_fwd_kernel\w*'.*?Used (\d+) registers", r.stderr, re.S)
    assert [int(n) for n in got] == [want, want], r.stderr
