"""What the compiler gives a kernel, where its speed hangs on how many CTAs an SM holds."""
import os
import re
import subprocess

import pytest

REGISTERS = 65536  # of an SM


def resources(source, tmp_path):
    """{mangled kernel name: registers a thread} of one source file."""
    from top_routing_grouped_gb300 import build as b
    obj = os.path.join(str(tmp_path), "x.o")
    r = subprocess.run([b.nvcc(), *b.common_flags(), "-Xptxas", "-v", "-c", os.path.join(b.CSRC, source), "-o", obj],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return {m[1]: int(m[2]) for m in re.finditer(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", r.stderr + r.stdout, re.S)}


@pytest.mark.parametrize("source, kernel, threads, ctas", [("permute.cu", "permute_kernel", 256, 2)])
def test_registers_leave_room_for_the_ctas(tmp_path, source, kernel, threads, ctas):
    """Registers are given to a warp in steps of 256, eight a thread."""
    found = {n: r for n, r in resources(source, tmp_path).items() if kernel in n}
    assert found
    for name, r in found.items():
        assert ctas * threads * (-(-r // 8) * 8) <= REGISTERS, (name, r)
