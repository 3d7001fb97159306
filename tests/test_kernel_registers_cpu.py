"""What the compiler reports of kernels whose speed hangs on their registers."""

import os
import re
import subprocess

from residual_vector_quantisation_gb300 import build as rqb


def resources(name, folder):
    """{kernel's mangled name: (registers, bytes spilled)} of a source file."""
    cmd = [rqb.nvcc(), *rqb.ARCH, *rqb.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(rqb.CSRC, name), "-o",
           os.path.join(folder, "out.o")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Compiling entry function '(\S+)'.*?(\d+) bytes spill stores.*?Used (\d+) registers", r.stderr, re.S)
    return {kernel: (int(registers), int(spilled)) for kernel, spilled, registers in found}


def test_the_beam_step_of_up_to_32_kept_spills_nothing(tmp_path):
    """Two blocks of 512 threads an SM have 64 registers a thread; 16-bit rows need fewer."""
    step = {k: v for k, v in resources("rvq_beam.cu", str(tmp_path)).items() if "k_beam_group" in k and "Li4E" not in k}
    assert len(step) == 3
    for kernel, (registers, spilled) in step.items():
        assert spilled == 0, kernel
        assert registers <= (64 if "If" in kernel else 56), kernel
