"""Host-side test (compiles, launches nothing): the kernels that stream a decode step's weights keep everything in
registers.  How the compiler inlines the CUDA headers' functions into one kernel depends on their other uses in the
module, so a new operator can change a kernel whose source it does not touch."""
import os
import re
import subprocess

from w8a8_int8_quantized_qk_b200 import build as qkbuild


def test_decode_kernels_do_not_spill(tmp_path):
    flags = ["-cubin" if f == "-shared" else f for f in qkbuild.NVCC_FLAGS]
    run = subprocess.run([qkbuild.nvcc(), *flags, "-Xptxas", "-v", "-I", qkbuild.INCLUDE, "-I", qkbuild.CSRC, "-o",
                          str(tmp_path / "qk.cubin"), os.path.join(qkbuild.CSRC, "qk_lib.cu")],
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    found = re.findall(r"Compiling entry function '(\S*gemv_i8_(?:prefetch_)?kernel\S*)'.*?(\d+) bytes spill stores, "
                       r"(\d+) bytes spill loads", run.stdout + run.stderr, re.S)
    assert len(found) >= 14
    assert [f for f in found if f[1:] != ("0", "0")] == []
