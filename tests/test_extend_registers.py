"""The chunk-attention kernels share 72 registers a thread out among their roles;
a build whose compiler gave them another count would refuse every call."""
import os
import re
import subprocess

from decode_attention_q4kv_b200 import build as B


def test_every_chunk_kernel_has_the_registers_it_shares_out(tmp_path):
    src = os.path.join(B.CSRC, "extend.cu")
    r = subprocess.run([B.nvcc(), *B.ARCH, *B.FLAGS, "-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "extend.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    text = r.stdout + r.stderr
    assert "setmaxnreg" not in text, "the compiler ignores the shares"
    wanted = int(re.search(r"kRegs = (\d+)", open(src).read()).group(1))
    kernels = re.findall(r"Compiling entry function '(\w*extend_kernel\w*)'.*?Used (\d+) registers", text, re.S)
    assert len(kernels) == 8 and {int(n) for _, n in kernels} == {wanted}
