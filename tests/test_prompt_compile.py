"""The prompt attention's kernels hold everything in registers: what is in local
memory is a cold miss where a role starts (one prompt of 64 tokens took 7.1 us
instead of 6.7 while the loading warp kept its counts there)."""
import os
import re
import subprocess

from fp8_paged_kv_kvq_gb300 import build as kbuild


def test_no_local_memory(tmp_path):
    src = os.path.join(kbuild.CSRC, "kvq_prompt.cu")
    cmd = [kbuild.nvcc(), *kbuild._flags(("-Xptxas", "-v")), "-c", src, "-o",
           str(tmp_path / "prompt.o")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    uses = re.findall(r"(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads",
                      res.stderr + res.stdout)
    assert len(uses) == 2 and all(u == ("0", "0", "0") for u in uses), uses
