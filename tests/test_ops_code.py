"""Compiled-code checks of the operators around the step (no GPU needed): no
kernel uses scratch memory, and none contains packed-fp32 arithmetic."""
import os
import re
import shutil
import subprocess

import pytest

from matrix_orthogonalizing_optimizer_amd import build as B

SOURCES = ["row_ops.hip", "linear8_y.hip", "linear8_dw.hip", "linear8_dx.hip"]


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_no_packed_fp32(src, tmp_path):
    h = B._hipcc()
    if not (os.path.exists(h) or shutil.which(h)):
        pytest.skip("hipcc not available")
    out = tmp_path / (src + ".s")
    cmd = [h] + B.hip_flags() + ["--cuda-device-only", "-S", "-o", str(out), "-Rpass-analysis=kernel-resource-usage",
                                 os.path.join(B.CSRC, src)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert names and len(names) == len(scratch)
    assert not [(n, s) for n, s in zip(names, scratch) if s]
    assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32\b", out.read_text())
