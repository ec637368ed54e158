"""The int8 product's LDS copies are inline assembly: the scan of
test_dma_hazards on its source."""
import os
import shutil
import subprocess

import pytest

from test_dma_hazards import ROOT, _violations


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc is not installed")
def test_int8_copies_wait_for_their_registers(tmp_path):
    from quant_integer_gemm_amd import build
    out = tmp_path / "gemm_i8.s"
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S",
                        os.path.join(ROOT, "quant_integer_gemm_amd", "csrc", "gemm_i8.hip"), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = out.read_text().split("\n")
    assert sum(1 for l in lines if l.strip().startswith("global_load_lds")) > 0
    bad = _violations(lines)
    assert not bad, f"copies too close to a write of their registers (copy line, write line, wait states): {bad[:5]}"
