"""What the compiler does not see in the attention kernels' inline assembly, checked on
the built code without a GPU: the copies into LDS wait for the registers that they
read (as test_dma_hazards checks other sources), and a row broadcast in a multiply-add
stands behind the wait states that follow a write of its source."""
import os
import re
import shutil
import subprocess

import pytest

import test_dma_hazards as dma

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") is not None or os.path.exists("/opt/rocm/bin/hipcc")


def _assembly(tmp_path, src):
    from quant_integer_gemm_amd import build
    out = tmp_path / (src + ".s")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S",
                        os.path.join(ROOT, "quant_integer_gemm_amd", "csrc", src), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text().split("\n")


@pytest.mark.skipif(not HIPCC, reason="hipcc is not installed")
def test_copies_wait_for_their_registers(tmp_path):
    lines = _assembly(tmp_path, "attend_prompt.hip")
    assert sum(1 for line in lines if line.strip().startswith("global_load_lds")) > 0
    assert not dma._violations(lines)[:5]


def _early(lines):
    """(line, text) of row-broadcast multiply-adds whose broadcast source was written by a VALU
    instruction less than two wait states before, or whose operands an MFMA wrote less than
    24 before."""
    bad = []
    for j, line in enumerate(lines):
        t = line.strip()
        if not t.startswith("v_fmac_f32_dpp"):
            continue
        regs = [int(r) for r in re.findall(r"\bv(\d+)\b", t)]
        source, ws = regs[1], 0
        for i in range(j - 1, -1, -1):
            u = lines[i].strip()
            if re.match(r"^(\.LBB\d+_\d+|_Z\w+):", u) or ws >= 24:
                break
            if not u or u.startswith((";", ".")):
                continue
            d = re.match(r"v_\S+\s+v(?:\[(\d+):(\d+)\]|(\d+))", u)
            if d:
                lo = int(d.group(1) or d.group(3))
                hi = int(d.group(2) or d.group(3))
                if u.startswith("v_mfma"):
                    if any(lo <= r <= hi for r in regs):
                        bad.append((j + 1, u))
                elif lo <= source <= hi and ws < 2 and not u.startswith("v_fmac_f32_dpp"):
                    bad.append((j + 1, u))
            nop = re.match(r"s_nop\s+(\d+)", u)
            ws += int(nop.group(1)) + 1 if nop else 1
    return bad


def test_the_scan_sees_short_waits():
    assert _early(["v_lshlrev_b32_e32 v3, 16, v4", "s_nop 0", "v_fmac_f32_dpp v1, v3, v2 row_newbcast:0"])
    assert not _early(["v_lshlrev_b32_e32 v3, 16, v4", "s_nop 1", "v_fmac_f32_dpp v1, v3, v2 row_newbcast:0"])
    assert _early(["v_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], 0", "s_nop 7", "v_fmac_f32_dpp v1, v30, v2 row_newbcast:0"])


@pytest.mark.skipif(not HIPCC, reason="hipcc is not installed")
def test_row_broadcasts_wait_for_their_source(tmp_path):
    lines = _assembly(tmp_path, "attend_kv4.hip")
    assert sum(1 for line in lines if line.strip().startswith("v_fmac_f32_dpp")) > 0
    assert not _early(lines)[:5]
