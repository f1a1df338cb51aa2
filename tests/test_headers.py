"""The kernels' shared headers: any of them can be included beside any other."""
import glob
import os
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "block_quantized_gemv_w4a8_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_shared_headers_go_together(tmp_path):
    """One source includes them all (but the gates', which are parts of one source): no two functions of
    one name, of which a file could get the wrong one."""
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    names = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "qgemv_*.h")) if not p.endswith("_api.h"))
    assert {"qgemv_attn.h", "qgemv_rows.h", "qgemv_layer.h"} <= set(names)
    src = tmp_path / "all.hip"
    src.write_text("".join(f'#include "{n}"\n' for n in names))
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-std=c++17", "-fsyntax-only", "-Wno-unused-function",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
