"""The compiled kernels of the recurrent layer's operators (CPU only): no buffer store of more than
eight bytes has an SGPR offset.  The compiler puts no wait between such a store and an instruction
that writes its data registers, and the store has then written the new values now and then."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from selective_state_space_54_amd import build as hipbuild

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["gated_recurrence.hip", "causal_conv.hip", "residual_norm.hip"]


def wide_stores_with_offset(asm_text):
    """Lines with a buffer store of three or four words whose offset is a scalar register."""
    bad = []
    for i, line in enumerate(asm_text.split("\n")):
        m = re.match(r"\s*buffer_store_dwordx[34]\s+[^,]+,\s*[^,]+,\s*s\[[^\]]+\],\s*(\S+)", line)
        if m and re.match(r"(s\d+|m0)", m.group(1)):
            bad.append(i + 1)
    return bad


def test_a_scalar_offset_is_found():
    asm = "\n".join(["\tbuffer_store_dwordx4 v[0:3], v89, s[28:31], s71 offen",
                     "\tbuffer_store_dwordx4 v[0:3], v89, s[28:31], 0 offen",
                     "\tbuffer_store_dwordx2 v[0:1], v89, s[28:31], s71 offen"])
    assert wide_stores_with_offset(asm) == [1]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", SOURCES)
def test_no_wide_buffer_store_has_a_scalar_offset(source):
    os.makedirs(hipbuild.OBJ_DIR, exist_ok=True)
    outdir = tempfile.mkdtemp(prefix="rl_asm_", dir=hipbuild.OBJ_DIR)
    try:
        dst = os.path.join(outdir, source + ".s")
        r = subprocess.run([HIPCC, *hipbuild.HIPCC_FLAGS, "-I", hipbuild.INCLUDE, "-I", hipbuild.CSRC,
                            "--cuda-device-only", "-S", os.path.join(hipbuild.CSRC, source), "-o", dst],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        text = open(dst).read()
        assert "s_endpgm" in text
        assert not wide_stores_with_offset(text)
    finally:
        shutil.rmtree(outdir, ignore_errors=True)
