"""The compiled linear attention kernels have matrix products of one kind each (CPU only):
all of 32 terms in bfloat16, all of 4 in float32.  A product of another length into
registers that one of 32 terms has just written has given wrong sums now and then."""
import os
import re
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from selective_state_space_54_amd import build as hipbuild

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
KINDS = {"bf16": "v_mfma_f32_16x16x32_bf16", "fp32": "v_mfma_f32_16x16x4_f32"}


def products(asm_text):
    """kernel -> the set of its matrix instructions."""
    found, kernel = {}, None
    for line in asm_text.split("\n"):
        m = re.match(r"^(_Z\S+):", line)
        if m:
            kernel = m.group(1)
        m = re.match(r"\s*(v_s?mfma\w+)", line)
        if m:
            found.setdefault(kernel, set()).add(m.group(1))
    return found


def test_products_are_found():
    asm = "\n".join(["_Za:", "\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]",
                     "_Zb:", "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[0:3], v[4:7], 0",
                     "\tv_mfma_f32_16x16x16_bf16 v[0:3], v[8:9], v[4:5], v[0:3]"])
    assert {k: len(v) for k, v in products(asm).items()} == {"_Za": 1, "_Zb": 2}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_one_kind_of_matrix_product_a_kernel():
    srcs = [s for s in hipbuild.sources() if os.path.basename(s).startswith("la_")]
    assert len(srcs) >= 10
    os.makedirs(hipbuild.OBJ_DIR, exist_ok=True)
    outdir = tempfile.mkdtemp(prefix="la_asm_", dir=hipbuild.OBJ_DIR)

    def compiled(src):
        dst = os.path.join(outdir, os.path.basename(src) + ".s")
        cmd = [HIPCC, *hipbuild.HIPCC_FLAGS, "-I", hipbuild.INCLUDE, "-I", hipbuild.CSRC,
               "--cuda-device-only", "-S", src, "-o", dst]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        with open(dst) as f:
            return products(f.read())

    try:
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            for src, kernels in zip(srcs, pool.map(compiled, srcs)):
                name = os.path.basename(src)
                kind = KINDS["bf16" if "bf16" in name else "fp32"]
                assert kernels, name
                for kernel, kinds in kernels.items():
                    assert kinds == {kind}, (name, kernel, kinds)
    finally:
        shutil.rmtree(outdir, ignore_errors=True)
