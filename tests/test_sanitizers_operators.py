"""The host code of the scan's and the logits' entry points under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU (tests/sanitize/operators_driver.c), built as in
test_sanitizers.py."""
from __future__ import annotations

import concurrent.futures as cf
import os

import pytest

from speculative_decode_amd import build as hip_build
from test_sanitizers import CSRC, ENV, HERE, OUT, ROOT, SAN, _digest, _run


def test_operators_host_code_under_asan_ubsan():
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    clang = "/opt/rocm/llvm/bin/clang++"
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not available")
    os.makedirs(OUT, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in hip_build.SOURCES]
    headers = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith(".h")]
    headers.append(os.path.join(ROOT, "include", "mil_ssm.h"))
    driver = os.path.join(HERE, "operators_driver.c")
    # the sanitizers go to the host pass only: each flag behind -Xarch_host
    host_san = [a for f in SAN for a in ("-Xarch_host", f)]
    key = _digest(srcs + headers + [driver], hip_build.FLAGS + host_san)
    exe = os.path.join(OUT, f"operators_driver_{key}")
    if not os.path.exists(exe):
        def compile_one(src):
            obj = os.path.join(OUT, f"{os.path.basename(src)}.{key}.o")
            _run([hipcc, *hip_build.FLAGS, *host_san, "-c", src, "-o", obj])
            return obj

        with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
            objs = list(ex.map(compile_one, srcs))
        dobj = os.path.join(OUT, f"operators_driver.{key}.o")
        _run([clang, "-x", "c", "-std=c11", "-O1", *SAN, f"-I{os.path.join(ROOT, 'include')}", "-c", driver,
              "-o", dobj])
        _run([clang, *SAN, "-o", exe, dobj, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    r = _run([exe], env=ENV)
    assert r.stdout.strip().endswith("OK"), r.stdout
    assert "runtime error" not in r.stderr and "ERROR: AddressSanitizer" not in r.stderr, r.stderr
