"""The host layer of the calls around a cache's attention, and the plans of
calls over 4-bit caches, with AddressSanitizer and UndefinedBehaviorSanitizer on
the CPU (serve_sanitize_driver.cpp): exit status 0 and no sanitizer report."""
import os

import pytest

from tests.test_oracle_sanitizers import ROOT, SAN, run


def test_serving_host_layer_under_asan_ubsan(tmp_path):
    hipcc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    host_san = []
    for f in SAN:
        host_san += ["-Xarch_host", f]
    csrc = os.path.join(ROOT, "gguf_dequant_matvec_amd", "csrc")
    common = ["-x", "hip", "-std=c++17", "-O1", "-g", "--offload-arch=gfx950", "-I" + os.path.join(ROOT, "include"),
              "-I" + csrc, *host_san]
    objs = []
    for src in (os.path.join(csrc, "qmv_serve_api.cpp"), os.path.join(csrc, "qmv_attn_api.cpp"),
                os.path.join(csrc, "qmv_attn_plan.cpp"), os.path.join(ROOT, "tests", "serve_sanitize_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        rc, out = run([hipcc, *common, "-c", src, "-o", obj], ROOT)
        assert rc == 0, out
        objs.append(obj)
    exe = str(tmp_path / "serve_san")
    rc, out = run([hipcc, "--offload-arch=gfx950", *host_san, *objs, "-o", exe], ROOT)
    assert rc == 0, out
    rc, out = run([exe], ROOT, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert rc == 0 and "ok" in out and "runtime error" not in out and "Sanitizer" not in out, out
