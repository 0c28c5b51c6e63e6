"""The operators' host planning (include/qsgd_ops.h) under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by a small program (no kernel is launched)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_sgd_amd", "csrc")


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_host_planning_of_the_operators_under_sanitizers(tmp_path):
    objs, running = [], []
    for src in (os.path.join(CSRC, "int8_api.hip"), os.path.join(CSRC, "distill_api.hip"),
                os.path.join(ROOT, "tests", "sanitize", "ops_host_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        running.append(subprocess.Popen(
            ["/opt/rocm/bin/hipcc", "-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
             "-I", CSRC, "-c", src, "-o", obj], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
        objs.append(obj)
    for p in running:
        out, _ = p.communicate(timeout=900)
        assert p.returncode == 0, out[-3000:]
    exe = str(tmp_path / "ops_host")
    link = subprocess.run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-fsanitize=address", "-fsanitize=undefined",
                           "-fno-gpu-sanitize", *objs, "-o", exe], capture_output=True, text=True, timeout=600)
    assert link.returncode == 0, link.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "ok" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])
