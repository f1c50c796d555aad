"""The host code of the operators around the loss (argument checks, workspace sizes, the
AdamW plan) built with AddressSanitizer and UndefinedBehaviorSanitizer, driven by
tests/sanitize/ops_host_checks.cpp.  CPU only, and the device code is not instrumented, as
in test_sanitized_host.py, whose host flags it takes."""
import os
import subprocess

import pytest

from grpo_policy_loss_amd import build as libbuild
from tests.test_sanitized_host import HERE, HOST_SANITIZE, ROOT


def test_operators_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    try:
        hipcc = libbuild.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    objs, procs = [], []
    for src in libbuild.SOURCES:
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        flags = [f for f in libbuild.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"] + HOST_SANITIZE
        cmd = [hipcc, *flags, "-c", os.path.join(libbuild.CSRC, src), "-o", obj]
        procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
        objs.append(obj)
    for p in procs:
        out, _ = p.communicate(timeout=600)
        assert p.returncode == 0, out.decode(errors="replace")[-3000:]
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc)))
    clangxx = "/opt/rocm/llvm/bin/clang++"
    exe = str(tmp_path / "ops_host_checks")
    cmd = [clangxx, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-I", os.path.join(ROOT, "include"), os.path.join(HERE, "sanitize", "ops_host_checks.cpp"),
           *objs, "-L", os.path.join(rocm, "lib"), "-lamdhip64",
           "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "host checks passed" in r.stdout
