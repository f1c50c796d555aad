"""Instances of the operators' kernels, from their gfx950 code objects (CPU only: hipcc
cross-compiles)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import yaml

from grpo_policy_loss_amd import build as libbuild

READELF = "/opt/rocm/llvm/bin/llvm-readelf"


def _compile(source, out):
    try:
        hipcc = libbuild.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    if not os.path.exists(READELF):
        pytest.skip("llvm-readelf not available")
    cmd = [hipcc, *libbuild.HIPCC_FLAGS, "--cuda-device-only", "--no-gpu-bundle-output", "-c",
           os.path.join(libbuild.CSRC, source), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    notes = subprocess.run([READELF, "--notes", out], capture_output=True, text=True, timeout=120).stdout
    start = notes.index("---")
    return {k[".name"]: k for k in yaml.safe_load(notes[start:notes.index("\n...", start)])["amdhsa.kernels"]}


@pytest.fixture(scope="module")
def norm(tmp_path_factory):
    return _compile("norm.hip", str(tmp_path_factory.mktemp("co") / "norm.co"))


def _backward(kernels):
    """{(type, lanes, vectors, with bias): kernel} of k_norm_bwd."""
    found = {}
    for name, k in kernels.items():
        m = re.search(r"k_norm_bwdI(DF16b|f)Li(\d+)ELi(\d+)ELb([01])E", name)
        if m:
            found["bf16" if m[1] == "DF16b" else "f32", int(m[2]), int(m[3]), m[4] == "1"] = k
    return found


def test_backward_instances_are_those_that_rows_get(norm):
    found = _backward(norm)
    assert len(found) >= 30
    for bias in (False, True):
        assert ("bf16", 512, 1, bias) in found
        assert ("f32", 512, 1, bias) not in found      # 512 lanes of one vector are for 16-bit rows
        assert ("f32", 1024, 4, bias) in found and ("bf16", 1024, 4, bias) not in found


def test_backward_instances_hold_their_rows_in_registers(norm):
    """All but those of rows above 8192 elements, where every other form is slower still."""
    for (t, lanes, vectors, bias), k in _backward(norm).items():
        if vectors < 4:
            assert k[".vgpr_spill_count"] == k[".private_segment_fixed_size"] == 0, (t, lanes, vectors, bias)
    assert ("bf16", 256, 2, True) not in _backward(norm) and ("bf16", 256, 2, False) in _backward(norm)
