"""What the speed of the log-probabilities' tiles rests on, from their gfx950 code objects (CPU only: hipcc
cross-compiles): as many blocks of 4 waves share a CU's 512 registers a lane and 160 KB of LDS as they were
measured with."""
import pytest

from tests.test_operator_resources import _compile

FLOAT, BF16 = "f", "DF16b"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return _compile("tile64.hip", str(tmp_path_factory.mktemp("co") / "tile64.co"))


@pytest.mark.parametrize("name,t,rows,blocks", [
    ("k64_lse", FLOAT, 64, 4), ("k64_dz", FLOAT, 64, 4), ("k64_grads", FLOAT, 64, 4),      # (with two: 1060 in the place of 945 us)
    ("k64_dz", BF16, 64, 4), ("k64_grads", BF16, 64, 4),
    ("k64_lse", FLOAT, 32, 4), ("k64_dz", FLOAT, 32, 4), ("k64_grads", FLOAT, 32, 3), ("k64_dz", BF16, 32, 8), ("k64_grads", BF16, 32, 5)])
def test_blocks_that_fit_a_cu(kernels, name, t, rows, blocks):
    found = [k for n, k in kernels.items() if f"{name}I{t}Li{rows}E" in n]
    assert len(found) == 1, (name, sorted(kernels))
    registers = -(-found[0][".vgpr_count"] // 8) * 8      # given out by eight, of both kinds together
    assert 512 // registers >= blocks
    assert 160 * 1024 // found[0][".group_segment_fixed_size"] >= blocks
