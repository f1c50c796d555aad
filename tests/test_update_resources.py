"""Instances of the 64 x 64 tiles, the losses over given log-probabilities and the gradients' norm, from
their gfx950 code objects (CPU only: hipcc cross-compiles): registers hold what they take, and two
blocks of the tiles fit a CU's 160 KB of LDS."""
import pytest

from tests.test_operator_resources import _compile


@pytest.mark.parametrize("source,names,lds", [("tile64.hip", ("k64_lse", "k64_merge", "k64_dz", "k64_grads", "k64_join"), 80 * 1024),
                                              ("losses.hip", ("k_clip_rows", "k_clip_segments", "k_clip_finish", "k_clip_bwd", "k_pref_rows",
                                                              "k_pref_segments", "k_pref_finish", "k_pref_bwd"), 8192),
                                              ("gradnorm.hip", ("k_grad_norm", "k_grad_finish", "k_grad_clip"), 8192)])
def test_no_spills(source, names, lds, tmp_path):
    kernels = _compile(source, str(tmp_path / "x.co"))
    for name in names:
        assert any(name in k for k in kernels), name
    for name, k in kernels.items():
        assert k[".vgpr_spill_count"] == k[".private_segment_fixed_size"] == 0, name
        assert k[".group_segment_fixed_size"] <= lds, name


def test_tiles_leave_room_for_two_blocks():
    """256 threads of at most 256 registers: two waves a SIMD."""
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        for name, k in _compile("tile64.hip", d + "/x.co").items():
            assert k[".vgpr_count"] <= 256, name
