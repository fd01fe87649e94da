"""Registers of the tree speculation kernels: the wavefronts per SIMD that
their notes count on (a workgroup of four wavefronts is one of them on every
SIMD of a compute unit), no scratch, and LDS for as many workgroups."""
import pytest

from gated_delta_rule_27_amd import build

# kernel, its instances by a part of the symbol, wavefronts per SIMD at least
WAVES = [
    ("kda_tree_decode.hip", "tree_decode_small_kernel", "", 4),
    ("kda_tree_decode.hip", "tree_decode_kernel", "Li1E", 4),
    ("kda_tree_decode.hip", "tree_decode_kernel", "Li2E", 3),
    ("kda_tree_decode.hip", "tree_decode_kernel", "Li3E", 2),
    ("kda_tree_decode.hip", "tree_decode_kernel", "Li4E", 2),
    ("kda_tree_commit.hip", "tree_commit_kernel", "Lb0E", 4),
    ("kda_tree_commit.hip", "tree_commit_kernel", "Lb1E", 3),
    ("kda_tree_accept.hip", "tree_accept_kernel", "", 4),       # one workgroup of sixteen
    ("kda_layer.hip", "tree_prologue_kernel", "", 4),
]


@pytest.fixture(scope="module")
def usage():
    return {src: build.resource_usage(src) for src in {w[0] for w in WAVES}}


@pytest.mark.parametrize("src,kernel,part,waves", WAVES)
def test_tree_kernels_hold_their_wavefronts(usage, src, kernel, part, waves):
    found = {k: v for k, v in usage[src].items() if kernel in k and part in k.split(kernel)[1]}
    assert len(found) >= 2, (kernel, part)   # (both types)
    for k, v in found.items():
        assert v["occupancy"] >= waves, (k, v)
        assert v["scratch"] == 0, (k, v)
