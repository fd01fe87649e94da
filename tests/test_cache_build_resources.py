"""Registers of the 8-bit cache's and of sampling's kernels: the wavefronts per SIMD
that their notes count on (a workgroup of four wavefronts is one of them on every
SIMD of a compute unit), no scratch."""
import pytest

from gated_delta_rule_27_amd import build

# kernel, its instances by a part of the symbol, wavefronts per SIMD at least, scratch bytes at most
WAVES = [
    ("kda_cache.hip", "cache_store_kernel", "", 5, 0),
    ("kda_cache.hip", "cache_load_kernel", "Lb0E", 5, 0),
    ("kda_cache.hip", "cache_load_kernel", "Lb1E", 3, 0),
    ("kda_cache.hip", "cache_fold_kernel", "IDF16bLi8E", 5, 0),
    ("kda_cache.hip", "cache_fold_kernel", "IfLi8E", 4, 0),
    ("kda_cache.hip", "cache_fold_kernel", "IDF16bLi16E", 3, 0),
    ("kda_cache.hip", "cache_fold_kernel", "IfLi16E", 3, 0),
    ("kda_cache_decode.hip", "cache_decode_kernel", "", 4, 0),
    ("kda_sample.hip", "sample_tiles_kernel", "", 8, 0),
    ("kda_sample.hip", "sample_rows_kernel", "", 4, 0),       # one workgroup of sixteen
    ("kda_sample.hip", "sample_probs_kernel", "", 8, 0),
]


@pytest.fixture(scope="module")
def usage():
    return {src: build.resource_usage(src) for src in {w[0] for w in WAVES}}


@pytest.mark.parametrize("src,kernel,part,waves,scratch", WAVES)
def test_kernels_hold_their_wavefronts(usage, src, kernel, part, waves, scratch):
    found = {k: v for k, v in usage[src].items() if kernel in k and part in k.split(kernel)[1]}
    assert found, (kernel, part)
    for k, v in found.items():
        assert v["occupancy"] >= waves, (k, v)
        assert v["scratch"] <= scratch, (k, v)
