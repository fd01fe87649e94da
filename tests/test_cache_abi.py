"""Refusals of the 8-bit state cache's calls, on the CPU: the C ABI with fake
pointers (validation rejects every call before any HIP call), and the Python
binding's checks."""
import os

import pytest
import torch

import gated_delta_rule_27_amd as kda
from test_tree_abi import (ALIAS, BAD_DTYPE, BAD_SHAPE, BF16, D, F32, MISALIGNED, NULL_ARG, OK, P, call, meta)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_27_amd import build
        build.build()
    return kda.lib()


STORE = dict(S=P(0), page=P(1), B=4, P=6, H=2, Dk=D, Dv=D, codes=P(2), scale=P(3), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD_SHAPE), (dict(P=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(H=65537), BAD_SHAPE),
    (dict(Dk=64), BAD_SHAPE), (dict(Dv=64), BAD_SHAPE), (dict(page=None, B=7), BAD_SHAPE), (dict(B=1 << 24, H=1), BAD_SHAPE),
    (dict(S=None), NULL_ARG), (dict(codes=None), NULL_ARG), (dict(scale=None), NULL_ARG),
    (dict(S=P(0, 4)), MISALIGNED), (dict(codes=P(2, 8)), MISALIGNED), (dict(scale=P(3, 4)), MISALIGNED),
    (dict(page=P(1, 2)), MISALIGNED),
    (dict(codes=P(0)), ALIAS), (dict(scale=P(0)), ALIAS), (dict(scale=P(2)), ALIAS), (dict(codes=P(1)), ALIAS),
    (dict(scale=P(1)), ALIAS), (dict(scale=P(2, 6 * 2 * D * D - 16)), ALIAS), (dict(codes=P(0, 4 * 2 * D * D * 4 - 16)), ALIAS),
    (dict(B=0, S=None), OK), (dict(P=0, codes=None), OK),
])
def test_store_refusals(L, kw, code):
    assert call(L.kda_cache_store, STORE, kw) == code


LOAD = dict(codes=P(0), scale=P(1), page=P(2), k=P(3), la=P(4), u=P(5), n=P(6), B=4, P=6, H=2, W=8, Dk=D, Dv=D, dt=BF16,
            S=P(7), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), BAD_DTYPE), (dict(B=-1), BAD_SHAPE), (dict(W=0), BAD_SHAPE), (dict(W=17), BAD_SHAPE), (dict(H=0), BAD_SHAPE),
    (dict(Dk=64), BAD_SHAPE), (dict(page=None, B=7), BAD_SHAPE), (dict(B=1 << 24, H=1), BAD_SHAPE),
    (dict(codes=None), NULL_ARG), (dict(scale=None), NULL_ARG), (dict(S=None), NULL_ARG), (dict(la=None), NULL_ARG),
    (dict(k=None), NULL_ARG), (dict(u=None), NULL_ARG),
    (dict(u=P(5, 8)), MISALIGNED), (dict(S=P(7, 4)), MISALIGNED), (dict(n=P(6, 2)), MISALIGNED), (dict(codes=P(0, 1)), MISALIGNED),
    (dict(S=P(0)), ALIAS), (dict(S=P(1)), ALIAS), (dict(S=P(2)), ALIAS), (dict(S=P(3)), ALIAS), (dict(S=P(6)), ALIAS),
    (dict(B=0, S=None), OK),
    # without windows their length, type and counts are not looked at
    (dict(k=None, la=None, u=None, W=0, dt=9, n=P(6, 1), B=0), OK),
    (dict(k=None, la=None, u=None, W=0, dt=9, S=P(0)), ALIAS),
])
def test_load_refusals(L, kw, code):
    assert call(L.kda_cache_load, LOAD, kw) == code


DECODE = dict(q=P(0), k=P(1), v=P(2), la=P(3), beta=P(4), codes=P(5), scale=P(6), wk=P(7), wa=P(8), wu=P(9), n=P(10), B=4, H=2,
              W=8, Dk=D, Dv=D, dt=F32, o=P(11), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), BAD_DTYPE), (dict(B=-1), BAD_SHAPE), (dict(W=0), BAD_SHAPE), (dict(W=17), BAD_SHAPE), (dict(H=65537), BAD_SHAPE),
    (dict(Dv=64), BAD_SHAPE), (dict(B=1 << 24, H=1), BAD_SHAPE),
    (dict(q=None), NULL_ARG), (dict(n=None), NULL_ARG), (dict(wu=None), NULL_ARG), (dict(o=None), NULL_ARG),
    (dict(beta=P(4, 2)), MISALIGNED), (dict(wk=P(7, 8)), MISALIGNED), (dict(n=P(10, 1)), MISALIGNED), (dict(o=P(11, 4)), MISALIGNED),
    (dict(o=P(0)), ALIAS), (dict(o=P(5)), ALIAS), (dict(wk=P(1)), ALIAS), (dict(wu=P(2)), ALIAS), (dict(wa=P(7)), ALIAS),
    (dict(wu=P(10)), ALIAS), (dict(o=P(9)), ALIAS), (dict(wk=P(6)), ALIAS),
    (dict(B=0, q=None, n=None), OK),
])
def test_decode_refusals(L, kw, code):
    assert call(L.kda_cache_decode, DECODE, kw) == code


FOLD = dict(codes=P(0), scale=P(1), wk=P(2), wa=P(3), wu=P(4), n=P(5), B=4, H=2, W=8, Dk=D, Dv=D, dt=BF16, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), BAD_DTYPE), (dict(B=-1), BAD_SHAPE), (dict(W=0), BAD_SHAPE), (dict(W=17), BAD_SHAPE), (dict(Dk=1), BAD_SHAPE),
    (dict(B=1 << 24, H=1), BAD_SHAPE),
    (dict(codes=None), NULL_ARG), (dict(wa=None), NULL_ARG),
    (dict(codes=P(0, 8)), MISALIGNED), (dict(n=P(5, 2)), MISALIGNED),
    (dict(codes=P(2)), ALIAS), (dict(scale=P(4)), ALIAS), (dict(scale=P(0)), ALIAS), (dict(codes=P(5)), ALIAS),
    (dict(B=0, codes=None), OK),
])
def test_fold_refusals(L, kw, code):
    assert call(L.kda_cache_fold, FOLD, kw) == code


def test_the_largest_batch_gets_past_the_shapes(L):
    most = (1 << 24) - 1
    assert call(L.kda_cache_decode, DECODE, dict(B=most, H=1, W=1, o=P(0))) == ALIAS
    assert call(L.kda_cache_fold, FOLD, dict(B=most, H=1, W=1, scale=P(0))) == ALIAS


def test_binding_refuses_what_is_not_on_a_gpu():
    c, s, w = meta(2, 3, D, D, dtype=torch.int8), meta(2, 3, D), (meta(2, 3, 4, D),) * 3
    x, n = meta(2, 3, D), meta(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_cache_store(meta(2, 3, D, D))
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_cache_load(c, s)
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_cache_decode(x, x, x, x, meta(2, 3), c, s, w, n)
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_cache_fold(c, s, w)


def test_binding_names_what_is_missing_or_misshapen():
    x, n = meta(2, 3, D), meta(2, dtype=torch.int32)
    c, s = meta(2, 3, D, D, dtype=torch.int8), meta(2, 3, D)
    with pytest.raises(TypeError, match="n_win is required"):
        kda.kda_cache_decode(x, x, x, x, meta(2, 3), c, s, (x,) * 3, None)
    with pytest.raises(ValueError, match="codes must be"):
        kda.kda_cache_load(meta(2, 3, D, dtype=torch.int8), s)
    with pytest.raises(TypeError, match="codes must be a torch.Tensor"):
        kda.kda_cache_fold(None, s, (x,) * 3)
    with pytest.raises(ValueError, match="4 dimensions"):
        kda.kda_cache_store(x)
