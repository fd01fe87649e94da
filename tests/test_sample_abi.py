"""Refusals of kda_sample, on the CPU: the C ABI with fake pointers (validation
rejects every call before any HIP call), and the Python binding's checks."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_27_amd as kda
from test_tree_abi import ALIAS, BAD_DTYPE, BAD_SHAPE, F32, MISALIGNED, NULL_ARG, OK, P, WORKSPACE, call, meta


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_27_amd import build
        build.build()
    return kda.lib()


BIG = 1 << 35
SAMPLE = dict(logits=P(0), u=P(1), T=P(2), k=P(3), p=P(4), m=P(5), R=4, V=1000, dt=F32, token=P(6), probs=P(7), ws=P(8),
              size=ctypes.c_size_t(BIG), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), BAD_DTYPE),
    (dict(R=-1), BAD_SHAPE), (dict(V=0), BAD_SHAPE), (dict(V=(1 << 22) + 1), BAD_SHAPE), (dict(R=1 << 22, V=1), BAD_SHAPE),
    (dict(R=1 << 14, V=1 << 22), BAD_SHAPE),
    (dict(logits=None), NULL_ARG), (dict(token=None), NULL_ARG), (dict(u=None, probs=None), NULL_ARG), (dict(ws=None), NULL_ARG),
    (dict(logits=P(0, 4)), MISALIGNED), (dict(probs=P(7, 8)), MISALIGNED), (dict(ws=P(8, 8)), MISALIGNED),
    (dict(u=P(1, 2)), MISALIGNED), (dict(T=P(2, 1)), MISALIGNED), (dict(k=P(3, 2)), MISALIGNED), (dict(p=P(4, 3)), MISALIGNED),
    (dict(m=P(5, 2)), MISALIGNED), (dict(token=P(6, 1)), MISALIGNED),
    (dict(size=ctypes.c_size_t(4 * 12 + 4 * 40 - 1)), WORKSPACE), (dict(size=ctypes.c_size_t(0)), WORKSPACE),
    (dict(probs=P(0)), ALIAS), (dict(probs=P(1)), ALIAS), (dict(token=P(1)), ALIAS), (dict(token=P(7)), ALIAS),
    (dict(ws=P(0)), ALIAS), (dict(ws=P(7)), ALIAS), (dict(ws=P(6)), ALIAS), (dict(token=P(3)), ALIAS),
    (dict(probs=P(0, 4 * 1000 * 4 - 16)), ALIAS), (dict(ws=P(2)), ALIAS),
    (dict(R=0, logits=None, ws=None), OK),
])
def test_sample_refusals(L, kw, code):
    assert call(L.kda_sample, SAMPLE, kw) == code


def test_without_random_numbers_the_token_is_not_looked_at(L):
    assert call(L.kda_sample, SAMPLE, dict(u=None, token=P(0, 1), ws=P(7))) == ALIAS


def test_workspace_size(L):
    # a float and a double a tile of 1024, and what is kept of a row
    size = L.kda_sample_workspace_size
    assert size(0, 5) == 0 and size(-1, 5) == 0 and size(5, 0) == 0 and size(1 << 22, 1) == 0 and size(1, (1 << 22) + 1) == 0
    assert size(1, 1) >= 12 + 40 and size(256, 160000) >= 256 * (157 * 12 + 40)
    for R, V in ((1, 1), (3, 1025), (256, 160000), (2048, 500)):
        assert call(L.kda_sample, SAMPLE, dict(R=R, V=V, size=ctypes.c_size_t(size(R, V) - 1))) == WORKSPACE
        assert call(L.kda_sample, SAMPLE, dict(R=R, V=V, size=ctypes.c_size_t(size(R, V)), probs=P(0))) == ALIAS


def test_the_largest_calls_get_past_the_shapes(L):
    assert call(L.kda_sample, SAMPLE, dict(R=(1 << 22) - 1, V=1, token=P(1))) == ALIAS
    assert call(L.kda_sample, SAMPLE, dict(R=((1 << 24) - 1) // 1025, V=1 << 22, token=P(1))) == ALIAS


def test_binding_refuses():
    x, u = meta(2, 9), meta(2)
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_sample(x, u)
    with pytest.raises(TypeError, match="logits must be a torch.Tensor"):
        kda.kda_sample([1.0], u)
    with pytest.raises(TypeError, match="logits must be a torch.Tensor"):
        kda.kda_sample(torch.tensor(1.0), u)
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.kda_sample(x.half().to("cuda") if torch.cuda.is_available() else _Fake(x.half()), u)


class _Fake(torch.Tensor):
    """A tensor that says it is on a GPU."""
    def __new__(cls, t):
        return t.as_subclass(cls)

    def get_device(self):
        return 0
