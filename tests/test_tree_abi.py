"""Refusals of the tree speculative decoding calls, on the CPU: the C ABI with
fake pointers (validation rejects every call before any HIP call), and the
Python binding's shape, dtype and device checks (no call gets past them
without a GPU tensor)."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_27_amd as kda

OK, NULL_ARG, BAD_SHAPE, BAD_DTYPE, MISALIGNED, ALIAS, WORKSPACE, DEVICE = range(8)
F32, BF16 = 0, 1
D = 128
BASE, GAP = 1 << 40, 1 << 36


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_27_amd import build
        build.build()
    return kda.lib()


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * GAP + off)


def call(fn, defaults, kw):
    assert set(kw) <= set(defaults), kw
    a = dict(defaults, **kw)
    return fn(*a.values())


PROLOGUE = dict(xq=P(0), xk=P(1), xv=P(2), a=P(3), b=P(4), w=P(5), bias=P(6), parent=P(7), n=P(8),
                B=4, N=8, H=2, D=D, dt=BF16, state=P(9), eps=1e-6, q=P(10), k=P(11), v=P(12),
                la=P(13), beta=P(14), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), BAD_DTYPE),
    (dict(B=-1), BAD_SHAPE), (dict(N=0), BAD_SHAPE), (dict(N=65), BAD_SHAPE),
    (dict(H=0), BAD_SHAPE), (dict(H=65537), BAD_SHAPE), (dict(D=64), BAD_SHAPE),
    (dict(B=1 << 30, H=4), BAD_SHAPE), (dict(B=(1 << 31) - 1, N=64, H=1), BAD_SHAPE),
    (dict(eps=-1.0), BAD_SHAPE), (dict(eps=float("nan")), BAD_SHAPE), (dict(eps=float("inf")), BAD_SHAPE),
    (dict(xq=None), NULL_ARG), (dict(b=None), NULL_ARG), (dict(w=None), NULL_ARG),
    (dict(beta=None), NULL_ARG), (dict(la=None), NULL_ARG),
    (dict(xk=P(1, 8)), MISALIGNED), (dict(state=P(9, 2)), MISALIGNED), (dict(b=P(4, 1)), MISALIGNED),
    (dict(parent=P(7, 2)), MISALIGNED), (dict(n=P(8, 1)), MISALIGNED), (dict(bias=P(6, 4)), MISALIGNED),
    (dict(q=P(0)), ALIAS), (dict(k=P(9)), ALIAS), (dict(v=P(10)), ALIAS), (dict(beta=P(4)), ALIAS),
    (dict(la=P(7)), ALIAS), (dict(beta=P(8)), ALIAS), (dict(q=P(0, 4 * 8 * 2 * D * 2 - 16)), ALIAS),
    (dict(B=0, xq=None, q=None), OK),
])
def test_tree_prologue_refusals(L, kw, code):
    assert call(L.kda_tree_prologue, PROLOGUE, kw) == code


DECODE = dict(q=P(0), k=P(1), v=P(2), la=P(3), beta=P(4), S=P(5), parent=P(6), n=P(7), B=4, N=8,
              H=2, Dk=D, Dv=D, dt=BF16, o=P(8), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), BAD_DTYPE),
    (dict(B=-1), BAD_SHAPE), (dict(N=0), BAD_SHAPE), (dict(N=65), BAD_SHAPE), (dict(H=0), BAD_SHAPE),
    (dict(Dk=64), BAD_SHAPE), (dict(Dv=256), BAD_SHAPE), (dict(B=1 << 30, H=4), BAD_SHAPE),
    (dict(q=None), NULL_ARG), (dict(S=None), NULL_ARG), (dict(o=None), NULL_ARG), (dict(beta=None), NULL_ARG),
    (dict(S=P(5, 8)), MISALIGNED), (dict(o=P(8, 2)), MISALIGNED), (dict(beta=P(4, 1)), MISALIGNED),
    (dict(parent=P(6, 2)), MISALIGNED), (dict(n=P(7, 2)), MISALIGNED),
    (dict(o=P(0)), ALIAS), (dict(o=P(5)), ALIAS), (dict(o=P(6)), ALIAS), (dict(o=P(7)), ALIAS),
    (dict(B=0, q=None, S=None, o=None), OK),
])
def test_tree_decode_refusals(L, kw, code):
    assert call(L.kda_tree_decode, DECODE, kw) == code


ACCEPT = dict(p=P(0), q=P(1), tokens=P(2), parent=P(3), n=P(4), u=P(5), B=4, N=8, V=1000, dt=F32,
              path=P(6), m=P(7), next=P(8), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), BAD_DTYPE),
    (dict(B=-1), BAD_SHAPE), (dict(N=0), BAD_SHAPE), (dict(N=65), BAD_SHAPE), (dict(V=0), BAD_SHAPE),
    (dict(V=(1 << 22) + 1), BAD_SHAPE),
    (dict(p=None), NULL_ARG), (dict(tokens=None), NULL_ARG), (dict(u=None), NULL_ARG),
    (dict(path=None), NULL_ARG), (dict(m=None), NULL_ARG), (dict(next=None), NULL_ARG),
    (dict(p=P(0, 4)), MISALIGNED), (dict(q=P(1, 8)), MISALIGNED), (dict(u=P(5, 2)), MISALIGNED),
    (dict(tokens=P(2, 1)), MISALIGNED), (dict(next=P(8, 2)), MISALIGNED),
    (dict(path=P(0)), ALIAS), (dict(path=P(2)), ALIAS), (dict(m=P(6)), ALIAS), (dict(next=P(7)), ALIAS),
    (dict(next=P(5)), ALIAS), (dict(m=P(4)), ALIAS), (dict(path=P(1, 16)), ALIAS),
    (dict(B=0, p=None, tokens=None), OK),
])
def test_tree_accept_refusals(L, kw, code):
    assert call(L.kda_tree_accept, ACCEPT, kw) == code


COMMIT = dict(k=P(0), v=P(1), la=P(2), beta=P(3), S=P(4), path=P(5), n=P(6), B=4, N=8, P=6, H=2,
              Dk=D, Dv=D, dt=BF16, xq=P(7), xk=P(8), xv=P(9), state=P(10), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), BAD_DTYPE),
    (dict(B=-1), BAD_SHAPE), (dict(N=0), BAD_SHAPE), (dict(P=0), BAD_SHAPE), (dict(P=(1 << 24) + 1), BAD_SHAPE),
    (dict(H=0), BAD_SHAPE), (dict(Dk=32), BAD_SHAPE), (dict(Dv=64), BAD_SHAPE), (dict(B=1 << 30, H=4), BAD_SHAPE),
    (dict(k=None), NULL_ARG), (dict(S=None), NULL_ARG), (dict(path=None), NULL_ARG), (dict(xk=None), NULL_ARG),
    (dict(S=P(4, 4)), MISALIGNED), (dict(path=P(5, 2)), MISALIGNED), (dict(state=P(10, 8)), MISALIGNED),
    (dict(xv=P(9, 2)), MISALIGNED), (dict(beta=P(3, 1)), MISALIGNED), (dict(n=P(6, 3)), MISALIGNED),
    (dict(S=P(0)), ALIAS), (dict(S=P(5)), ALIAS), (dict(state=P(7)), ALIAS), (dict(state=P(4)), ALIAS),
    (dict(S=P(6)), ALIAS), (dict(state=P(3)), ALIAS),
    (dict(B=0, k=None, S=None, path=None), OK),
    # without a history its inputs are not looked at
    (dict(state=None, xq=P(4, 2), xk=None, xv=None, B=0), OK),
])
def test_tree_commit_refusals(L, kw, code):
    assert call(L.kda_tree_commit, COMMIT, kw) == code


def meta(*shape, dtype=torch.float32):
    """A tensor without memory: its shape and type are checked before its place."""
    return torch.empty(shape, dtype=dtype)


def test_binding_refuses_what_is_not_on_a_gpu():
    x = meta(2, 4, 3, 128)
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_tree_decode(x, x, x, x, meta(2, 4, 3), meta(2, 3, 128, 128))
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_tree_accept(meta(2, 4, 9), None, meta(2, 4, dtype=torch.int32), meta(2, 4))
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_tree_commit(x, x, x, meta(2, 4, 3), meta(2, 3, 128, 128), meta(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="ROCm device"):
        kda.kda_tree_prologue(x, x, x, x, meta(2, 4, 3), meta(3, 3, 128, 4), meta(3, 128))


def test_binding_names_what_is_missing_or_misshapen():
    x = meta(2, 4, 3, 128)
    with pytest.raises(TypeError, match="S is required"):
        kda.kda_tree_decode(x, x, x, x, meta(2, 4, 3), None)
    with pytest.raises(ValueError, match="4 dimensions"):
        kda.kda_tree_decode(meta(4, 3, 128), x, x, x, meta(2, 4, 3), meta(2, 3, 128, 128))
    with pytest.raises(TypeError, match="p must be a torch.Tensor"):
        kda.kda_tree_accept([1], None, meta(2, 4), meta(2, 4))


@pytest.mark.parametrize("fn,defaults,most,rest", [
    ("kda_tree_prologue", PROLOGUE, (1 << 23) - 1, dict(N=1, H=1)),
    ("kda_tree_decode", DECODE, (1 << 23) - 1, dict(N=1, H=1)),
    ("kda_tree_commit", COMMIT, (1 << 23) - 1, dict(N=1, P=1, H=1)),
    ("kda_tree_accept", ACCEPT, (1 << 22) - 1, dict(N=1, V=1, path=P(0))),
])
def test_batches_larger_than_a_launch_are_refused(L, fn, defaults, most, rest):
    """One more sequence than a launch holds is a bad shape; the most that it
    holds gets past the shapes (to the alias check of overlapping buffers)."""
    alias = dict(rest, **({"path": P(0)} if fn == "kda_tree_accept" else
                          {"S": P(0)} if fn == "kda_tree_commit" else
                          {"o": P(0)} if fn == "kda_tree_decode" else {"q": P(0)}))
    assert call(getattr(L, fn), defaults, dict(alias, B=most + 1)) == BAD_SHAPE
    assert call(getattr(L, fn), defaults, dict(alias, B=most)) == ALIAS
