"""kda_tree_prologue against the fp64 oracle (oracle/tree.py: each node's path
through the layer prologue as a sequence of its own) and, for a chain,
bit for bit against kda_prologue.

Tolerance, normwise: half a step of the output type (bf16 2^-8) plus, for the
fp32 arithmetic, 1e-5: the 4-term convolution, exp, reciprocal and square
root are good to a few 2^-24 each, |input of a sigmoid| * 2^-24 < 1e-6 more.
"""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import tree as otree
from gpu_util import case, check, need_gpu, np_
from tree_util import SENTINEL, i32, random_trees

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}
NAMES = ("q", "k", "v", "log_alpha", "beta")
IN = ("xq", "xk", "xv", "a_raw", "b_raw")


def _inputs(B, N, H, dtype, seed, history):
    d = kda_inputs.layer_inputs(B * N, H, dtype=dtype, device="cuda", seed=seed, lengths=[N] * B,
                                conv_state=history)
    x = [d[n].view(B, N, *d[n].shape[1:]) for n in IN]
    return d, x


@pytest.mark.parametrize("dtype,B,N,H,shape,counts,history", [
    ("bf16", 3, 1, 3, "tree", None, True),
    ("f32", 2, 1, 1, "tree", [1, 0], False),
    ("bf16", 3, 8, 4, "tree", [8, 3, 0], True),
    ("f32", 3, 9, 5, "forest", [9, 8, 1], True),        # a node past a wave's 8
    ("bf16", 2, 17, 2, "star", None, False),
    ("f32", 2, 30, 2, "chain", [30, 17], True),
    ("bf16", 2, 64, 3, "forest", [64, 70], True),       # counts are clamped
    ("f32", 1, 64, 2, "tree", None, False),
])
def test_tree_prologue_matches_oracle(dtype, B, N, H, shape, counts, history):
    kda = need_gpu()
    case(f"tree_prologue {dtype} B={B} N={N} H={H} {shape} counts={counts} history={history}")
    d, x = _inputs(B, N, H, dtype, 70 + N, history)
    par = random_trees(B, N, N, shape)
    out = tuple(torch.full(x[0].shape, SENTINEL, dtype=x[0].dtype, device="cuda") for _ in range(4)) + (
        torch.full((B, N, H), SENTINEL, dtype=x[0].dtype, device="cuda"),)
    before = None if d["conv_state"] is None else d["conv_state"].clone()
    got = kda.kda_tree_prologue(*x, d["conv_w"], d["a_bias"], i32(par), i32(counts),
                                d["conv_state"], out=out)
    torch.cuda.synchronize()
    if before is not None:
        assert torch.equal(before, d["conv_state"])
    for b in range(B):
        n = N if counts is None else min(N, counts[b])
        if n:
            ref = otree.prologue(*[np_(t[b]) for t in x], np_(d["conv_w"]), np_(d["a_bias"]), par[b], n,
                                 None if before is None else np_(before[b]))
            for name, g, r in zip(NAMES, got, ref):
                check(f"{name} of sequence {b}", np_(g[b, :n]), r, TOL[dtype])
        for name, g in zip(NAMES, got):
            assert torch.all(g[b, n:] == SENTINEL), f"{name}: rows past the nodes of sequence {b}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_prologue_of_a_chain_has_the_prologues_bits(dtype):
    kda = need_gpu()
    B, N, H = 5, 13, 3
    case(f"tree_prologue chain vs prologue {dtype}")
    d, x = _inputs(B, N, H, dtype, 3, True)
    got = kda.kda_tree_prologue(*x, d["conv_w"], d["a_bias"], conv_state=d["conv_state"])
    ref = kda.kda_prologue(*[d[n] for n in IN], d["conv_w"], d["a_bias"], cu_seqlens=d["cu_seqlens"],
                           conv_state=d["conv_state"], store_state=False)
    torch.cuda.synchronize()
    for name, g, r in zip(NAMES, got, ref):
        assert torch.equal(g.reshape(r.shape), r), name


@pytest.mark.parametrize("dtype,B,N,H", [("bf16", 1101, 5, 1), ("f32", 2051, 33, 2), ("bf16", 643, 20, 9)])
def test_tree_prologue_of_large_batches_has_the_bits_of_small_ones(dtype, B, N, H):
    """Workgroups take several sequences each from some thousands of slices
    on: the outputs, and the rows left as they were, are those of the same
    sequences in calls of 100."""
    kda = need_gpu()
    case(f"tree_prologue in groups {dtype} B={B} N={N} H={H}")
    d, x = _inputs(B, N, H, dtype, 5, True)
    par = i32(random_trees(B, N, 8, "forest"))
    counts = i32(np.random.default_rng(1).integers(-1, N + 2, size=B))
    fill = lambda n: tuple(torch.full((n,) + x[j].shape[1:], SENTINEL, dtype=x[0].dtype, device="cuda")
                           for j in range(5))
    got = kda.kda_tree_prologue(*x, d["conv_w"], d["a_bias"], par, counts, d["conv_state"], out=fill(B))
    for b in range(0, B, 100):
        s = slice(b, min(b + 100, B))
        ref = kda.kda_tree_prologue(*[t[s].contiguous() for t in x], d["conv_w"], d["a_bias"], par[s].contiguous(),
                                    counts[s].contiguous(), d["conv_state"][s].contiguous(), out=fill(s.stop - b))
        for name, g, r in zip(NAMES, got, ref):
            assert torch.equal(g[s], r), (name, b)
