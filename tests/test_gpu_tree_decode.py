"""kda_tree_decode and kda_tree_commit against the fp64 oracle (oracle/tree.py:
every node's path run token by token as a sequence of its own).

Tolerances, normwise (max error / max value).  Output rounding: half a step,
2^-8 for bf16.  Before it, in fp32: a 128-term sum is off by at most 128 *
2^-24 = 7.6e-6 of its terms' size, and a decay e^{G} by (|G| + the log alpha
sum's terms) * 2^-24, at |G| <= 80 and 64 terms 8.6e-6, on both factors of a
pair; bf16 rows held as two bf16 leave 2^-17 per product.  Three such sums
follow each other (held, solve, output): 1e-4 covers them, and is the
library's fp32 tolerance.
"""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import tree as otree
from gpu_util import case, check, need_gpu, np_
from tree_util import SENTINEL, i32, node_inputs, random_trees

pytestmark = pytest.mark.gpu

TOL_O = {"f32": 1e-4, "bf16": 2.0 ** -8 + 1e-4}
TOL_S = 1e-4   # states are fp32 whatever the inputs


DECODE = [
    # dtype, B, N, H, shape, n_node, decay mean
    ("bf16", 3, 1, 2, "tree", None, -2.0),              # the pending token alone
    ("f32", 3, 1, 1, "tree", [1, 0, 1], -2.0),
    ("bf16", 4, 8, 3, "chain", None, -2.0),
    ("f32", 4, 8, 3, "tree", [8, 0, 5, 1], -2.0),
    ("bf16", 3, 15, 2, "star", [15, 14, 2], -2.0),
    ("f32", 3, 16, 2, "forest", None, -2.0),
    ("bf16", 3, 16, 2, "chain", None, 0.0),
    ("bf16", 3, 17, 2, "tree", [17, 16, 3], -2.0),      # a node past a tile of 16
    ("f32", 2, 31, 3, "tree", None, 0.0),
    ("f32", 2, 33, 1, "forest", [33, 32], -2.0),
    ("bf16", 2, 48, 2, "tree", [48, 7], -2.0),
    ("f32", 2, 49, 2, "star", None, -2.0),
    ("bf16", 2, 63, 1, "forest", [63, 40], -1.0),
    ("bf16", 2, 64, 2, "tree", None, -2.0),
    ("f32", 2, 64, 2, "chain", None, -2.0),             # 64 levels
    ("bf16", 2, 64, 1, "chain", None, -4.0),
]


def _check_decode(kda, w, par, counts, dtype, none_parent=False, o=None):
    B, N, H = w["beta"].shape
    S0 = w["S"].clone()
    o = torch.full((B, N, H, 128), SENTINEL, dtype=w["q"].dtype, device="cuda")
    kda.kda_tree_decode(w["q"], w["k"], w["v"], w["log_alpha"], w["beta"], w["S"],
                        None if none_parent else i32(par), i32(counts), o=o)
    torch.cuda.synchronize()
    assert torch.equal(w["S"], S0), "the cached state moved"
    got = np_(o)
    for b in range(B):
        n = N if counts is None else max(0, min(N, counts[b]))
        if n:
            ref = otree.decode(*[np_(w[x][b]) for x in ("q", "k", "v", "log_alpha", "beta", "S")],
                               par[b], n)
            check(f"o of sequence {b} ({n} nodes)", got[b, :n], ref, TOL_O[dtype])
        assert np.all(got[b, n:] == SENTINEL), f"rows past the nodes of sequence {b} written"
    return o


@pytest.mark.parametrize("dtype,B,N,H,shape,counts,mu", DECODE)
def test_tree_decode_matches_oracle(dtype, B, N, H, shape, counts, mu):
    kda = need_gpu()
    case(f"tree_decode {dtype} B={B} N={N} H={H} {shape} counts={counts} mu={mu}")
    w = node_inputs(B, N, H, dtype, seed=900 + N + B, decay_mu=mu)
    _check_decode(kda, w, random_trees(B, N, N + H, shape), counts, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [12, 13, 16, 40, 64])
def test_tree_decode_at_the_decay_bound(dtype, N):
    """log alpha = -5 everywhere on a chain: |G| reaches 60 at 12 nodes (the
    factored Gram entries), 65 at 13 (levels of decay), 320 at 64."""
    kda = need_gpu()
    case(f"tree_decode at the decay bound {dtype} N={N}")
    w = node_inputs(2, N, 2, dtype, seed=77 + N)
    w["log_alpha"].fill_(-5.0)
    _check_decode(kda, w, random_trees(2, N, 1, "chain"), None, dtype, none_parent=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_decode_mixed_decay(dtype):
    """One branch decays to nothing while another keeps everything: the
    shared range check must not cost the second its precision."""
    kda = need_gpu()
    N = 40
    case(f"tree_decode mixed decay {dtype}")
    w = node_inputs(2, N, 2, dtype, seed=31)
    par = np.tile(np.array([-1, 0] + list(range(0, N - 2)), dtype=np.int32), (2, 1))  # two combs
    w["log_alpha"].fill_(-0.01)
    w["log_alpha"][:, 1::2] = -5.0
    w["log_alpha"][1, :, :, 64:] = 0.0
    _check_decode(kda, w, par, [N, 33], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,shape", [(16, "chain"), (30, "chain"), (33, "forest"), (48, "chain"), (64, "chain"),
                                     (64, "forest"), (64, "comb")])
def test_tree_decode_levels_of_decay(dtype, N, shape):
    """Decays of 0, -0.01 and -5 mixed over nodes and channels, so that a tile
    holds nodes of every depth of decay (to -320) beside each other: pairs
    near each other far below keep their entries' precision."""
    kda = need_gpu()
    case(f"tree_decode levels of decay {dtype} N={N} {shape}")
    w = node_inputs(3, N, 2, dtype, seed=300 + N)
    g = torch.Generator(device="cuda").manual_seed(N)
    pick = torch.randint(0, 3, w["log_alpha"].shape, generator=g, device="cuda")
    w["log_alpha"].copy_(torch.tensor([0.0, -0.01, -5.0], device="cuda")[pick])
    w["log_alpha"][1, :, :, :40] = -5.0
    if shape == "comb":   # a long spine; on it and on the cached state, short branches in turn
        par = np.full((3, N), -1, dtype=np.int32)
        for i in range(1, N):
            par[:, i] = i - 1 if i < N // 2 else ([N // 2 - 1, -1, i - 2][i % 3])
    else:
        par = random_trees(3, N, N, shape)
    _check_decode(kda, w, par, [N, N, N - 3], dtype)


def test_tree_decode_of_a_chain_is_the_chain_verify():
    """parent = None gives kda_decode_multi's verify pass, to rounding."""
    kda = need_gpu()
    B, K, H = 16, 7, 4
    case("tree_decode chain vs decode_multi")
    w = node_inputs(B, K, H, "f32", seed=5)
    args = [w[x] for x in ("q", "k", "v", "log_alpha", "beta")]
    o1 = kda.kda_tree_decode(*args, w["S"])
    o2 = kda.kda_decode_multi(*args, w["S"], update_state=False)
    torch.cuda.synchronize()
    check("o", np_(o1), np_(o2).astype(np.float64), 1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "beta"])
def test_tree_decode_siblings_do_not_see_each_other(dtype, name):
    """A NaN or infinity of a node makes NaN of the node's outputs and of its
    descendants' (q: the node's alone; v: one column); every other row keeps
    its bits."""
    kda = need_gpu()
    B, N, H = 2, 40, 2
    case(f"tree_decode non-finite {name} in one branch, {dtype}")
    w = node_inputs(B, N, H, dtype, seed=8)
    par = random_trees(B, N, 3, "tree")
    a = [w[x] for x in ("q", "k", "v", "log_alpha", "beta")]
    n = [N, N - 5]
    args = (w["S"], i32(par), i32(n))
    o1 = kda.kda_tree_decode(*a, *args, o=torch.zeros_like(w["v"]))
    ways = otree.paths(par[0], N)
    for node, value in ((5, float("nan")), (37, float("inf")), (0, float("-inf"))):
        old = w[name][0, node, 1].clone()
        w[name][1, N - 5:] = float("nan")          # (rows past the nodes are not read)
        if name == "beta":
            w[name][0, node, 1] = value
        else:
            w[name][0, node, 1, 77] = value
        o2 = kda.kda_tree_decode(*a, *args, o=torch.zeros_like(w["v"]))
        torch.cuda.synchronize()
        assert torch.equal(o1[1], o2[1]) and torch.equal(o1[0, :, 0], o2[0, :, 0])
        for i in range(N):
            hit = i == node if name == "q" else node in ways[i]
            if not hit:
                assert torch.equal(o1[0, i, 1], o2[0, i, 1]), i
            elif name == "v":
                assert torch.isnan(o2[0, i, 1, 77]), i
                keep = torch.arange(128, device="cuda") != 77
                assert torch.equal(o1[0, i, 1][keep], o2[0, i, 1][keep]), i
            else:
                assert not torch.isfinite(o2[0, i, 1]).any(), i
        w[name][0, node, 1] = old


COMMIT = [
    # dtype, B, N, P, H, n_path, history, decay mean
    ("bf16", 4, 8, 8, 3, [8, 0, 1, 3], True, -2.0),
    ("f32", 4, 8, 4, 3, [4, 2, 0, 1], True, -2.0),
    ("bf16", 2, 1, 1, 1, None, True, -2.0),
    ("f32", 3, 20, 16, 2, [16, 15, 9], True, 0.0),
    ("bf16", 3, 20, 17, 2, [17, 16, -4], True, -2.0),     # one token past a block of 16
    ("f32", 2, 64, 64, 1, [64, 99], False, -4.0),         # counts are clamped
    ("f32", 2, 100, 70, 1, [70, 65], True, -2.0),         # path longer than a wavefront
]


@pytest.mark.parametrize("dtype,B,N,P,H,n_path,conv,mu", COMMIT)
def test_tree_commit_matches_oracle(dtype, B, N, P, H, n_path, conv, mu):
    kda = need_gpu()
    case(f"tree_commit {dtype} B={B} N={N} P={P} H={H} n_path={n_path} history={conv} mu={mu}")
    w = node_inputs(B, N, H, dtype, seed=40 + N + P, decay_mu=mu)
    rng = np.random.default_rng(N * P)
    path = np.stack([np.sort(rng.permutation(N)[:P]) for _ in range(B)]).astype(np.int32)
    x = [torch.randn_like(w["k"]) for _ in range(3)]
    hist = torch.randn((B, 3, 3, H, 128), device="cuda").to(w["k"].dtype)
    S, h1 = w["S"].clone(), hist.clone()
    got = kda.kda_tree_commit(w["k"], w["v"], w["log_alpha"], w["beta"], S, i32(path),
                              i32(n_path), conv=(*x, h1) if conv else None)
    torch.cuda.synchronize()
    assert got is S
    for b in range(B):
        m = P if n_path is None else max(0, min(P, n_path[b]))
        rS, rh = otree.commit(*[np_(w[t][b]) for t in ("k", "v", "log_alpha", "beta", "S")],
                              path[b, :m], [np_(t[b]) for t in x], np_(hist[b]))
        if m == 0:
            assert torch.equal(S[b], w["S"][b]) and torch.equal(h1[b], hist[b])
            continue
        check(f"S of sequence {b} ({m} tokens)", np_(S[b]), rS, TOL_S)
        if conv:
            assert np.array_equal(np_(h1[b]), rh), f"history of sequence {b}"
    if not conv:
        assert torch.equal(h1, hist)


def test_tree_commit_path_ends_before_what_is_no_node():
    kda = need_gpu()
    B, N, P, H = 4, 6, 6, 2
    case("tree_commit paths with -1 and out-of-range entries, a node twice")
    w = node_inputs(B, N, H, "f32", seed=12)
    path = np.array([[0, 2, -1, 3, 4, 5], [1, 6, 0, 0, 0, 0], [-1, 0, 1, 2, 3, 4],
                     [0, 3, 3, 5, 1 << 30, 0]], dtype=np.int32)
    S = w["S"].clone()
    kda.kda_tree_commit(w["k"], w["v"], w["log_alpha"], w["beta"], S, i32(path))
    torch.cuda.synchronize()
    for b, way in enumerate(([0, 2], [1], [], [0, 3, 3, 5])):
        rS, _ = otree.commit(*[np_(w[t][b]) for t in ("k", "v", "log_alpha", "beta", "S")], way)
        check(f"S of sequence {b}", np_(S[b]), rS, TOL_S)
    assert torch.equal(S[2], w["S"][2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_commit_at_the_decay_bound(dtype):
    kda = need_gpu()
    B, N, H = 2, 40, 2
    case(f"tree_commit at the decay bound {dtype}")
    w = node_inputs(B, N, H, dtype, seed=13)
    w["log_alpha"].fill_(-5.0)
    path = np.tile(np.arange(N, dtype=np.int32), (B, 1))
    S = w["S"].clone()
    kda.kda_tree_commit(w["k"], w["v"], w["log_alpha"], w["beta"], S, i32(path))
    torch.cuda.synchronize()
    for b in range(B):
        rS, _ = otree.commit(*[np_(w[t][b]) for t in ("k", "v", "log_alpha", "beta", "S")], path[b])
        check(f"S of sequence {b}", np_(S[b]), rS, TOL_S)


def test_tree_commit_of_a_chain_is_the_replay():
    """Along a chain: kda_decode_multi's replay, to rounding."""
    kda = need_gpu()
    B, K, H = 8, 7, 4
    case("tree_commit chain vs decode_multi replay")
    w = node_inputs(B, K, H, "bf16", seed=14)
    n = i32([7, 0, 1, 2, 3, 4, 5, 6])
    S1, S2 = w["S"].clone(), w["S"].clone()
    kda.kda_tree_commit(w["k"], w["v"], w["log_alpha"], w["beta"], S1,
                        i32(np.tile(np.arange(K), (B, 1))), n)
    kda.kda_decode_multi(w["q"], w["k"], w["v"], w["log_alpha"], w["beta"], S2, n)
    torch.cuda.synchronize()
    check("S", np_(S1), np_(S2).astype(np.float64), 1e-5)
