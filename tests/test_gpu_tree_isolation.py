"""What a NaN or infinity of one node reaches in kda_tree_decode, at every
size's code (up to 8 nodes, 16, 32, 48, 64) and under mild decay and decay at
the bound, where the couplings are formed level by level; and the decay bound
at the smallest sizes.

k, log alpha, beta: whole rows of the node and of its descendants; v: the one
column of those rows; q: the node's own row alone.

Other rows keep their bits while |G| stays below 64.  Beyond, the levels that
a tile's couplings are summed over are counted from the tile's greatest G,
which the node's own log alpha (taken as 0) may move: there the other rows
agree to the output's rounding, two halves of a step (eps), and 50 * 2^-24 for
the fp32 evaluation of each (two exponentials, two products and two G of a
coupling, 14 units of 2^-24; three sums of up to 144 products, 36).
"""
import numpy as np
import pytest
import torch

from oracle import tree as otree
from gpu_util import case, need_gpu, nerr, np_
from tree_util import SENTINEL, i32, node_inputs, random_trees

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
COLUMN = 77


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("strong", [False, True], ids=["mild", "bound"])
@pytest.mark.parametrize("N", [2, 5, 8, 12, 16, 20, 33, 40, 64])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "beta"])
def test_non_finite_inputs_reach_descendants_only(dtype, strong, N, name):
    kda = need_gpu()
    case(f"tree_decode, non-finite {name}, {dtype} N={N} {'decay at the bound' if strong else 'mild decay'}")
    B, H = 2, 2
    w = node_inputs(B, N, H, dtype, seed=8 + N)
    if strong:
        w["log_alpha"].fill_(-5.0)
        # two chains side by side, the second from the cached state
        par = np.tile(np.array([i - 1 if i != N // 4 else -1 for i in range(N)], dtype=np.int32), (B, 1))
    else:
        par = random_trees(B, N, 3, "tree")
        if N > 4:
            par[:, N // 2] = -1
    a = [w[x] for x in ("q", "k", "v", "log_alpha", "beta")]
    n = [N, max(N - 2, 1)]
    args = (w["S"], i32(par), i32(n))
    bits = not strong or name not in ("log_alpha",) or N <= 8
    o1 = kda.kda_tree_decode(*a, *args, o=torch.full_like(w["v"], SENTINEL))
    ways = otree.paths(par[0], N)
    tol = torch.finfo(DT[dtype]).eps * (dtype == "bf16") + 2 * 50 * 2.0 ** -24
    w[name][1, n[1]:] = float("nan")   # (rows past the nodes are not read)
    for node, value in ((N - 1, float("inf")), (N // 2, float("nan")), (0, float("-inf"))):
        old = w[name][0, node, 1].clone()
        if name == "beta":
            w[name][0, node, 1] = value
        else:
            w[name][0, node, 1, COLUMN] = value
        o2 = kda.kda_tree_decode(*a, *args, o=torch.full_like(w["v"], SENTINEL))
        torch.cuda.synchronize()
        assert torch.equal(o1[1], o2[1]) and torch.equal(o1[0, :, 0], o2[0, :, 0])
        other = torch.ones((N, 128), dtype=torch.bool, device="cuda")
        for i in range(N):
            if not (i == node if name == "q" else node in ways[i]):
                continue
            if name == "v":
                other[i, COLUMN] = False
                assert torch.isnan(o2[0, i, 1, COLUMN]), i
            else:
                other[i] = False
                bad = ~torch.isfinite(o2[0, i, 1]) if name == "q" else torch.isnan(o2[0, i, 1])
                assert bad.all(), i
        x, y = o1[0, :, 1][other], o2[0, :, 1][other]
        assert torch.isfinite(y).all()
        if bits:
            assert torch.equal(x, y), node
        else:
            assert nerr(np_(y), np_(x)) <= tol, node
        w[name][0, node, 1] = old


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["chain", "star", "forest"])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9])
def test_the_decay_bound_at_small_sizes(dtype, shape, N):
    """log alpha = -5 everywhere: |G| of 40 at 8 nodes in a chain.

    Tolerance: half a step of the output's type, and 50 * 2^-24 of the terms
    that are summed before it.  Of the terms, not of their sum: with one node
    the output is S^T (q e^-5) + <q, k> u, and where <q, k> = 7e-4 is what is
    left of terms that add up to 0.62 in size, an error of 2^-24 of these is
    900 * 2^-24 of the output (kda_decode_multi's 3e-6 there).  The terms are
    at most sum |q k| |u| with |u| <= max |v| + |S^T k|, and sum |q| |S| e^-5."""
    kda = need_gpu()
    case(f"tree_decode at the decay bound, {dtype} N={N} {shape}")
    w = node_inputs(3, N, 2, dtype, seed=60 + N)
    w["log_alpha"].fill_(-5.0)
    par = random_trees(3, N, N, shape)
    n = [N, max(N - 1, 1), 1]
    o = kda.kda_tree_decode(*[w[x] for x in ("q", "k", "v", "log_alpha", "beta")], w["S"], i32(par), i32(n),
                            o=torch.full_like(w["v"], SENTINEL))
    torch.cuda.synchronize()
    half = torch.finfo(DT[dtype]).eps / 2 * (dtype == "bf16")
    for b in range(3):
        d = {x: np_(w[x][b]).astype(np.float64) for x in ("q", "k", "v", "log_alpha", "beta", "S")}
        ref = otree.decode(*d.values(), par[b], n[b])
        q, k, S = np.abs(d["q"][:n[b]]), np.abs(d["k"][:n[b]]), np.abs(d["S"]).max()
        u = np.abs(d["v"]).max() + k.sum(-1).max() * S * np.exp(-5.0)
        terms = (q * k).sum(-1).max() * u + q.sum(-1).max() * S * np.exp(-5.0)
        err = np.abs(np_(o[b, :n[b]]) - ref).max()
        bound = half * np.abs(ref).max() + 50 * 2.0 ** -24 * terms
        print(f"    sequence {b}: off by {err:.2e} (bound {bound:.2e}), outputs up to {np.abs(ref).max():.2e}", flush=True)
        assert err <= bound
        assert (o[b, n[b]:] == SENTINEL).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [12, 20, 40, 64])
def test_the_lowest_log_alpha_reaches_descendants_only(dtype, N):
    """A finite log alpha far outside its contract, the type's lowest value:
    like an infinity it stays with its node and the nodes below it."""
    kda = need_gpu()
    case(f"tree_decode, lowest log alpha, {dtype} N={N}")
    w = node_inputs(1, N, 2, dtype, seed=9 + N)
    par = random_trees(1, N, 4, "tree")
    a = [w[x] for x in ("q", "k", "v", "log_alpha", "beta")]
    o1 = kda.kda_tree_decode(*a, w["S"], i32(par))
    tol = torch.finfo(DT[dtype]).eps * (dtype == "bf16") + 2 * 50 * 2.0 ** -24   # (as above)
    ways = otree.paths(par[0], N)
    for node in (N // 2, 3):
        old = w["log_alpha"][0, node, 1].clone()
        w["log_alpha"][0, node, 1, COLUMN] = torch.finfo(DT[dtype]).min
        o2 = kda.kda_tree_decode(*a, w["S"], i32(par))
        torch.cuda.synchronize()
        other = torch.tensor([node not in ways[i] for i in range(N)], device="cuda")
        assert other.sum() >= 3 and torch.equal(o1[0, :, 0], o2[0, :, 0])
        assert torch.isfinite(o2[0, other, 1]).all()
        assert nerr(np_(o2[0, other, 1]), np_(o1[0, other, 1])) <= tol, node
        w["log_alpha"][0, node, 1] = old
