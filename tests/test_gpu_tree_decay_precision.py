"""kda_tree_decode's decays: fp32 outputs of nodes below strong decay, against
the fp64 oracle, to what 32-bit factors leave.

Tolerance, normwise, in units of 2^-24.  A coupling <q_i e^{G_i}, k_j e^{-G_j}>
has two exponentials good to two ulp (4 each), two products (1 each) and two G
off by at most 2^-23 (2 each): 14.  Three sums of up to 144 products of the
values' own size follow each other (held, solve, output), each rounding by
sqrt(144): 36.  Together 50 * 2^-24 = 3.0e-6.  A running sum of log alpha held
in one float is off by half an ulp of its size, 32 units at |G| of 64 and 128
at 256, on its own.
"""
import pytest
import torch

from oracle import tree as otree
from gpu_util import case, check, need_gpu, np_
from tree_util import i32, node_inputs, random_trees

pytestmark = pytest.mark.gpu

TOL = 50 * 2.0 ** -24


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("shape", ["chain", "comb"])
@pytest.mark.parametrize("N", [5, 8, 14, 16, 24, 32, 48, 64])
def test_running_decay_is_not_held_in_one_float(N, shape, seed):
    """A spine of log alpha -4.75 on average, then nodes that keep all but a
    bit: four in a row (chain), or a chain of them on each of three nodes of
    the spine (comb)."""
    kda = need_gpu()
    case(f"tree_decode below strong decay, N={N} {shape} seed={seed}")
    w = node_inputs(2, N, 2, "f32", seed=seed)
    g = torch.Generator(device="cuda").manual_seed(50 + seed)
    w["log_alpha"].uniform_(-5.0, -4.5, generator=g)
    par = random_trees(2, N, seed, "chain")
    keep = N - 4 if shape == "chain" else N // 2
    w["log_alpha"][:, keep:].uniform_(-2e-3, 0.0, generator=g)
    if shape == "comb":
        for i in range(keep, N):
            par[:, i] = i - 3 if i - 3 >= keep else (keep - 1) * (i - keep + 1) // 3
    o = kda.kda_tree_decode(*[w[x] for x in ("q", "k", "v", "log_alpha", "beta")], w["S"], i32(par))
    torch.cuda.synchronize()
    for b in range(2):
        ref = otree.decode(*[np_(w[x][b]) for x in ("q", "k", "v", "log_alpha", "beta", "S")], par[b], N)
        check(f"o of sequence {b}", np_(o[b]), ref, TOL)
