"""kda_tree_commit's decays: the state of paths whose tokens decay strongly,
against the fp64 oracle, to what 32-bit factors leave.

Tolerance, normwise, in units of 2^-24.  An exponential is good to two ulp
(4), its product with k to half of one (1): a coupling has two of each (10), a
token's row in the new state one (5).  Sums of 128 and 16 products of the
values' own size round by sqrt(144) (12), the state's update of 16 by 4.
Together 31 * 2^-24 = 1.9e-6.  A running sum of log alpha held in one float is
off by half an ulp of its size, 32 such units at |G| of 64, on its own.
"""
import numpy as np
import pytest
import torch

from oracle import tree as otree
from gpu_util import case, check, need_gpu, np_
from tree_util import i32, node_inputs

pytestmark = pytest.mark.gpu

TOL = 31 * 2.0 ** -24


def _strong_then_hardly(x, g):
    """Twelve tokens of -4.75 on average, then four that keep all but a bit."""
    x.copy_(torch.empty(x.shape, device="cuda").uniform_(-5.0, -4.5, generator=g))
    x[:, -4:] = torch.empty(x[:, -4:].shape, device="cuda").uniform_(-2e-3, 0.0, generator=g).to(x.dtype)


def _of_every_size(x, g):
    x.copy_(torch.empty(x.shape, device="cuda").uniform_(-5.0, 0.0, generator=g))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", [0, 1, 2])
@pytest.mark.parametrize("N,decay", [(16, _strong_then_hardly), (48, _strong_then_hardly), (16, _of_every_size),
                                     (64, _of_every_size)])
def test_running_decay_is_not_held_in_one_float(dtype, seed, N, decay):
    kda = need_gpu()
    case(f"tree_commit of {N} tokens, {decay.__name__} {dtype} seed={seed}")
    w = node_inputs(2, N, 2, dtype, seed=seed)
    decay(w["log_alpha"], torch.Generator(device="cuda").manual_seed(50 + seed))
    path = np.tile(np.arange(N, dtype=np.int32), (2, 1))
    S = w["S"].clone()
    kda.kda_tree_commit(w["k"], w["v"], w["log_alpha"], w["beta"], S, i32(path))
    torch.cuda.synchronize()
    for b in range(2):
        ref, _ = otree.commit(*[np_(w[t][b]) for t in ("k", "v", "log_alpha", "beta", "S")], path[b])
        check(f"S of sequence {b}", np_(S[b]), ref, TOL)
