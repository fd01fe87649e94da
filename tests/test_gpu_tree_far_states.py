"""kda_tree_commit on states past 2^32 elements: what the last sequences'
states and histories become, against the fp64 oracle and against a copy kept
from before (that they moved at all)."""
import numpy as np
import pytest
import torch

from oracle import tree as otree
from gpu_util import case, check, need_gpu, np_
from tree_util import i32

pytestmark = pytest.mark.gpu


def test_states_past_32_bits_move():
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of free memory")
    B, N, H = 2740, 5, 96
    case(f"tree_commit with B={B} N={N} H={H}")
    assert B * H * 128 * 128 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(6)
    # one tensor for every input: its values are fit for k and for log alpha
    x = torch.empty((B, N, H, 128), dtype=torch.bfloat16, device="cuda").uniform_(-0.08, 0.0, generator=g)
    beta = torch.empty((B, N, H), dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.0, generator=g)
    S = torch.empty((B, H, 128, 128), device="cuda").uniform_(-1.0, 1.0, generator=g)
    hist = torch.zeros((B, 3, 3, H, 128), dtype=torch.bfloat16, device="cuda")
    path = i32(np.tile(np.array([0, 2, 3, 4], dtype=np.int32), (B, 1)))
    m = torch.full((B,), 4, dtype=torch.int32, device="cuda")
    m[B - 2] = 0                                   # the last sequence but one keeps what it has
    some = (0, B // 2, B - 2, B - 1)
    before = {b: S[b].clone() for b in some}
    assert (B - 1) * H * 128 * 128 > 2 ** 32 - 2 ** 22
    kda.kda_tree_commit(x, x, x, beta, S, path, m, conv=(x, x, x, hist))
    torch.cuda.synchronize()
    for b in some:
        if b == B - 2:
            assert torch.equal(S[b], before[b]) and (hist[b] == 0).all()
            continue
        heads = slice(0, H, 19)
        moved = (S[b] != before[b]).float().mean().item()
        assert moved > 0.99, (b, moved)
        v = np_(x[b][:, heads])
        ref, _ = otree.commit(v, v, v, np_(beta[b][:, heads]), np_(before[b][heads]), [0, 2, 3, 4])
        # 31 * 2^-24: exponentials, products and sums of 32-bit factors, as for shorter batches
        check(f"S of sequence {b}", np_(S[b][heads]), ref, 31 * 2.0 ** -24)
        assert torch.equal(hist[b], x[b, 2:5].expand(3, 3, H, 128))
