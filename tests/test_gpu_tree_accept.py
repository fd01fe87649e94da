"""kda_tree_accept against the rejection walk written on normalised
distributions (oracle/tree.py), and the distribution of what it emits.

All results are whole numbers and have to be equal; both sides decide in
fp64, so a random case whose nearest border is under 1e-12 (in probability;
the sums' rounding is below 1e-13) would be undecidable and none is drawn.
"""
import numpy as np
import pytest
import torch

from oracle import tree as otree
from gpu_util import case, need_gpu, np_
from tree_util import i32, random_trees

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(B, N, V, dtype, seed, par, drafts, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    lt = torch.randn((B, N, V), generator=g) * sharp
    lq = lt + torch.randn((B, N, V), generator=g)
    p = torch.softmax(lt.double(), -1).to(DT[dtype])
    q = torch.softmax(lq.double(), -1)[:, :max(N - 1, 0)].to(DT[dtype]) if drafts else None
    tokens = torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        for i in range(1, N):
            r = int(par[b, i])
            if not 0 <= r < i:
                continue
            w = torch.softmax((lq if drafts else lt)[b, r].double(), -1)
            tokens[b, i] = int(torch.multinomial(w, 1, generator=g))
    u = torch.rand((B, N), generator=g)
    return p, q, tokens, u


def _check(kda, p, q, tokens, u, par, counts, none_parent=False):
    B, N, V = p.shape
    path, m, nxt = kda.kda_tree_accept(p.cuda(), None if q is None else q.cuda(), tokens.cuda(), u.cuda(),
                                       None if none_parent else i32(par), i32(counts))
    torch.cuda.synchronize()
    path, m, nxt = path.cpu().numpy(), m.cpu().numpy(), nxt.cpu().numpy()
    lengths = []
    for b in range(B):
        n = N if counts is None else max(0, min(N, counts[b]))
        way, token, margin = otree.accept(np_(p[b]), None if q is None else np_(q[b]), tokens[b].numpy(),
                                          u[b].numpy(), par[b], n)
        assert margin > 1e-12, "the case has no answer to compare"
        assert path[b].tolist() == way + [-1] * (N - len(way)), b
        assert m[b] == len(way) and nxt[b] == token, (b, m[b], nxt[b], way, token)
        lengths.append(len(way))
    print(f"    accepted {np.mean(lengths):.2f} of {N} nodes on average", flush=True)
    return lengths


@pytest.mark.parametrize("dtype,B,N,V,shape,counts,drafts", [
    ("f32", 5, 1, 1000, "tree", [1, 0, 1, 1, -2], True),     # the pending token alone
    ("f32", 16, 4, 7, "chain", None, True),
    ("f32", 40, 8, 1023, "chain", None, True),               # a vocabulary of less than a tile
    ("bf16", 40, 8, 1024, "chain", None, True),
    ("f32", 20, 8, 1025, "chain", [8, 0, 3, 1] * 5, False),
    ("bf16", 20, 13, 2051, "tree", None, True),
    ("f32", 20, 30, 517, "tree", None, True),
    ("f32", 20, 40, 50, "star", None, True),                 # many children of one node
    ("f32", 20, 40, 50, "star", None, False),                # and the same token twice
    ("bf16", 20, 64, 300, "tree", [64, 63, 2, 40] * 5, False),
    ("f32", 12, 64, 33, "forest", None, True),               # nodes that are never reached
    ("f32", 3, 5, 70001, "tree", None, True),                # more than 64 tiles
    ("bf16", 3, 5, 150001, "tree", None, False),
    ("f32", 4, 3, 1, "tree", None, True),                    # a vocabulary of one
])
def test_tree_accept_matches_oracle(dtype, B, N, V, shape, counts, drafts):
    kda = need_gpu()
    case(f"tree_accept {dtype} B={B} N={N} V={V} {shape} counts={counts} drafts={drafts}")
    par = random_trees(B, N, V + N, shape)
    par[:, :1] = -1
    _check(kda, *_inputs(B, N, V, dtype, V + B, par, drafts), par, counts, shape == "chain")


def test_tree_accept_all_and_none():
    """u = 0 accepts every node along a chain, u just under 1 against a draft
    that the target hates refuses the first."""
    kda = need_gpu()
    B, N, V = 3, 6, 400
    case("tree_accept u at its ends")
    par = random_trees(B, N, 0, "chain")
    p, q, tokens, u = _inputs(B, N, V, "f32", 4, par, True)
    u[0] = 0.0
    u[0, 0] = 0.5
    u[1:] = float(np.nextafter(np.float32(1), np.float32(0)))
    for i in range(1, N):
        p[1:, i - 1, tokens[1:, i].long()] = 0.0
    lengths = _check(kda, p, q, tokens, u, par, None)
    assert lengths == [N, 1, 1]


def test_tree_accept_empty_residuals():
    """p = q: a refused draft (u >= 1 is outside the contract, zero mass is
    not) leaves nothing, and the token comes from p itself; zeros in p and q
    and one-hot rows."""
    kda = need_gpu()
    case("tree_accept residuals without mass")
    B, N, V = 4, 3, 9
    par = np.tile(np.array([-1, 0, 0], dtype=np.int32), (B, 1))
    p = torch.zeros((B, N, V))
    p[:, :, 4] = 1.0
    p[2:, :, 4] = 0.5
    p[2:, :, 8] = 0.5
    q = p[:, :N - 1].clone()
    tokens = torch.tensor([[0, 3, 3], [0, 4, 4], [0, 3, 0], [0, 7, 8]], dtype=torch.int32)
    u = torch.full((B, N), 0.75)
    path, m, nxt = kda.kda_tree_accept(p.cuda(), q.cuda(), tokens.cuda(), u.cuda(), i32(par))
    torch.cuda.synchronize()
    # tokens that the target and the draft give no mass are refused and take the whole residual with them
    assert m.tolist() == [1, 2, 1, 1] or m.tolist() == [1, 2, 1, 2], m
    for b in range(B):
        way, token, _ = otree.accept(p[b].numpy(), q[b].numpy(), tokens[b].numpy(), u[b].numpy(), par[b], N)
        assert path[b].tolist()[:len(way)] == way and int(m[b]) == len(way) and int(nxt[b]) == token, b


def test_tree_accept_tokens_outside_the_vocabulary():
    kda = need_gpu()
    case("tree_accept tokens outside [0, V)")
    B, N, V = 6, 4, 100
    par = np.tile(np.array([-1, 0, 0, 2], dtype=np.int32), (B, 1))
    p, q, tokens, u = _inputs(B, N, V, "f32", 9, par, True)
    tokens[:, 1] = torch.tensor([-1, V, 1 << 30, -(1 << 31), V + 1, -5], dtype=torch.int32)
    tokens[3:, 3] = V
    _check(kda, p, q, tokens, u, par, None)


def test_tree_accept_stays_in_range_on_bad_probabilities():
    """NaN, negative, infinite and all-zero rows (outside the contract): the
    results stay in range."""
    kda = need_gpu()
    case("tree_accept bad probabilities")
    B, N, V = 8, 6, 1500
    par = random_trees(B, N, 2, "tree")
    for drafts in (True, False):
        p, q, tokens, u = _inputs(B, N, V, "f32", 10, par, drafts)
        p[0] = float("nan")
        p[1] = 0.0
        p[2] = -1.0
        p[3] = float("inf")
        if drafts:
            q[4] = float("nan")
            q[5] = 0.0
            q[6] = float("inf")
        u[7] = float("nan")
        path, m, nxt = kda.kda_tree_accept(p.cuda(), None if q is None else q.cuda(), tokens.cuda(), u.cuda(),
                                           i32(par))
        torch.cuda.synchronize()
        assert ((nxt >= 0) & (nxt < V)).all(), nxt
        assert ((m >= 1) & (m <= N)).all(), m
        assert ((path >= -1) & (path < N)).all()


@pytest.mark.parametrize("drafts", [True, False])
def test_tree_accept_emits_the_targets_distribution(drafts):
    """Over many sequences with the same p and q: the first emitted token (the
    token of the first accepted child, or the next token) has the target's
    distribution, with three children drawn from q at the root.  65,536
    samples of 6 tokens: a frequency's standard deviation is at most
    sqrt(p (1 - p) / 65536) = 0.002; five of them are allowed."""
    kda = need_gpu()
    case(f"tree_accept distribution drafts={drafts}")
    B, N, V = 65536, 4, 6
    g = torch.Generator().manual_seed(99)
    p1 = torch.tensor([0.30, 0.05, 0.25, 0.10, 0.20, 0.10])
    q1 = torch.tensor([0.10, 0.30, 0.20, 0.25, 0.05, 0.10])
    par = np.tile(np.array([-1, 0, 0, 0], dtype=np.int32), (B, 1))
    p = p1.expand(B, N, V).contiguous()
    q = q1.expand(B, N - 1, V).contiguous() if drafts else None
    tokens = torch.multinomial(q1 if drafts else torch.ones(V), B * N, replacement=True,
                               generator=g).view(B, N).int()
    u = torch.rand((B, N), generator=g)
    path, m, nxt = kda.kda_tree_accept(p.cuda(), None if q is None else q.cuda(), tokens.cuda(), u.cuda(),
                                       i32(par))
    torch.cuda.synchronize()
    path, m, nxt = path.cpu(), m.cpu(), nxt.cpu().long()
    first = torch.where(m > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0].long(), nxt)
    freq = torch.bincount(first, minlength=V).double() / B
    sd = torch.sqrt(p1 * (1 - p1) / B)
    print(f"    accepted {float((m > 1).float().mean()):.3f}; frequencies {freq.tolist()}", flush=True)
    assert ((freq - p1).abs() < 5 * sd).all(), (freq, p1)
