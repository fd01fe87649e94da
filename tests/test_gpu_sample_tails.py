"""Draws from rows whose tails weigh next to nothing one token at a time, and something
together: masked tokens are never drawn, and what is drawn lies at its random number.

Sums are whole numbers of 2^-F of the largest weight, F = 62 minus the vocabulary's bits
(50 at most).  Token by token each is off by half of one at the most, V 2^-(F + 1) in
all, and by tiles of 1024 each of those; the sums' own roundings, 1e-12, come on top."""
import numpy as np
import pytest
import torch

from gpu_util import case, need_gpu, np_
from test_gpu_sample import DT, INF, NAN, gpu

pytestmark = pytest.mark.gpu


def bound(V):
    return (V + V // 1024 + 1) * 2.0 ** -(min(62 - V.bit_length(), 50) + 1) + 1e-12


def drawn_at(l, token, u, T=1.0, keep=None):
    """The kept token's share of the row from before it to after it holds u, within the bound."""
    l = np.asarray(l, np.float64)
    with np.errstate(invalid="ignore"):
        w = np.exp((l - l.max()).astype(np.longdouble) / np.longdouble(T))
    if keep is not None:
        w = np.where(keep, w, 0)
    assert w[token] > 0, f"token {token} of logit {l[token]} weighs nothing"
    cum = np.cumsum(w) / w.sum()
    before = cum[token - 1] if token else 0
    off = max(float(before) - u, u - float(cum[token]))
    assert off <= bound(len(l)), f"token {token} holds {before} to {cum[token]}, u = {u}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1025, 32000, 160000])
@pytest.mark.parametrize("tail", [-31.0, -33.0, -34.0, -36.0, -39.0])
def test_a_masked_token_is_never_drawn_beside_a_thin_tail(V, dtype, tail):
    kda = need_gpu()
    case(f"thin tail V={V} {dtype} {tail}")
    heads = [(V // 2,), (V - 1,), (1,), (V // 5, V - 7), (V // 3, V // 2)]     # (rows of one token, and of two equal ones)
    x = torch.full((len(heads), V), tail, device="cuda")
    for r, at in enumerate(heads):
        x[r, list(at)] = 0.0
        x[r, 0] = -INF
    x = x.to(DT[dtype])
    l = np_(x)
    # (whether the tail's part of the first and of the last tile of 1024 is a unit)
    some = np.exp(tail) * min(1022, (V - 1) % 1024 + 1) * 2.0 ** min(62 - V.bit_length(), 50) >= 1
    for u in (0.0, NAN, 2.0 ** -24, 0.25, 0.5, 1 - 2.0 ** -24, 1.0):
        token, probs = kda.kda_sample(x, gpu([u] * len(heads)), probs=True)
        torch.cuda.synchronize()
        assert (probs.gather(1, token[:, None].long()) > 0).all(), u
        for r in range(len(heads)):
            t, at = int(token[r]), 0.0 if u != u else u
            drawn_at(l[r], t, at)
            # (inside a tile weights count in 2^-50 of its largest: beside a 1 a tail of -36 is 0.26 of that, nothing.
            # So these hold where the tile at that end has no head, or the tail's tokens are more than half of 2^-50)
            thick = np.exp(tail) * 2.0 ** 50 > 0.5
            if some and at == 0.0 and (thick or min(heads[r]) >= 1024):
                assert t == 1, (r, t)       # the first one that is not masked
            if some and at == 1.0 and (thick or max(heads[r]) // 1024 < (V - 1) // 1024):
                assert t == V - 1, (r, t)   # the last one


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("u", [0.0, NAN, 1.0])
def test_masked_tiles_before_and_behind(u, dtype):
    """A masked first tile, one of a thin tail, and one token of weight far behind; and the other way round."""
    kda = need_gpu()
    V = 160000
    case(f"masked tiles u={u} {dtype}")
    x = torch.full((4, V), -INF, device="cuda")
    x[0, 1024:2048], x[0, 5000] = -35.0, 0.0
    x[1, 1030:1033], x[1, 5000] = -35.0, 0.0           # (less than a unit together: nothing)
    x[2, 5000], x[2, 150000:150900] = 0.0, -33.0
    x[3, 0], x[3, 100000:] = 0.0, -34.0
    x = x.to(DT[dtype])
    token, probs = kda.kda_sample(x, gpu([u] * 4), probs=True)
    torch.cuda.synchronize()
    assert token.tolist() == ([5000, 5000, 150899, V - 1] if u == 1.0 else [1024, 5000, 5000, 0])
    assert (probs.gather(1, token[:, None].long()) > 0).all()


@pytest.mark.parametrize("V", [3000, 32000, 160001])
def test_thin_tails_behind_every_filter(V):
    """Kept or not, by each filter: the token is kept and lies at its random number."""
    kda = need_gpu()
    case(f"thin tails, filters V={V}")
    T = [1.0, 0.5, 3.0, 1.0]
    x = torch.full((4, V), -34.0, device="cuda")
    x[:, ::2] -= 0.5
    x[0, V // 2] = 0.0
    x[1] *= 0.5
    x[1, [7, V - 9]] = 0.0
    x[2] *= 3.0
    x[2, V - 1] = 0.0
    x[3, 40:80] = -1.0
    x[:, 0] = -INF
    l = np_(x)
    for k, p, m in ((None, None, 1e-17), (None, None, 1e-15), ([V - 1] * 4, None, None), ([V // 2] * 4, None, 1e-16),
                    ([5] * 4, None, None), (None, [1 - 2.0 ** -24] * 4, None), (None, [0.9] * 4, 1e-15)):
        m = None if m is None else [m] * 4
        for u in (0.0, 0.5, 1 - 2.0 ** -24, 1.0):
            token, probs = kda.kda_sample(x, gpu([u] * 4), gpu(T), gpu(k, torch.int32), gpu(p), gpu(m), probs=True)
            torch.cuda.synchronize()
            keep = np_(probs) > 0
            for r in range(4):
                drawn_at(l[r], int(token[r]), u, T[r], keep[r])


@pytest.mark.parametrize("V,tail", [(160000, -31.5), (1 << 22, -28.5), (1 << 22, -27.0)])
def test_borders_hold_within_what_the_sums_leave_out(V, tail):
    """Tails of tokens that each weigh less than half a unit are left out of the sums by token: a share of top-p, and
    a random number, are met within V 2^-(F + 1) of the sum, at four million tokens more than a step of either."""
    kda = need_gpu()
    case(f"borders V={V} {tail}")
    x = torch.full((6, V), tail, device="cuda")
    x[:, [3, V // 2, V - 5]] = torch.tensor([0.0, -0.5, -1.0], device="cuda")
    l = np_(x[0]).astype(np.float64)
    w = np.exp((l - l.max()).astype(np.longdouble))
    w = w / w.sum()
    order = np.lexsort((np.arange(V), -l))
    share = np.cumsum(w[order])
    p = [1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -20, 0.984375, 0.5, 1.0]
    u = [1 - 2.0 ** -24, 1 - 2.0 ** -22, 1.0, 1 - 2.0 ** -19, 0.0, 0.25]
    for top_p, min_p in ((p, None), (None, [1e-30] * 6), (p, [1e-30] * 6), (None, None)):
        token, probs = kda.kda_sample(x, gpu(u), None, None, gpu(top_p), gpu(min_p), probs=True)
        torch.cuda.synchronize()
        for r in range(6):
            keep = np_(probs[r]) > 0
            n = int(keep.sum())
            assert keep[order[:n]].all()        # the first n
            if top_p is not None and p[r] < 1:
                assert share[n - 1] >= p[r] - bound(V) and (n == 1 or share[n - 2] < p[r] + bound(V)), (r, n)
            else:
                assert n == V
            drawn_at(l, int(token[r]), u[r], 1.0, keep)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 3000, 40000])
def test_rows_without_a_finite_logit(V, dtype):
    """-1 and no probabilities where every logit is -infinity or NaN; among +infinities one of those."""
    kda = need_gpu()
    case(f"rows without a finite logit V={V} {dtype}")
    x = torch.full((4, V), -INF, device="cuda")
    x[1, ::2] = NAN
    x[2, [V // 2, V - 1]] = INF
    x[3] = NAN
    x[3, V // 3] = INF
    x = x.to(DT[dtype])
    for ask in ({}, dict(top_k=gpu([2] * 4, torch.int32)), dict(top_p=gpu([0.9] * 4)), dict(min_p=gpu([0.5] * 4)),
                dict(temperature=gpu([0.0] * 4))):
        token, probs = kda.kda_sample(x, gpu([0.75] * 4), probs=True, **ask)
        torch.cuda.synchronize()
        greedy = "temperature" in ask
        assert token.tolist() == [-1, -1, V // 2 if greedy else V - 1, V // 3]
        assert (probs[:2] == 0).all() and (probs.sum(1) == gpu([0.0, 0.0, 1.0, 1.0])).all()
        assert probs[2, V // 2] == (1.0 if greedy else 0.5) and probs[3, V // 3] == 1.0
