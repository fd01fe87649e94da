"""Sampling on the GPU against a sorted row in extended precision.

Tokens are equal wherever the oracle's nearest border lies further than `slack`
from the random number.  Weights are rounded to 2^-F of the largest, F = 62 minus
the vocabulary's bits (50 at most): a sum of V of them, each off by a random half
of that at most, is off by some sqrt(V / 12) 2^-F, 7e-12 at 160,000 tokens and 1e-9
at four million; the inputs here are checked to lie further away.  Probabilities
are within 4.5 * 2^-24 of themselves and half a step of their type (2^f by the
hardware, an ulp or 2 * 2^-24; its argument's rounding, 0.35 * 2^-24; one rounding to
the type, beside fp32's for bf16).
"""
import numpy as np
import pytest
import torch

from oracle import sample as osamp
from gpu_util import case, need_gpu, np_

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
NAN, INF = float("nan"), float("inf")


def gpu(x, dtype=torch.float32):
    return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")


def check(kda, logits, u, T=None, k=None, p=None, m=None, slack=1e-11):
    """Tokens and probabilities of every row, with and without each other."""
    R, V = logits.shape
    args = (gpu(T), gpu(k, torch.int32), gpu(p), gpu(m))
    uu = gpu(u)
    token, probs = kda.kda_sample(logits, uu, *args, probs=True)
    alone, none = kda.kda_sample(logits, uu, *args)
    no, only = kda.kda_sample(logits, None, *args, probs=True)
    torch.cuda.synchronize()
    assert none is None and no is None
    assert torch.equal(token, alone) and torch.equal(probs, only)
    l, got, tok = np_(logits).astype(np.float64), np_(probs).astype(np.float64), token.cpu().numpy()
    f32 = lambda x, r, none: none if x is None else float(np.float32(x[r]))  # noqa: E731
    half = HALF["bf16" if logits.dtype == torch.bfloat16 else "f32"]
    for r in range(R):
        t, pr, margin = osamp.row(l[r], f32(u, r, None), f32(T, r, 1.0), 0 if k is None else k[r], f32(p, r, 1.0),
                                  f32(m, r, 0.0))
        assert margin > slack, f"row {r}: a border {margin:.1e} away: another input is needed"
        assert tok[r] == t, f"row {r}: token {tok[r]}, {t} expected (border {margin:.1e} away)"
        off = np.abs(got[r] - pr)
        # (below the smallest normal number of the type a step is absolute)
        ok = off <= (4.5 * 2.0 ** -24 + half) * pr + 2.0 ** -126
        assert ok.all(), f"row {r}: probability {got[r][~ok][:3]} at {np.nonzero(~ok)[0][:3]}, {pr[~ok][:3]} expected"
        assert ((got[r] > 0) <= (pr > 0)).all()
    return tok


def rows(R, V, dtype, seed, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, V), generator=g, device="cuda") * 2.5
    if kind == "peaked":
        at = torch.randint(0, V, (R, 40), generator=g, device="cuda")
        x.scatter_(1, at, 14 + 2 * torch.randn((R, 40), generator=g, device="cuda"))
    if kind == "coarse":
        x = torch.round(x)
    return x.to(DT[dtype])


def uniform(R, seed):
    return [float(x) for x in np.random.default_rng(seed).random(R, dtype=np.float32)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 5000, 20011])
def test_every_filter_at_sizes_around_tiles_and_lists(V, dtype):
    kda = need_gpu()
    case(f"sample V={V} {dtype}")
    R = 12
    x, u = rows(R, V, dtype, V, "peaked" if V % 2 else "normal"), uniform(R, V)
    T = [0.7, 1.0, 1.3, 0.0] * 3
    k = [1, 2, 5, 50, 0, -3, V, V + 1, max(1, V - 1), max(1, V // 2), 7, 1 << 30]
    p = [0.9, 0.5, 0.99, 1.0, 0.1, 0.95, 0.8, 0.3, 0.999, 2.0, 0.6, 0.7]
    m = [0.05, 0.0, 0.3, 0.1, 1e-6, 0.01, -1.0, 0.02, 0.5, 0.001, 1.0, 7.0]
    check(kda, x, u)
    check(kda, x, u, T)
    check(kda, x, u, None, k)
    check(kda, x, u, T, None, p)
    check(kda, x, u, T, None, None, m)
    check(kda, x, u, T, k, p)
    check(kda, x, u, T, k, None, m)
    check(kda, x, u, T, None, p, m)
    check(kda, x, u, T, k, p, m)


@pytest.mark.parametrize("V,dtype,kind", [(32000, "f32", "peaked"), (50021, "bf16", "normal"), (160001, "f32", "normal"),
                                          (160000, "bf16", "peaked"), (400000, "f32", "normal"), (32000, "bf16", "coarse")])
def test_large_vocabularies(V, dtype, kind):
    kda = need_gpu()
    R = 6
    case(f"sample V={V} {dtype} {kind}")
    x, u = rows(R, V, dtype, 5, kind), uniform(R, 6)
    T = [0.6, 1.0, 1.4, 0.9, 3.0, 1.0]
    check(kda, x, u, T)
    check(kda, x, u, T, [40, 1000, 2000, 20000, V - 1, 1])
    check(kda, x, u, T, None, [0.9, 0.3, 0.95, 0.999, 0.8, 0.5])
    check(kda, x, u, T, [40, 200, 3000, 20000, 0, 17], [0.9, 0.3, 0.95, 0.99, 0.8, 0.5])
    check(kda, x, u, T, [0, 200, 0, 20000, 0, 17], [0.9, 1.0, 0.95, 0.99, 0.8, 1.0], [0.1, 0.01, 1e-4, 1e-7, 0.02, 0.9])
    check(kda, x, u, T, None, None, [0.1, 0.01, 1e-4, 1e-7, 0.02, 0.9])
    check(kda, x, u, T, [5000] * R, None, [0.1, 0.01, 1e-4, 1e-7, 0.02, 0.9])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [32768, 40001, 160000, 262144])
def test_rows_whose_tiles_are_unlike(V, dtype):
    """A row's parts say little about its whole: sorted rows, rows whose tiles differ by residue, rows with most tiles
    masked, two values alone."""
    kda = need_gpu()
    R = 12
    x = rows(R, V, "f32", V + 1)
    t = torch.arange(V, device="cuda") // 1024
    some = (t // 16 + t) % 4 == 0
    x[0], x[1] = torch.sort(x[0]).values, torch.sort(x[1], descending=True).values
    x[2, some] -= 6
    x[3, ~some] -= 6
    x[4, some] = -INF
    x[5, ~some] = -INF
    x[6, V // 3:] = -INF
    x[7, : V - 3 * 1024] = -INF
    x[8] = torch.where(torch.arange(V, device="cuda") % 3 == 0, 1.5, -0.5)
    x[9] = torch.where(some, 2.0, 0.0) + x[9] * 1e-3
    x[10, 17] += 25
    x[11] *= 0.1
    x = x.to(DT[dtype])
    for j, p in enumerate((0.5, 0.9, 0.99, 0.9997)):
        u = uniform(R, V + j)
        case(f"sample tiles V={V} {dtype} p={p}")
        check(kda, x, u, None, None, [p] * R, slack=1e-10)
    check(kda, x, uniform(R, 3), [1.7] * R, None, [0.93] * R, [1e-5] * R, slack=1e-10)


@pytest.mark.parametrize("V,dtype,kind", [(524288, "bf16", "normal"), (524289, "f32", "peaked"), (1 << 22, "bf16", "normal")])
def test_the_largest_vocabularies(V, dtype, kind):
    """Around the most tiles whose groups' maxima are kept, and the most tokens."""
    kda = need_gpu()
    R = 2
    case(f"sample V={V} {dtype} {kind}")
    x, u = rows(R, V, dtype, 50, kind), uniform(R, 51)
    T = [0.7, 1.2]
    check(kda, x, u, T, slack=1e-8)
    check(kda, x, u, T, [3000, 40], [0.9, 0.8], slack=1e-8)
    check(kda, x, u, T, None, [0.9, 0.4], slack=1e-8)
    check(kda, x, u, T, [0, V // 3], [0.6, 1.0], [0.01, 1e-5], slack=1e-8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100, 3000, 40000])
def test_equal_logits_go_by_index(V, dtype):
    """Every logit the same: the k kept are the first k, sums are whole numbers
    of the weight 1 (met exactly at a half, a quarter), the drawn index is
    floor(u * number of them)."""
    kda = need_gpu()
    case(f"equal logits V={V} {dtype}")
    x = torch.full((8, V), -3.5, dtype=DT[dtype], device="cuda")
    u = [0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.125, 0.1, 0.9]
    k = [1, 8, 64, V // 2, V, 0, 16, 32]
    assert list(check(kda, x, u)[:4]) == [0, V // 4, V // 2, 3 * V // 4]
    check(kda, x, u, None, k)
    check(kda, x, u, None, None, [0.5, 0.25, 0.75, 0.125, 1.0, 0.5, 0.0, 0.5])
    check(kda, x, u, None, k, [0.5, 0.25, 0.75, 0.5, 0.5, 0.25, 0.5, 0.5])
    check(kda, x, u, None, k, [0.5] * 8, [1.0] * 8)
    check(kda, x, u, None, [V - 1] * 8, None, [1.0] * 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_values_many_times(dtype):
    """Whole logits: thousands of ties at every border."""
    kda = need_gpu()
    V, R = 30011, 8
    case(f"coarse logits {dtype}")
    x, u = rows(R, V, dtype, 8, "coarse"), uniform(R, 9)
    check(kda, x, u, [1.0] * R, [1, 3, 100, 1000, 5000, 20000, 30000, 12345])
    check(kda, x, u, [1.0] * R, None, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99, 0.999, 0.05])
    check(kda, x, u, [2.0] * R, [25000] * R, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99, 0.999, 0.05], [0.01] * R)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [257, 9000, 70001])
def test_masked_rows(V, dtype):
    """-infinity, the type's lowest value, NaN and +infinity."""
    kda = need_gpu()
    case(f"masks V={V} {dtype}")
    R = 10
    x, u = rows(R, V, dtype, 10), uniform(R, 11)
    low = torch.finfo(DT[dtype]).min
    x[0] = -INF                        # nothing left
    x[1, :] = -INF
    x[1, V - 1] = -7.0                 # one left, the last
    x[2, : V - 3] = low                # masked by the lowest value
    x[3] = low                         # all of it
    x[4, ::2] = -INF
    x[5, 5] = INF                      # an infinite logit takes it all
    x[6, [3, V - 2]] = INF             # two share it
    x[7, ::3] = NAN
    x[8] = NAN
    x[9, 1:] = -INF
    for T in (None, [1.0] * R, [0.0] * R, [INF] * R, [1e-38] * R):
        tok = check(kda, x, u, T)
        assert tok[0] == -1 and tok[8] == -1 and tok[1] == V - 1 and tok[5] == 5 and tok[9] == 0
    for k in (1, 2, 40, V - 1):
        check(kda, x, u, [0.8] * R, [k] * R)
        check(kda, x, u, [0.8] * R, [k] * R, [0.9] * R, [0.01] * R)
    check(kda, x, u, [0.8] * R, None, [0.9] * R)
    check(kda, x, u, [0.8] * R, None, None, [0.01] * R)
    check(kda, x, u, [INF] * R, [7] * R, [0.7] * R, [0.5] * R)


@pytest.mark.parametrize("V", [900, 33000])
def test_what_lies_outside_the_ranges(V):
    """Temperatures, shares and random numbers that are no such thing."""
    kda = need_gpu()
    case(f"odd requests V={V}")
    x = rows(8, V, "f32", 12, "peaked")
    u = [-1.0, 0.0, 1.0, 2.0, NAN, INF, -INF, 0.5]
    check(kda, x, u)
    check(kda, x, u, None, [30] * 8)
    check(kda, x, u, None, None, [0.9] * 8)
    v = uniform(8, 13)
    check(kda, x, v, [-1.0, 0.0, -0.0, NAN, 1e-45, 1e30, INF, 1.0])
    check(kda, x, v, None, None, [-1.0, 0.0, NAN, 1e-30, 1 - 2.0 ** -24, 5.0, INF, -INF])
    check(kda, x, v, None, None, None, [-1.0, 0.0, NAN, 1e-30, 1.0, 5.0, INF, 1e-38])
    check(kda, x, v, None, [-(1 << 31), -1, 0, 1, V, V + 1, (1 << 31) - 1, V - 1])


def test_far_logits_weigh_nothing_and_near_ones_are_told_apart():
    kda = need_gpu()
    case("spread logits")
    V = 5000
    x = torch.linspace(-3e38, 3e38, V, device="cuda").expand(4, V).contiguous()
    check(kda, x, [0.1, 0.9, 0.5, 0.5], [1.0, 1e30, 1e37, 1e38])      # (its step overflows: infinities and NaN)
    x = (torch.linspace(-1, 1, V, device="cuda") * 3e38).expand(4, V).contiguous()
    assert torch.isfinite(x).all()
    tok = check(kda, x, [0.1, 0.9, 0.5, 0.5], [1.0, 1e30, 1e37, 1e38])
    assert tok[0] == V - 1
    # neighbours in the last bit, a temperature that makes something of it
    y = (1000 + torch.arange(V, device="cuda").float() * 2.0 ** -13).flip(0).expand(4, V).contiguous()
    check(kda, y, [0.1, 0.9, 0.5, 0.7], [0.01, 0.1, 1.0, 0.05], [5, 500, 4000, 4999], [0.5, 0.9, 0.99, 0.8])


@pytest.mark.parametrize("V", [70, 3000, 40000])
def test_zeros_of_both_signs(V):
    """Log-probabilities, whose largest may be 0; both zeros are one value, where
    they are the largest, where a filter ends and where a tile holds nothing else."""
    kda = need_gpu()
    case(f"zeros V={V}")
    x = -rows(6, V, "f32", 40).abs()
    x[0, ::7] = 0.0
    x[0, ::14] = -0.0
    x[1] = -0.0
    x[1, 1::2] = 0.0
    x[2, V // 2] = -0.0
    x[3] = torch.round(rows(1, V, "f32", 41)[0])
    x[4] = 0.0
    x[4, V - 1] = 1e-45
    x[5] = -1e-45
    x[5, 3] = -0.0
    u = uniform(6, 42)
    for T in ([0.0] * 6, [1.0] * 6):
        check(kda, x, u, T)
    check(kda, x, u, None, [3, 5, 1, V // 3, 2, 2])
    check(kda, x, u, None, [V // 2] * 6)
    check(kda, x, u, None, None, [0.7, 0.3, 0.9, 0.8, 0.3, 0.6])
    check(kda, x, u, None, None, None, [1.0] * 6)
    check(kda, x.bfloat16(), u, [1.0] * 6, [V // 3] * 6, [0.9] * 6, [0.5] * 6)


def test_leading_dimensions_and_given_outputs():
    kda = need_gpu()
    case("[B, N, V] logits, as the verification of drafts has its probabilities")
    B, N, V = 3, 4, 1500
    x = rows(B * N, V, "bf16", 14).view(B, N, V)
    u = torch.rand((B, N), device="cuda")
    T = torch.full((B, N), 0.8, device="cuda")
    token = torch.empty((B, N), dtype=torch.int32, device="cuda")
    probs = torch.empty_like(x)
    t, p = kda.kda_sample(x, u, T, token=token, probs=probs)
    assert t is token and p is probs
    flat, fp = kda.kda_sample(x.view(B * N, V), u.view(-1), T.view(-1), probs=True)
    assert torch.equal(token.view(-1), flat) and torch.equal(probs.view(B * N, V), fp)
    one, _ = kda.kda_sample(x[0, 0], u[0, 0], T[0, 0])
    assert one.shape == () and int(one) == int(token[0, 0])
    e, ep = kda.kda_sample(x[:0], u[:0], T[:0], probs=True)
    assert e.shape == (0, N) and ep.shape == (0, N, V)


def test_rows_past_32_bits():
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    R, V = 70000, 65537
    case(f"R={R} V={V}")
    assert (R - 1) * V > 2 ** 32
    x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    part = rows(2, V, "bf16", 15)
    x[0], x[R - 1] = part[0], part[1]
    u = torch.full((R,), 0.5, device="cuda")
    p = torch.full((R,), 0.5, device="cuda")
    token, probs = kda.kda_sample(x, u, None, None, p, probs=True)
    few, fp = kda.kda_sample(part, u[:2], None, None, p[:2], probs=True)
    torch.cuda.synchronize()
    assert token[0] == few[0] and token[R - 1] == few[1]
    assert torch.equal(probs[0], fp[0]) and torch.equal(probs[R - 1], fp[1])
    # the others are flat: half of them kept, the middle of those drawn
    half = (V + 1) // 2
    assert (token[1:R - 1] == half // 2).all()
    assert (probs[R // 2, :half] > 0).all() and (probs[R // 2, half:] == 0).all()


def test_the_draw_follows_the_probabilities():
    """Tokens of evenly spread random numbers: each as often as its probability
    says, to one."""
    kda = need_gpu()
    n, V = 4096, 3001
    case("frequencies")
    x = rows(1, V, "f32", 16, "peaked").expand(n, V).contiguous()
    u = ((torch.arange(n, device="cuda") + 0.5) / n).float()
    T, k, p = torch.full((n,), 0.9, device="cuda"), torch.full((n,), 300, dtype=torch.int32, device="cuda"), torch.full((n,), 0.97, device="cuda")
    token, probs = kda.kda_sample(x, u, T, k, p, probs=True)
    torch.cuda.synchronize()
    assert (token[1:] >= token[:-1]).all()
    hist = torch.bincount(token.long(), minlength=V).double()
    assert ((hist - n * probs[0].double()).abs() <= 1 + n * V * 2.0 ** -24).all()


def test_graph_replays_and_streams():
    kda = need_gpu()
    R, V = 5, 20000
    case("captured and on two streams")
    x = rows(R, V, "f32", 17, "peaked")
    u, T, p = (torch.zeros(R, device="cuda") for _ in range(3))
    T.fill_(0.9)
    p.fill_(0.8)
    k = torch.full((R,), 60, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.kda_sample(x, u, T, k, p, probs=True)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):          # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kda.kda_sample(x, u, T, k, p, probs=True)
        graphs.append((g, out))
    for r in range(4):
        x.copy_(rows(R, V, "f32", 30 + r, "peaked" if r % 2 else "normal"))
        u.copy_(torch.rand(R, device="cuda"))
        k.fill_(60 if r < 2 else 9000)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        t, pr = kda.kda_sample(x, u, T, k, p, probs=True)
        torch.cuda.synchronize()
        for _, (gt, gp) in graphs:
            assert torch.equal(gt, t) and torch.equal(gp, pr), r
    want = [kda.kda_sample(y, u, T, k, p, probs=True) for y in (x, x.flip(1).contiguous())]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ins = (x, x.flip(1).contiguous())
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, y in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(kda.kda_sample(y, u, T, k, p, probs=True))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_verification_of_drafts_takes_the_probabilities():
    """A draft model's tokens and probabilities and the target's probabilities,
    all from logits, through kda_tree_accept: with the drafts' logits the
    target's own every draft is accepted."""
    kda = need_gpu()
    B, N, V = 4, 6, 3000
    case("sample -> accept")
    target = rows(B * N, V, "f32", 18, "peaked").view(B, N, V)
    ask = (torch.full((B, N), 0.8, device="cuda"), torch.full((B, N), 50, dtype=torch.int32, device="cuda"),
           torch.full((B, N), 0.9, device="cuda"))
    drawn, q = kda.kda_sample(target, torch.rand((B, N), device="cuda"), *ask, probs=True)
    _, p = kda.kda_sample(target, None, *ask, probs=True)
    tokens = torch.cat([torch.zeros((B, 1), dtype=torch.int32, device="cuda"), drawn[:, :-1]], 1).contiguous()
    u = torch.rand((B, N), device="cuda")
    path, n, nxt = kda.kda_tree_accept(p, q[:, :-1].contiguous(), tokens, u)
    torch.cuda.synchronize()
    assert (n == N).all() and (path == torch.arange(N, device="cuda", dtype=torch.int32)).all()
    last, _ = kda.kda_sample(target[:, -1].contiguous(), u[:, 0].contiguous(), *(x[:, 0].contiguous() for x in ask))
    assert torch.equal(nxt, last)
