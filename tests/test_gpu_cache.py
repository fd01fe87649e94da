"""The 8-bit state cache on the GPU: store, load, decode and fold against the
float64 oracle within bounds that count roundings, and what they leave alone."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from cache_util import D, DT, SENTINEL, i32, states, token, window, within
from gpu_util import case, need_gpu, np_

pytestmark = pytest.mark.gpu


def pool(P, H):
    return (torch.full((P, H, D, D), SENTINEL, dtype=torch.int8, device="cuda"),
            torch.full((P, H, D), float(SENTINEL), device="cuda"))


def same_codes(codes, scale, S):
    """Bit for bit what the definition gives."""
    c, s = oc.quantise(np_(S))
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scale.cpu().numpy(), s)


@pytest.mark.parametrize("B,H,spread", [(1, 1, 0.0), (2, 3, 1.0), (5, 7, 5.0), (3, 96, 1.0)])
def test_store_gives_the_codes_and_load_the_values(B, H, spread):
    kda = need_gpu()
    case(f"store/load B={B} H={H} spread={spread}")
    S = states(B, H, 1, spread)
    codes, scale = kda.kda_cache_store(S)
    back = kda.kda_cache_load(codes, scale)
    torch.cuda.synchronize()
    same_codes(codes, scale, S)
    # a code times its scale, rounded once
    c, s = codes.cpu().numpy().astype(np.float32), scale.cpu().numpy()
    assert np.array_equal(back.cpu().numpy(), np.swapaxes(c, -1, -2) * s[..., None])
    # half a step, and the roundings of the scale, the factor and the product (127 steps of 2^-24 each)
    step = np_(S.abs().amax(-1, keepdim=True)) / 127
    within("values", np_(back), np_(S), (0.5 + 4 * 127 * oc.EPS) * step + 0 * np_(S))


def test_ties_round_to_even_and_borders_hold():
    kda = need_gpu()
    case("ties, empty rows, smallest held row, extremes")
    S = torch.zeros((1, 1, D, D), device="cuda")
    S[0, 0, 0] = torch.arange(D, device="cuda") - 63.5        # (row 0: halves under a scale of 0.5)
    S[0, 0, 0, 0] = 127.0
    S[0, 0, 1, 5] = 2.0 ** -100
    S[0, 0, 1, 6] = -(2.0 ** -101)
    S[0, 0, 2, 5] = 2.0 ** -101                                # not held
    S[0, 0, 3] = 3.4e38
    S[0, 0, 4, 127] = -3.4e38
    S[0, 0, 5] = -0.0
    S[0, 0, 6, 3] = 1e-45
    codes, scale = kda.kda_cache_store(S)
    back = kda.kda_cache_load(codes, scale)
    torch.cuda.synchronize()
    same_codes(codes, scale, S)
    assert (back[0, 0, 2] == 0).all() and (back[0, 0, 6] == 0).all() and back[0, 0, 1, 5] > 0
    assert torch.isfinite(back).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_reads_back_as_nan_alone(bad):
    kda = need_gpu()
    case(f"store of {bad}")
    S = states(2, 3, 3)
    S[1, 2, 40, 17] = bad
    back = kda.kda_cache_load(*kda.kda_cache_store(S))
    torch.cuda.synchronize()
    nan = torch.isnan(back)
    assert nan[1, 2, 40].all() and nan.sum() == D


def test_pages_named_and_not_named():
    kda = need_gpu()
    B, H, P = 6, 5, 9
    case("store into pages: shuffled, outside, one page twice")
    S = states(B, H, 4)
    page = [7, -1, 3, 7, 9, 0]          # 7 twice: the later state counts; -1 and 9 are no pages
    codes, scale = pool(P, H)
    kda.kda_cache_store(S, codes, scale, i32(page))
    torch.cuda.synchronize()
    for p, b in ((7, 3), (3, 2), (0, 5)):
        same_codes(codes[p], scale[p], S[b])
    for p in set(range(P)) - {0, 3, 7}:
        assert (codes[p] == SENTINEL).all() and (scale[p] == SENTINEL).all()
    out = torch.full((5, H, D, D), 5.0, device="cuda")
    kda.kda_cache_load(codes, scale, i32([3, 3, -5, 1 << 30, 0]), S=out)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and (out[2:4] == 5.0).all()
    assert torch.equal(out[0], kda.kda_cache_load(codes, scale)[3])
    assert torch.equal(out[4], kda.kda_cache_load(codes, scale)[0])


def test_many_states_for_one_page_the_last_one_counts():
    kda = need_gpu()
    B, H = 700, 1
    case("store of 700 states into one page")
    S = states(B, H, 5)
    codes, scale = pool(2, H)
    kda.kda_cache_store(S, codes, scale, i32([1] * B))
    torch.cuda.synchronize()
    same_codes(codes[1], scale[1], S[B - 1, :])
    assert (codes[0] == SENTINEL).all()


SIZES = [
    # B, H, W, dtype, log alpha around -5 sigmoid(mu)
    (1, 1, 1, "bf16", -2.0), (2, 3, 4, "f32", -2.0), (3, 5, 8, "bf16", -2.0), (3, 7, 16, "f32", 1.0),
    (4, 2, 13, "bf16", 3.0), (2, 1, 16, "bf16", -6.0), (9, 3, 5, "f32", 8.0),
]


def counts(B, most):
    """Every place of the batch another length: none, all, in between."""
    return [(most * b) // max(1, B - 1) if B > 1 else most for b in range(B)]


@pytest.mark.parametrize("B,H,W,dtype,mu", SIZES)
def test_load_applies_the_window(B, H, W, dtype, mu):
    kda = need_gpu()
    case(f"load with window B={B} H={H} W={W} {dtype} mu={mu}")
    codes, scale = kda.kda_cache_store(states(B, H, 6))
    win = window(B, H, W, dtype, 7, mu)
    n = counts(B, W)
    for x in win:                           # what lies behind the last token is not looked at
        for b in range(B):
            x[b, :, n[b]:] = float("nan")
    got = np_(kda.kda_cache_load(codes, scale, None, win, i32(n)))
    c, s, w = codes.cpu().numpy(), scale.cpu().numpy(), [np_(x).astype(np.float64) for x in win]
    for b in range(B):
        for h in range(H):
            ref, bound = oc.state(c[b, h], s[b, h], *(x[b, h] for x in w), n[b])
            within(f"S[{b},{h}]", got[b, h], ref, bound)


@pytest.mark.parametrize("B,H,W,dtype,mu", SIZES)
def test_fold_rounds_what_load_gives(B, H, W, dtype, mu):
    kda = need_gpu()
    case(f"fold B={B} H={H} W={W} {dtype} mu={mu}")
    codes, scale = kda.kda_cache_store(states(B, H, 8))
    win = window(B, H, W, dtype, 9, mu)
    n = counts(B, W)
    c0, s0 = codes.clone(), scale.clone()
    kda.kda_cache_fold(codes, scale, win, i32(n))
    torch.cuda.synchronize()
    w = [np_(x).astype(np.float64) for x in win]
    got, sc = oc.values(codes.cpu().numpy(), scale.cpu().numpy()), scale.cpu().numpy().astype(np.float64)
    for b in range(B):
        if n[b] == 0:
            assert torch.equal(codes[b], c0[b]) and torch.equal(scale[b], s0[b])
            continue
        for h in range(H):
            ref, bound = oc.state(c0[b, h].cpu().numpy(), s0[b, h].cpu().numpy(), *(x[b, h] for x in w), n[b])
            step = np.abs(ref).max(-1) / 127
            far = bound.max(-1)             # of any entry of the row
            within(f"scale[{b},{h}]", sc[b, h], step, far / 127 + 2 * oc.EPS * step)
            within(f"S[{b},{h}]", got[b, h], ref, bound + ((0.5 + 4 * 127 * oc.EPS) * step + 2 * far)[:, None])


def test_fold_and_load_take_the_whole_window_without_counts_and_clamp_them():
    kda = need_gpu()
    B, H, W = 4, 3, 6
    case("counts: none given, negative, past the window")
    codes, scale = kda.kda_cache_store(states(B, H, 10))
    win = window(B, H, W, "bf16", 11)
    full = kda.kda_cache_load(codes, scale, None, win)
    none = kda.kda_cache_load(codes, scale)
    got = kda.kda_cache_load(codes, scale, None, win, i32([W, W + 5, -3, 0]))
    torch.cuda.synchronize()
    assert torch.equal(got[:2], full[:2]) and torch.equal(got[2:], none[2:]) and not torch.equal(full, none)
    c1, s1 = codes.clone(), scale.clone()
    kda.kda_cache_fold(codes, scale, win, i32([W, W + 5, -3, 0]))
    kda.kda_cache_fold(c2 := c1.clone(), s2 := s1.clone(), win)
    torch.cuda.synchronize()
    assert torch.equal(codes[:2], c2[:2]) and torch.equal(scale[:2], s2[:2])
    assert torch.equal(codes[2:], c1[2:]) and torch.equal(scale[2:], s1[2:])
    # a fold is a store of what a load gives
    same_codes(c2, s2, full)


@pytest.mark.parametrize("B,H,W,dtype,mu", SIZES + [(1, 96, 8, "bf16", -2.0), (5, 31, 3, "f32", -2.0)])
def test_decode_reads_the_state_and_appends(B, H, W, dtype, mu):
    kda = need_gpu()
    case(f"decode B={B} H={H} W={W} {dtype} mu={mu}")
    codes, scale = kda.kda_cache_store(states(B, H, 12, 2.0))
    win = window(B, H, W, dtype, 13, mu)
    n = counts(B, W - 1)
    q, k, v, la, beta = token(B, H, dtype, 14, mu)
    for x in win:
        for b in range(B):
            x[b, :, n[b]:] = float("nan")
    before = [x.clone() for x in win]
    o = kda.kda_cache_decode(q, k, v, la, beta, codes, scale, win, i32(n))
    torch.cuda.synchronize()
    half = oc.HALF[dtype]
    qn, kn, vn, ln, bn, on = (np_(x).astype(np.float64) for x in (q, k, v, la, beta, o))
    c, s, w = codes.cpu().numpy(), scale.cpu().numpy(), [np_(x).astype(np.float64) for x in win]
    for b in range(B):
        t = n[b]
        assert torch.equal(win[0][b, :, t], k[b]) and torch.equal(win[1][b, :, t], la[b])
        for x, y in zip(win, before):       # nothing else of the window is written
            rest = [i for i in range(W) if i != t]
            assert torch.equal(x[b, :, rest].view(torch.uint8), y[b, :, rest].view(torch.uint8))
        for h in range(H):
            u, bu, output = oc.decode(qn[b, h], kn[b, h], vn[b, h], ln[b, h], bn[b, h], c[b, h], s[b, h],
                                      *(x[b, h] for x in w), t)
            held = w[2][b, h, t]
            within(f"u[{b},{h}]", held, u, bu + half * (np.abs(u) + bu))
            ref, bo = output(held)
            within(f"o[{b},{h}]", on[b, h], ref, bo + half * (np.abs(ref) + bo))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_whole_numbers_is_exact(dtype):
    """Codes, vectors and updates that are whole numbers: no rounding at all."""
    kda = need_gpu()
    B, H, W = 2, 3, 5
    case(f"decode of whole numbers {dtype}")
    g = torch.Generator(device="cuda").manual_seed(3)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda").to(DT[dtype])

    codes = torch.randint(-127, 128, (B, H, D, D), generator=g, device="cuda").to(torch.int8)
    scale = torch.ones((B, H, D), device="cuda")
    win = (whole(-2, 3, B, H, W, D), torch.zeros((B, H, W, D), dtype=DT[dtype], device="cuda"), whole(-2, 3, B, H, W, D))
    q = torch.zeros((B, H, D), dtype=DT[dtype], device="cuda")
    k = q.clone()
    q[..., 5], q[..., 100], k[..., 9] = 3.0, -2.0, 1.0
    v, la, beta = whole(-9, 10, B, H, D), torch.zeros_like(q), torch.ones((B, H), dtype=DT[dtype], device="cuda")
    o = kda.kda_cache_decode(q, k, v, la, beta, codes, scale, win, i32([4, 2]))
    torch.cuda.synchronize()
    for b, n in ((0, 4), (1, 2)):
        S = oc.values(codes[b].cpu().numpy(), scale[b].cpu().numpy()) + np.einsum(
            "hti,htj->hij", np_(win[0][b])[:, :n].astype(np.float64), np_(win[2][b])[:, :n].astype(np.float64))
        assert np.array_equal(np_(win[2][b])[:, n], np_(v[b]) - S[:, 9])     # (at most 8 bits long)
        assert np.array_equal(np_(o[b]), np_(torch.tensor(3 * S[:, 5] - 2 * S[:, 100]).to(DT[dtype])))


def test_decode_with_scales_of_every_size():
    """Key channels from 2^-60 to 2^60 beside each other: each output is off by
    a part of the largest channel's own rounding, 2^-30 of it."""
    kda = need_gpu()
    B, H, W = 2, 2, 4
    case("decode, scales 2^-60 .. 2^60")
    S = states(B, H, 20) * torch.exp2(torch.linspace(-60, 60, D, device="cuda"))[:, None]
    codes, scale = kda.kda_cache_store(S)
    win = window(B, H, W, "f32", 21)
    q, k, v, la, beta = token(B, H, "f32", 22)
    o = kda.kda_cache_decode(q, k, v, la, beta, codes, scale, win, i32([0, 3]))
    torch.cuda.synchronize()
    a = [np_(x).astype(np.float64) for x in (q, k, v, la, beta)]
    w = [np_(x).astype(np.float64) for x in win]
    for b, n in ((0, 0), (1, 3)):
        for h in range(H):
            u, bu, output = oc.decode(*(x[b, h] for x in a), codes[b, h].cpu().numpy(), scale[b, h].cpu().numpy(),
                                      *(x[b, h] for x in w), n)
            held = w[2][b, h, n]
            within("u", held, u, bu + oc.EPS * np.abs(u))
            ref, bo = output(held)
            within("o", np_(o[b, h]), ref, bo + oc.EPS * np.abs(ref))


def test_idle_places_keep_everything():
    kda = need_gpu()
    B, H, W = 5, 6, 3
    case("idle places: n_win outside [0, W)")
    codes, scale = kda.kda_cache_store(states(B, H, 15))
    win = window(B, H, W, "bf16", 16)
    before = [x.clone() for x in win]
    x = token(B, H, "bf16", 17)
    o = torch.full((B, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_cache_decode(*x, codes, scale, win, i32([-1, 1, W, 1 << 30, -(1 << 31)]), o=o)
    torch.cuda.synchronize()
    for b in (0, 2, 3, 4):
        assert (o[b] == 5.0).all() and all(torch.equal(y[b], z[b]) for y, z in zip(win, before))
    assert not (o[1] == 5.0).any()


@pytest.mark.parametrize("which", range(6))
def test_what_a_nan_reaches(which):
    """A NaN of one head's vector, state or window reaches no other head."""
    kda = need_gpu()
    B, H, W = 2, 5, 4
    case(f"NaN in input {which}")
    codes, scale = kda.kda_cache_store(states(B, H, 18))
    win = window(B, H, W, "bf16", 19)
    x = token(B, H, "bf16", 20)
    ref = kda.kda_cache_decode(*x, codes, scale, tuple(y.clone() for y in win), i32([2, 3]))
    if which < 4:
        x[which][1, 2, 77] = float("nan")
    elif which == 4:
        scale[1, 2, 77] = float("nan")
    else:
        win[2][1, 2, 1, 77] = float("nan")
    o = kda.kda_cache_decode(*x, codes, scale, win, i32([2, 3]))
    torch.cuda.synchronize()
    nan = torch.isnan(o)
    if which in (2, 5):
        assert nan[1, 2, 77] and nan.sum() == 1
    else:
        assert nan[1, 2].all() and nan.sum() == D
    assert torch.equal(o[~nan], ref[~nan])
    if which == 0:      # a query's reaches no update
        assert not torch.isnan(win[2]).any()


def test_last_places_past_32_bits():
    """Codes past 2^32 bytes and windows past 2^31 elements."""
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free memory")
    B, H, W = 2740, 96, 8
    case(f"far states B={B} H={H}")
    assert (B - 1) * H * D * D > 2 ** 32 - 2 ** 22 and B * H * D * D > 2 ** 32
    few = (0, B - 1)
    part = states(2, H, 23)
    pw = window(2, H, W, "bf16", 24)
    small = kda.kda_cache_store(part)
    codes = torch.zeros((B, H, D, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((B, H, D), device="cuda")
    win = tuple(torch.zeros((B, H, W, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    kda.kda_cache_store(part, codes, scale, i32(few))
    for x, y in zip(win, pw):
        x[0], x[B - 1] = y[0], y[1]
    q = tuple(torch.zeros((B,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in token(2, H, "bf16", 25))
    pt = token(2, H, "bf16", 25)
    for x, y in zip(q, pt):
        x[0], x[B - 1] = y[0], y[1]
    n = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    o = kda.kda_cache_decode(*q, codes, scale, win, n)
    po = kda.kda_cache_decode(*pt, *small, pw, n[:2].contiguous())
    kda.kda_cache_fold(codes, scale, win, n + 1)
    kda.kda_cache_fold(*small, pw, n[:2] + 1)
    S = kda.kda_cache_load(codes, scale, i32([B - 1, 0, B]), win, i32([2, 4, 1]))
    pS = kda.kda_cache_load(*small, i32([1, 0]), pw, i32([2, 4]))
    torch.cuda.synchronize()
    for i, b in enumerate(few):
        assert torch.equal(o[b], po[i]) and torch.equal(codes[b], small[0][i]) and torch.equal(scale[b], small[1][i])
        assert all(torch.equal(x[b], y[i]) for x, y in zip(win, pw))
    assert torch.equal(S[:2], pS) and (S[2] == 0).all()
    assert (codes[1] == 0).all() and (o[1] == 0).all()


def test_far_fp32_states_store_and_load():
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    B, H = 2740, 96
    case(f"store and load of fp32 states past 2^32 elements B={B} H={H}")
    S = torch.zeros((B, H, D, D), device="cuda")
    part = states(1, H, 26)
    S[B - 1] = part[0]
    codes, scale = kda.kda_cache_store(S)
    S.zero_()
    kda.kda_cache_load(codes, scale, S=S)
    torch.cuda.synchronize()
    assert torch.equal(S[B - 1], kda.kda_cache_load(*kda.kda_cache_store(part))[0]) and (S[0] == 0).all()


def test_no_states_at_all():
    kda = need_gpu()
    case("B = 0")
    H, W = 3, 4
    codes, scale = kda.kda_cache_store(torch.zeros((0, H, D, D), device="cuda"))
    win = tuple(torch.zeros((0, H, W, D), device="cuda") for _ in range(3))
    n = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros((0, H, D), device="cuda")
    assert kda.kda_cache_decode(x, x, x, x, torch.zeros((0, H), device="cuda"), codes, scale, win, n).shape == (0, H, D)
    assert kda.kda_cache_load(codes, scale, None, win, n).shape == (0, H, D, D)
    kda.kda_cache_fold(codes, scale, win, n)
    full = kda.kda_cache_store(states(2, H, 1))
    assert kda.kda_cache_load(*full, i32([])).shape == (0, H, D, D)
    kda.kda_cache_store(torch.zeros((0, H, D, D), device="cuda"), *full, i32([]))
    torch.cuda.synchronize()


def test_the_binding_refuses_what_does_not_fit():
    kda = need_gpu()
    case("refusals with GPU tensors")
    B, H, W = 2, 3, 4
    codes, scale = kda.kda_cache_store(states(B, H, 1))
    win = window(B, H, W, "bf16", 2)
    q, k, v, la, beta = token(B, H, "bf16", 3)
    n = i32([0, 1])
    call = lambda **kw: kda.kda_cache_decode(**dict(dict(  # noqa: E731
        q=q, k=k, v=v, log_alpha=la, beta=beta, codes=codes, scale=scale, window=win, n_win=n), **kw))
    for kw, what in ((dict(k=k.float()), TypeError), (dict(codes=codes[:1]), ValueError), (dict(scale=scale.double()), TypeError),
                     (dict(window=win[:2]), ValueError), (dict(window=(win[0], win[1], win[2].float())), TypeError),
                     (dict(window=tuple(x.transpose(0, 1) for x in win)), ValueError), (dict(n_win=n.long()), TypeError),
                     (dict(n_win=n.cpu()), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                     (dict(codes=codes.transpose(2, 3)), ValueError), (dict(o=q), kda.KDAError),
                     (dict(window=(win[0], win[0], win[2])), kda.KDAError)):
        with pytest.raises(what):
            call(**kw)
    big = tuple(torch.zeros((B, H, 17, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    with pytest.raises(kda.KDAError):
        call(window=big)
    with pytest.raises(ValueError):
        kda.kda_cache_load(codes, scale, None, None, n)
    with pytest.raises(TypeError):
        kda.kda_cache_store(states(1, H, 1), codes)
    with pytest.raises(TypeError):
        kda.kda_cache_store(states(1, H, 1).bfloat16())
    with pytest.raises(kda.KDAError):
        kda.kda_cache_store(states(3, H, 1), codes, scale)      # (three states, two pages)
    torch.cuda.synchronize()
