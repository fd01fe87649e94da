"""What infinities of the 8-bit cache's inputs reach: as the header has it, no more and no less."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from cache_util import D, i32, states, token, window, within
from gpu_util import case, need_gpu, np_
from test_gpu_cache_range import decoded

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which,bad", [(0, INF), (0, -INF), (1, INF), (1, -INF), (3, INF)])
def test_an_infinity_makes_nan_of_its_head_alone(which, bad, dtype):
    kda = need_gpu()
    B, H, W = 2, 5, 4
    case(f"{bad} in input {which} {dtype}")
    codes, scale = kda.kda_cache_store(states(B, H, 1))
    win = window(B, H, W, dtype, 2)
    x = token(B, H, dtype, 3)
    clean = tuple(y.clone() for y in win)
    ref = kda.kda_cache_decode(*x, codes, scale, clean, i32([2, 3]))
    x[which][1, 2, 77] = bad
    o = kda.kda_cache_decode(*x, codes, scale, win, i32([2, 3]))
    torch.cuda.synchronize()
    nan, gone = torch.isnan(o), torch.isnan(win[2])
    assert nan[1, 2].all() and nan.sum() == D and torch.equal(o[~nan], ref[~nan])
    if which == 0:      # a query's reaches no update
        assert torch.equal(win[2], clean[2])
    else:
        assert gone[1, 2, 3].all() and gone.sum() == D and torch.equal(win[2][~gone], clean[2][~gone])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_minus_infinity_in_log_alpha_empties_key_channels(dtype):
    """In a window, first, between and last, and in the token itself."""
    kda = need_gpu()
    B, H, W = 3, 2, 9
    case(f"-infinity in log alpha {dtype}")
    S = states(B, H, 4)
    win = window(B, H, W, dtype, 5)
    win[1][:, :, 0, ::5] = -INF
    win[1][:, :, 3, 1::7] = -INF
    win[1][:, :, 6, 2::9] = -INF
    q, k, v, la, beta = token(B, H, dtype, 6)
    la[:, :, 3::11] = -INF
    codes, scale = kda.kda_cache_store(S)
    n = [8, 7, 4]
    got = np_(kda.kda_cache_load(codes, scale, None, win, i32(n)))
    fold = kda.kda_cache_load(*kda.kda_cache_fold(codes.clone(), scale.clone(), win, i32(n)))
    torch.cuda.synchronize()
    c, s, w = codes.cpu().numpy(), scale.cpu().numpy(), [np_(x).astype(np.float64) for x in win]
    for b in range(B):
        for h in range(H):
            ref, bound = oc.state(c[b, h], s[b, h], *(x[b, h] for x in w), n[b])
            within("S", got[b, h], ref, bound)
            step = np.abs(ref).max(-1, keepdims=True) / 127
            within("fold", np_(fold[b, h]), ref, 3 * bound.max(-1, keepdims=True) + (0.5 + 5 * 127 * oc.EPS) * step + 0 * ref)
    # every key channel of one sequence emptied by the token: the output is its own write
    la[1] = -INF
    o_before = tuple(x.clone() for x in win)
    decoded(kda, S, (q, k, v, la, beta), win, n, W)
    assert torch.equal(win[2][1, :, n[1]], (beta[1, :, None].float() * v[1].float()).to(v.dtype))
    assert torch.equal(win[1][:, :, :4], o_before[1][:, :, :4])


@pytest.mark.parametrize("which,bad", [(0, INF), (1, INF), (1, float("nan")), (2, -INF)])
def test_what_is_not_finite_in_a_window_stays_in_its_rows(which, bad):
    """Of k and log alpha one key channel's values, of u one value channel's; no other state's."""
    kda = need_gpu()
    B, H, W = 2, 3, 5
    case(f"{bad} in window {which}")
    codes, scale = kda.kda_cache_store(states(B, H, 7))
    win = window(B, H, W, "bf16", 8)
    ref = kda.kda_cache_load(codes, scale, None, win, i32([4, 5]))
    win[which][1, 1, 2, 77] = bad
    S = kda.kda_cache_load(codes, scale, None, win, i32([4, 5]))
    torch.cuda.synchronize()
    off = ~torch.isfinite(S)
    assert off[1, 1, 77].all() if which < 2 else off[1, 1, :, 77].all()
    assert off.sum() == D and torch.equal(S[~off], ref[~off])
    codes1, scale1 = kda.kda_cache_fold(codes.clone(), scale.clone(), win, i32([4, 5]))
    back = kda.kda_cache_load(codes1, scale1)
    torch.cuda.synchronize()
    lost = torch.isnan(back)
    # (a key channel with a value that is not finite reads back as NaN)
    assert lost[1, 1, 77].all() if which < 2 else lost[1, 1].all()
    assert lost.sum() == (D if which < 2 else D * D)
