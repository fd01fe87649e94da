"""Decode from 8-bit states whose key channels differ in size by anything: an output is off by
roundings of its own terms alone, as fp32 products have them, whatever the other value channels hold."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from cache_util import D, i32, states, token, window, within
from gpu_util import case, need_gpu, np_

pytestmark = pytest.mark.gpu


def decoded(kda, S, x, win, n, W):
    """kda_cache_decode of one token against the oracle, every element within its bound."""
    q, k, v, la, beta = x
    codes, scale = kda.kda_cache_store(S)
    before = [np_(y).astype(np.float64) for y in win]
    o = kda.kda_cache_decode(q, k, v, la, beta, codes, scale, win, i32(n))
    torch.cuda.synchronize()
    half = oc.HALF["f32" if q.dtype == torch.float32 else "bf16"]
    a = [np_(y).astype(np.float64) for y in x]
    c, s = codes.cpu().numpy(), scale.cpu().numpy()
    for b in range(S.shape[0]):
        for h in range(S.shape[1]):
            u, bu, output = oc.decode(*(y[b, h] for y in a), c[b, h], s[b, h], *(y[b, h] for y in before), n[b])
            held = np_(win[2][b, h, n[b]]).astype(np.float64)
            within("u", held, u, bu + half * (np.abs(u) + bu))
            ref, bo = output(held)
            within("o", np_(o[b, h]), ref, bo + half * (np.abs(ref) + bo))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [0, 8, 12, 20, 31, 38, 45, 62, 80, 100])
def test_a_large_key_channel_beside_value_channels_it_does_not_reach(power, dtype):
    kda = need_gpu()
    B, H, W = 2, 3, 4
    case(f"one channel 2^{power} times the others {dtype}")
    S = states(B, H, 1, 0.5)
    S[:, :, 37] *= 2.0 ** power
    S[:, :, 37, ::2] = 0.0
    q, k, v, la, beta = token(B, H, dtype, 2)
    win = window(B, H, W, dtype, 3)
    win[2][:, :, :, ::2] = 0.0
    v[0] = 0.0                       # (the update is then the read alone)
    decoded(kda, S, (q, k, v, la, beta), win, [0, 3], W)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("step", [10, 19, 25])
def test_value_channels_that_read_key_channels_of_their_own(step, dtype):
    """Key channels in eight groups, each 2^step under the last, each in value channels of its own: by codes, and by
    the vectors that read them, 2^-175 of the largest at the least."""
    kda = need_gpu()
    B, H, W = 2, 2, 3
    case(f"eight groups 2^{step} apart {dtype}")
    group = torch.arange(D, device="cuda") // 16
    own = (group[:, None] == torch.arange(D, device="cuda")[None] % 8).float()
    q, k, v, la, beta = token(B, H, dtype, 4)
    v = torch.zeros_like(v)
    win = tuple(torch.zeros_like(y) for y in window(B, H, W, dtype, 5))
    S = states(B, H, 6, 0.0) * own
    far = torch.exp2(50.0 - step * group.float())
    # (the store holds nothing below 2^-100)
    decoded(kda, S * torch.clamp(far, min=2.0 ** -80)[:, None], (q, k, v, la, beta), win, [0, 0], W)
    near = torch.exp2(-torch.clamp(step * group.float(), max=100.0))
    decoded(kda, S, ((q * near).to(q.dtype), (k * near).to(k.dtype), v, la, beta), win, [0, 0], W)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decayed_channels_beside_kept_ones(dtype):
    """Half of the key channels decay by e^-60 over the window, the others by nothing; each half in value channels of
    its own."""
    kda = need_gpu()
    B, H, W = 2, 3, 16
    case(f"decayed beside kept {dtype}")
    S = states(B, H, 7, 0.0)
    S[:, :, ::2, 64:] = 0.0
    S[:, :, 1::2, :64] = 0.0
    q, k, v, la, beta = token(B, H, dtype, 8)
    v = torch.zeros_like(v)
    win = window(B, H, W, dtype, 9)
    win[2].zero_()
    win[1][..., ::2], win[1][..., 1::2] = -4.0, 0.0
    decoded(kda, S, (q, k, v, la, beta), win, [15, 4], W)
