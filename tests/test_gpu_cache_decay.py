"""Windows that decay strongly: what is left of an early token is off by some roundings of its
own, however much it has decayed (the oracle's bound counts them: a decay to four of them,
whatever the sum of log alpha)."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from cache_util import DT, i32, states, window, within
from gpu_util import case, need_gpu, np_
from test_gpu_cache_range import decoded

pytestmark = pytest.mark.gpu


def strong(B, H, W, dtype, seed, kind):
    """Windows whose first tokens alone write: what is read has decayed over all the others.  |log alpha| up to 5."""
    k, la, u = window(B, H, W, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.rand(la.shape, generator=g, device="cuda")
    if kind == "strong":
        x = 4 + x
    elif kind == "mixed":            # strong ones beside ones that keep nearly all
        x = torch.where(torch.rand(la.shape, generator=g, device="cuda") < 0.7, 4.5 + 0.5 * x, 1e-3 * x)
    else:
        x = 1e-4 * x
    k[:, :, 2:] = 0.0
    u[:, :, 2:] = 0.0
    return k, (-x).to(DT[dtype]), u


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["strong", "mixed", "weak"])
@pytest.mark.parametrize("W", [5, 8, 16])
def test_what_decays_keeps_its_bits(W, kind, dtype):
    kda = need_gpu()
    B, H = 3, 4
    case(f"decays W={W} {kind} {dtype}")
    win = strong(B, H, W, dtype, 1, kind)
    codes, scale = kda.kda_cache_store(states(B, H, 2) * 2.0 ** 10)
    n = [W, W - 1, W // 2]
    S = np_(kda.kda_cache_load(codes, scale, None, win, i32(n)))
    c, s, w = codes.cpu().numpy(), scale.cpu().numpy(), [np_(x).astype(np.float64) for x in win]
    fc, fs = kda.kda_cache_fold(codes.clone(), scale.clone(), win, i32(n))
    got, fs = oc.values(fc.cpu().numpy(), fs.cpu().numpy()), fs.cpu().numpy().astype(np.float64)
    for b in range(B):
        for h in range(H):
            ref, bound = oc.state(c[b, h], s[b, h], *(x[b, h] for x in w), n[b])
            within(f"S[{b},{h}]", S[b, h], ref, bound)
            top = np.abs(ref).max(-1)
            held = top >= 2.0 ** -99
            far = bound.max(-1)
            within(f"scale[{b},{h}]", (fs[b, h] * held), top / 127 * held, (far / 127 + 2 * oc.EPS * top / 127))
            within(f"fold[{b},{h}]", got[b, h] * held[:, None], ref * held[:, None],
                   bound + ((0.5 + 4 * 127 * oc.EPS) * top / 127 + 2 * far)[:, None])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["strong", "mixed", "weak"])
@pytest.mark.parametrize("W", [6, 16])
def test_decode_of_what_has_decayed(W, kind, dtype):
    kda = need_gpu()
    B, H = 3, 4
    case(f"decode decays W={W} {kind} {dtype}")
    win = strong(B, H, W, dtype, 3, kind)
    q, la, _ = (x[:, :, 0].contiguous() for x in strong(B, H, 1, dtype, 4, kind))
    k = strong(B, H, 1, dtype, 6, kind)[0][:, :, 0].contiguous()
    v, beta = torch.zeros_like(q), torch.full((B, H), 0.5, dtype=DT[dtype], device="cuda")
    decoded(kda, states(B, H, 8) * 2.0 ** 10, (q, k, v, la, beta), win, [W - 1, W // 2, 0], W)
