"""Windows past 2^31 elements and 2^32 bytes: decode, fold and load at their far end."""
import pytest
import torch

from cache_util import D, i32, states, token, window
from gpu_util import case, need_gpu

pytestmark = pytest.mark.gpu


def test_windows_past_32_bits():
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free memory")
    B, H, W = 1025, 1024, 16
    case(f"far windows B={B} H={H} W={W}")
    # the last state's window begins past 2^31 elements (2^32 bytes), its places among them
    assert (B - 1) * H * W * D >= 2 ** 31 and B * H < 2 ** 24
    few = (0, B - 1)
    part = states(2, H, 1)
    pw = window(2, H, W, "bf16", 2)
    small = kda.kda_cache_store(part)
    codes = torch.zeros((B, H, D, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((B, H, D), device="cuda")
    kda.kda_cache_store(part, codes, scale, i32(few))
    win = tuple(torch.zeros((B, H, W, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    pt = token(2, H, "bf16", 3)
    x = tuple(torch.zeros((B,) + y.shape[1:], dtype=y.dtype, device="cuda") for y in pt)
    for far, near in zip(win + x, pw + pt):
        far[0], far[B - 1] = near[0], near[1]
    n = torch.full((B,), 14, dtype=torch.int32, device="cuda")
    o, po = kda.kda_cache_decode(*x, codes, scale, win, n), kda.kda_cache_decode(*pt, *small, pw, n[:2].contiguous())
    S = kda.kda_cache_load(codes, scale, i32([B - 1, 0, B]), win, i32([15, 3, 1]))
    pS = kda.kda_cache_load(*small, i32([1, 0]), pw, i32([15, 3]))
    kda.kda_cache_fold(codes, scale, win, n + 1)
    kda.kda_cache_fold(*small, pw, n[:2] + 1)
    torch.cuda.synchronize()
    assert torch.equal(S[:2], pS) and (S[2] == 0).all()
    for i, b in enumerate(few):
        assert torch.equal(o[b], po[i]) and torch.equal(codes[b], small[0][i]) and torch.equal(scale[b], small[1][i])
        assert all(torch.equal(y[b], z[i]) for y, z in zip(win, pw))
        assert (pw[2][i, :, 14] != 0).any()
    for b in (1, B // 2, B - 2):        # the others are empty, and stay so
        assert (codes[b] == 0).all() and (o[b] == 0).all() and all((y[b] == 0).all() for y in win)
