"""The 8-bit cache as a serving loop uses it: prompts, decode with folds, what a
conversation costs in exactness, graphs, streams."""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import cache as oc
from cache_util import D, DT, i32, states, token, window, within
from gpu_util import case, need_gpu, np_

pytestmark = pytest.mark.gpu


def empty_window(B, H, W, dtype):
    return tuple(torch.zeros((B, H, W, D), dtype=DT[dtype], device="cuda") for _ in range(3))


@pytest.mark.parametrize("dtype,W,steps", [("f32", 4, 13), ("f32", 1, 5), ("bf16", 8, 20)])
def test_a_conversation_stays_near_the_fp32_cache(dtype, W, steps):
    """A prompt's state stored, tokens decoded with a fold every W, against
    kda_decode_step on the fp32 state.  (I - beta k k^T) Diag(alpha) lengthens
    nothing where |k| <= 1, so what a fold (or the store) rounds away, and what
    an update's rounding to dt leaves out, is at most added up: the states are
    within the sum of the halves of the steps."""
    kda = need_gpu()
    B, H = 3, 5
    case(f"conversation {dtype} W={W} steps={steps}")
    d = kda_inputs.prefill_inputs(60, H, dtype=dtype, device="cuda", seed=1, lengths=[20, 7, 33])
    _, S = kda.kda_chunk_fwd(*(d[x] for x in ("q", "k", "v", "log_alpha", "beta")), cu_seqlens=d["cu_seqlens"])
    codes, scale = kda.kda_cache_store(S)
    win = empty_window(B, H, W, dtype)
    n = torch.zeros(B, dtype=torch.int32, device="cuda")

    def half_steps():
        # Frobenius norm of half a step everywhere (and a little for fp32 roundings)
        return (np_(scale).astype(np.float64) ** 2).sum(-1) ** 0.5 * 0.501 * np.sqrt(D)

    drift = half_steps()
    half = oc.HALF[dtype]
    for t in range(steps):
        x = token(B, H, dtype, 100 + t)
        o = kda.kda_cache_decode(*x, codes, scale, win, n)
        ref = kda.kda_decode_step(*x, S)
        u = np.linalg.norm(np_(win[2])[np.arange(B), :, np_(n)].astype(np.float64), axis=-1)
        klen = np.linalg.norm(np_(x[1]).astype(np.float64), axis=-1)
        assert (klen <= 1 + 2 ** -7).all()
        drift = drift * np.maximum(klen, 1) ** 2 + half * u * klen
        # o = S^T q, each rounded to dt; fp32 sums of 128 products
        size = np.linalg.norm(np_(ref).astype(np.float64), axis=-1) + drift
        far = np.linalg.norm(np_(o).astype(np.float64) - np_(ref).astype(np.float64), axis=-1)
        qlen = np.linalg.norm(np_(x[0]).astype(np.float64), axis=-1)
        norm_S = np.linalg.norm(np_(S).astype(np.float64).reshape(B, H, -1), axis=-1)
        assert (far <= qlen * drift + 2 * half * size + 64 * oc.EPS * qlen * norm_S).all(), (t, far / (qlen * drift))
        n = (n + 1) % W
        if (t + 1) % W == 0:
            kda.kda_cache_fold(codes, scale, win)
            drift = drift + half_steps()
    S8 = kda.kda_cache_load(codes, scale, None, win, n)
    far = np.linalg.norm((np_(S8).astype(np.float64) - np_(S)).reshape(B, H, -1), axis=-1)
    print(f"    state off by {far.max() / norm_S.min():.2e} of its size, bound {drift.max() / norm_S.min():.2e}")
    assert (far <= drift + 64 * oc.EPS * norm_S).all()


def test_a_decayed_state_keeps_its_codes():
    """Tokens that write nothing: folds only move the scales, by the decay."""
    kda = need_gpu()
    B, H, W = 2, 3, 8
    case("folds of decay alone")
    codes, scale = kda.kda_cache_store(states(B, H, 2))
    c0, s0 = codes.clone(), scale.double()
    win = list(window(B, H, W, "bf16", 3))
    win[2] = torch.zeros_like(win[2])
    for _ in range(20):
        kda.kda_cache_fold(codes, scale, win)
        s0 = s0 * torch.exp(win[1].double().sum(2))
    torch.cuda.synchronize()
    held = (s0 * 127 > 2.0 ** -99)
    assert torch.equal(codes.masked_fill(~held[..., None, :], 0), c0.masked_fill(~held[..., None, :], 0))
    # 20 folds: the decay to 8 * |G| + 8 roundings, the scale anew to two
    bound = 20 * oc.EPS * (9 * win[1].double().sum(2).abs() + 12) * s0
    within("scales", np_(scale * held), np_((s0 * held).float()).astype(np.float64), np_(bound) + 2 ** -24 * np_(s0))


def test_prefix_pages_restored_and_continued():
    """Snapshots of a prefill into pages, two requests restored from one of
    them and continued to the next snapshot, a third restored from that one:
    the first two get the same bits, the third the same state up to what the
    pages leave out."""
    kda = need_gpu()
    H, T = 4, 96
    case("prefix pages")
    d = kda_inputs.prefill_inputs(T, H, dtype="bf16", device="cuda", seed=5)
    x = tuple(d[n] for n in ("q", "k", "v", "log_alpha", "beta"))
    _, _, snap, _ = kda.kda_chunk_fwd_snap(*x, interval=32)
    codes = torch.zeros((8, H, D, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((8, H, D), device="cuda")
    kda.kda_cache_store(snap, codes, scale, i32([6, 1, 4]))
    h0 = kda.kda_cache_load(codes, scale, i32([1, 1, 4]))
    assert torch.equal(h0[0], h0[1])
    cu = i32([0, 32, 64, 64])
    more = tuple(torch.cat([y[64:], y[64:]]) for y in x)
    _, hT = kda.kda_chunk_fwd(*more, h0=h0, cu_seqlens=cu)
    c, s = kda.kda_cache_store(hT)
    win = empty_window(3, H, 4, "bf16")
    t = tuple(y[:1].expand(3, *y.shape[1:]).contiguous() for y in token(1, H, "bf16", 6))
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    o = kda.kda_cache_decode(*t, c, s, win, n)
    torch.cuda.synchronize()
    assert torch.equal(o[0], o[1])
    # half a step everywhere of each of the two pages; the prefill's bf16 products: 2e-2 of the state, as its own tests have it
    off = np_(hT[0]).astype(np.float64) - np_(hT[2])
    halves = sum(0.501 * np.sqrt(D * (np_(scale[p]).astype(np.float64) ** 2).sum()) for p in (1, 4))
    assert np.linalg.norm(off) <= halves + 2e-2 * np.linalg.norm(np_(hT[2])), (np.linalg.norm(off), halves)
    a = [np_(y).astype(np.float64) for y in t]
    zero = np.zeros((4, D))
    for h in range(H):
        u, bu, output = oc.decode(*(y[0, h] for y in a), c[0, h].cpu().numpy(), s[0, h].cpu().numpy(), zero, zero, zero, 0)
        held = np_(win[2][0, h, 0]).astype(np.float64)
        ref, bo = output(held)
        within("o", np_(o[0, h]), ref, bo + oc.HALF["bf16"] * (np.abs(ref) + bo))


def test_a_captured_loop_replays():
    """Decode, count, fold where full, in a graph: every replay against eager
    calls on a copy."""
    kda = need_gpu()
    B, H, W = 3, 4, 3
    case("graph of decode, count, fold")
    def fresh():
        codes, scale = kda.kda_cache_store(states(B, H, 7))
        return codes, scale, empty_window(B, H, W, "bf16"), i32([0, 1, 2])
    x = [y.clone() for y in token(B, H, "bf16", 0)]
    o = torch.zeros_like(x[2])

    def step(st, out):
        codes, scale, win, n = st
        kda.kda_cache_decode(*x, codes, scale, win, n, o=out)
        n.add_(1)
        full = torch.where(n >= W, n, torch.zeros_like(n))
        kda.kda_cache_fold(codes, scale, win, full)
        n.remainder_(W)

    a, b = fresh(), fresh()
    warm = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm, torch.zeros_like(o))
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, o)
    for r in range(5):
        for y, z in zip(x, token(B, H, "bf16", 30 + r)):
            y.copy_(z)
        g.replay()
        eager = torch.zeros_like(o)
        step(b, eager)
        torch.cuda.synchronize()
        assert torch.equal(o, eager), r
        for y, z in zip(a[:2] + a[2] + a[3:], b[:2] + b[2] + b[3:]):
            assert torch.equal(y, z), r


def test_two_streams_at_once():
    kda = need_gpu()
    B, H, W = 4, 8, 4
    case("two streams")
    runs = []
    for seed in (40, 41):
        codes, scale = kda.kda_cache_store(states(B, H, seed))
        runs.append([codes, scale, window(B, H, W, "bf16", seed), token(B, H, "bf16", seed)])
    n = torch.full((B,), 2, dtype=torch.int32, device="cuda")

    def go(r, fold=True):
        codes, scale, win, x = r[0].clone(), r[1].clone(), tuple(y.clone() for y in r[2]), r[3]
        o = kda.kda_cache_decode(*x, codes, scale, win, n)
        kda.kda_cache_fold(codes, scale, win, n + 1)
        return o, kda.kda_cache_load(codes, scale), win[2]

    want = [go(r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(go(r))
        torch.cuda.synchronize()
        for w, y in zip(want, got):
            assert all(torch.equal(i, j) for i, j in zip(w, y))
