"""Serving from an 8-bit cache of KDA states, and sampling: what is measured, and in plain form.

A serving step of a KDA model reads and writes the 128 x 128 fp32 state of every head for every token.  Here the cache
holds them in 8 bits, a scale per key channel, with the last few tokens' rank-one updates beside it as a window:

  cache_store   fp32 states (a prompt's last one, prefix snapshots) quantised into pages of the cache
  cache_load    pages read back into fp32 states, the window's updates applied
  cache_decode  one token per sequence: its output from one read of the 8-bit state and the window, its update appended
  cache_fold    a window's updates taken into the 8-bit state, in place
  sample        the next token from the logits by temperature, top-k, top-p, min-p and given random numbers, and the
                probabilities that are left (what the verification of drafts takes as the target's and the drafts')

Where `own` is false the operators are computed by elementary torch operations in 32 bits (the sums of sample in 64),
where it is true by the framework's entry points.  States come back as the values that codes and scales stand for.
"""
import math

import numpy as np
import torch

own = False

D = 128        # channels of a head (keys and values)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -100     # a row without anything larger is held as zeros


# ---- the cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one prompt has ended: its 96 heads' states into the cache
        dict(name="store B1", op="cache_store", B=1, H=96, paged=False),
        # prefix snapshots of a long prefill into pages, some of them not kept
        dict(name="store B256 pages", op="cache_store", B=256, H=96, paged=True),
        # a few requests that continue a conversation: few heads, odd sizes, fp32 windows of their own lengths
        dict(name="load B7 H31 window f32", op="cache_load", B=7, H=31, W=11, dtype="f32", paged=True, window=True),
        # a batch of requests restored from prefix pages, several from the same one
        dict(name="load B192 pages", op="cache_load", B=192, H=96, W=1, dtype="bf16", paged=True, window=False),
        # one user's token through one layer of 96 heads: latency
        dict(name="decode B1 W8", op="cache_decode", B=1, H=96, W=8, dtype="bf16", ragged=False),
        # few heads, odd sizes, windows of every length, some places of the batch idle, fp32
        dict(name="decode B23 H31 W13 f32", op="cache_decode", B=23, H=31, W=13, dtype="f32", ragged=True),
        # the decode benchmark's 256 x 96 states
        dict(name="decode B256 W8", op="cache_decode", B=256, H=96, W=8, dtype="bf16", ragged=True),
        # a small batch's windows, each as full as it happens to be
        dict(name="fold B5 H31 W16", op="cache_fold", B=5, H=31, W=16, dtype="bf16", ragged=True),
        # the serving batch's, every eight tokens
        dict(name="fold B256 W8", op="cache_fold", B=256, H=96, W=8, dtype="bf16", ragged=False),
        # one user's next token
        dict(name="sample R1 V32000 k p", op="sample", R=1, V=32000, dtype="f32", k=True, p=True, m=False, flat=False, probs=False),
        # a serving batch's, a large vocabulary, by mass alone
        dict(name="sample R256 V160000 p", op="sample", R=256, V=160000, dtype="f32", k=False, p=True, m=False, flat=False, probs=False),
        # a draft step: tokens and the distributions they are drawn from, for their verification; an odd vocabulary
        dict(name="sample R192 V50021 k p m probs bf16", op="sample", R=192, V=50021, dtype="bf16", k=True, p=True, m=True, flat=True, probs=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["cache_store", "cache_load", "cache_decode", "cache_decode", "cache_fold", "sample", "sample"])
    c = dict(op=op)
    if op == "sample":
        c.update(V=_spread(rng, 500, 160000), dtype=rng.choice(["bf16", "f32"]))
        c["R"] = _spread(rng, 1, max(1, min(2048, 192 * 50021 // c["V"])))
        c.update({x: rng.random() < 0.5 for x in ("k", "p", "m", "flat", "probs")})
        return c
    c["H"] = _spread(rng, 1, 96)
    c["B"] = _spread(rng, 1, max(1, min(256, 192 * 96 // c["H"])))
    if op in ("cache_store", "cache_load"):
        c["paged"] = rng.random() < 0.6
    if op != "cache_store":
        c.update(W=_spread(rng, 1, 16), dtype=rng.choice(["bf16", "bf16", "f32"]))
        c["window" if op == "cache_load" else "ragged"] = rng.random() < 0.6
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(op=op)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)

    if op == "sample":
        R, V = case["R"], case["V"]
        # many unlikely tokens; where the row is not flat, a few that hold most of its mass, as a language model has it
        x = torch.empty((R, V), dtype=DTYPES[case["dtype"]], device="cuda")
        step = max(1, (1 << 27) // V)
        for r in range(0, R, step):
            n = min(step, R - r)
            l = normal(n, V, std=2.5)
            if not case["flat"]:
                at = torch.randint(0, V, (n, 48), generator=gen, device="cuda")
                l.scatter_(1, at, torch.logsumexp(l, 1, keepdim=True) + 1.0 + 2.0 * normal(n, 48) - 2.0 * uniform(n, 1))
            x[r:r + n] = l.to(x.dtype)
        s.update(logits=x, u=uniform(R), temperature=0.5 + 0.8 * uniform(R), top_k=None, top_p=None, min_p=None)
        s["temperature"][whole(0, 16, R) == 0] = 0.0        # greedy requests
        if case["k"]:
            s["top_k"] = whole(1, 201, R) * (whole(0, 8, R) > 0)      # (some requests without)
        if case["p"]:
            s["top_p"] = 0.5 + 0.5 * uniform(R)
        if case["m"]:
            s["min_p"] = 0.1 * uniform(R)
        s["token"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty_like(x) if case["probs"] else None
        return s

    B, H = case["B"], case["H"]
    s.update(B=B, H=H)

    def states(n):
        # rows as decays leave them: of very different size
        S = torch.empty((n, H, D, D), device="cuda")
        for b in range(0, n, 32):
            m = min(32, n - b)
            S[b:b + m] = normal(m, H, D, D) * 0.1 * torch.exp(normal(m, H, D, 1))
        return S

    if op in ("cache_store", "cache_load"):
        pages = B + 3 if case["paged"] else B
        s["page"] = None
        if case["paged"]:
            order = uniform(pages).argsort().to(torch.int32)
            s["page"] = order[:B].clone()
            if op == "cache_load":      # some requests share a prefix
                s["page"] = torch.where(whole(0, 4, B) == 0, order[whole(0, B, B).long()], s["page"])
            if B > 1:                   # one has none
                s["page"][B // 2] = -1
    else:
        pages = B
    if op == "cache_store":
        s["S"] = states(B)
        s["codes"] = torch.zeros((pages, H, D, D), dtype=torch.int8, device="cuda")
        s["scale"] = torch.zeros((pages, H, D), device="cuda")
        return s
    s["codes"] = torch.empty((pages, H, D, D), dtype=torch.int8, device="cuda")
    s["scale"] = torch.empty((pages, H, D), device="cuda")
    for b in range(0, pages, 32):
        s["codes"][b:b + 32], s["scale"][b:b + 32] = _quantised(states(min(32, pages - b)))

    W, dt = case["W"], DTYPES[case["dtype"]]
    s["W"] = W

    def unit(*shape):
        x = normal(*shape, D)
        return (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)).to(dt)

    def decay(*shape):
        # retention from almost all to almost nothing
        return (-5.0 * torch.sigmoid(normal(*shape, D) - 2.0)).to(dt)

    s["window"] = s["n_win"] = None
    if op != "cache_load" or case["window"]:
        s["window"] = (unit(pages, H, W), decay(pages, H, W), (0.5 * normal(pages, H, W, D)).to(dt))
    if op == "cache_load":
        s["S"] = torch.zeros((B, H, D, D), device="cuda")
        if case["window"]:
            s["n_win"] = whole(0, W + 1, B)
        return s
    if op == "cache_fold":
        s["n_win"] = whole(0, W + 1, B) if case["ragged"] else torch.full((B,), W, dtype=torch.int32, device="cuda")
        return s
    s["n_win"] = whole(0, W, B) if case["ragged"] else torch.full((B,), W // 2, dtype=torch.int32, device="cuda")
    if case["ragged"] and B > 1:
        s["n_win"][B // 2] = -1         # an idle place of the batch
    s["q"], s["k"], s["log_alpha"] = unit(B, H), unit(B, H), decay(B, H)
    s["v"], s["beta"] = normal(B, H, D).to(dt), torch.sigmoid(normal(B, H)).to(dt)
    s["o"] = torch.zeros((B, H, D), dtype=dt, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _quantised(S):
    """Codes [.., value channel, key channel] and scales [.., key channel] of states [.., key, value]."""
    top = S.abs().amax(-1)
    held = top >= TINY
    scale = torch.where(held, top / 127.0, torch.zeros_like(top))
    inverse = torch.where(held, 127.0 / top, torch.zeros_like(top))
    codes = torch.round(S * inverse[..., None]).clamp(-127, 127).to(torch.int8)
    return codes.transpose(-1, -2).contiguous(), scale


def _values(codes, scale):
    """What codes and scales stand for, [.., value channel, key channel], in bf16."""
    return codes * scale[..., None, :].to(torch.bfloat16)


def _window(s, n, window):
    """For the first n[b] tokens of each window: the decay over all of them [B, H, D], their keys as far as they are
    decayed after the last one [B, H, W, D], and their updates."""
    k, la, u = (x.float() for x in window)
    ok = (torch.arange(s["W"], device="cuda") < n[:, None])[:, None, :, None]
    la = torch.where(ok, la, torch.zeros_like(la))
    left = la.flip(2).cumsum(2).flip(2)             # from each token on
    after = torch.cat([left[:, :, 1:], torch.zeros_like(left[:, :, :1])], 2)
    zero = torch.zeros_like(k)
    return torch.exp(left[:, :, 0]), torch.where(ok, k * torch.exp(after), zero), torch.where(ok, u, zero)


def _with_window(s, codes, scale, n, window):
    """fp32 states [B, H, key, value]."""
    S = codes.transpose(-1, -2).float() * scale[..., None]
    if window is None:
        return S
    decay, k, u = _window(s, n, window)
    return S * decay[..., None] + torch.matmul(k.transpose(-1, -2).contiguous(), u)


def _plain_store(s):
    codes, scale = _quantised(s["S"])
    if s["page"] is None:
        s["codes"].copy_(codes)
        s["scale"].copy_(scale)
        return
    pages = torch.arange(s["codes"].shape[0], device="cuda")
    hit = s["page"][None] == pages[:, None]         # [page, state]
    at, named = hit.int().argmax(1), hit.any(1)
    s["codes"].copy_(torch.where(named[:, None, None, None], codes[at], s["codes"]))
    s["scale"].copy_(torch.where(named[:, None, None], scale[at], s["scale"]))


def _plain_load(s):
    if s["page"] is None:
        return _with_window(s, s["codes"], s["scale"], s["n_win"], s["window"])
    at = s["page"].clamp(min=0).long()
    window = None if s["window"] is None else tuple(x[at] for x in s["window"])
    S = _with_window(s, s["codes"][at], s["scale"][at], s["n_win"], window)
    return torch.where((s["page"] >= 0)[:, None, None, None], S, s["S"])


def _plain_decode(s):
    B, W, n = s["B"], s["W"], s["n_win"]
    q, k, v, la = (s[x].float() for x in ("q", "k", "v", "log_alpha"))
    decay, kw, uw = _window(s, n, s["window"])
    now = torch.exp(la)
    P = s["codes"].transpose(-1, -2).float() * s["scale"][..., None]
    held = torch.matmul(torch.stack([k, q], 2) * (decay * now)[:, :, None], P)         # [B, H, 2, value]
    kw = kw * now[:, :, None]
    held = held + torch.matmul((torch.stack([k, q], 2)[:, :, :, None] * kw[:, :, None]).sum(-1), uw)
    u = (s["beta"].float()[..., None] * (v - held[:, :, 0])).to(s["v"].dtype)
    o = held[:, :, 1] + (k * q).sum(-1, keepdim=True) * u.float()
    ok = (n >= 0) & (n < W)
    s["o"].copy_(torch.where(ok[:, None, None], o.to(u.dtype), s["o"]))
    row = (torch.arange(W, device="cuda") == n[:, None])[:, None, :, None]
    for x, new in zip(s["window"], (s["k"], s["log_alpha"], u)):
        x.copy_(torch.where(row, new[:, :, None], x))


def _plain_fold(s):
    codes, scale = _quantised(_with_window(s, s["codes"], s["scale"], s["n_win"], s["window"]))
    some = s["n_win"] > 0
    s["codes"].copy_(torch.where(some[:, None, None, None], codes, s["codes"]))
    s["scale"].copy_(torch.where(some[:, None, None], scale, s["scale"]))


def _plain_sample(s):
    l, T = s["logits"].float(), s["temperature"].double()[:, None]
    R, V = l.shape
    l, order = torch.sort(l, dim=-1, descending=True, stable=True)
    rank = torch.arange(V, device="cuda")
    x = (l - l[:, :1].double()) / torch.where(T > 0, T, 1.0)
    w = torch.exp(x)
    keep = (T > 0) | (rank == 0)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((k < 1) | (rank < k))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cum = (w * keep).cumsum(-1)
        # the smallest leading set that reaches its share: those before which it was not reached
        before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], -1)
        keep = keep & ((p >= 1) | (before < p * cum[:, -1:]))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    w = torch.empty_like(w).scatter_(1, order, w * keep)
    cum = w.cumsum(-1)
    s["token"].copy_((cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(-1))
    if s["probs"] is not None:
        s["probs"].copy_(w / cum[:, -1:])


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        import gated_delta_rule_27_amd as kda
        if op == "cache_store":
            kda.kda_cache_store(s["S"], s["codes"], s["scale"], s["page"])
        elif op == "cache_load":
            return kda.kda_cache_load(s["codes"], s["scale"], s["page"], s["window"], s["n_win"], S=s["S"])
        elif op == "cache_decode":
            kda.kda_cache_decode(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["codes"], s["scale"], s["window"],
                                 s["n_win"], o=s["o"])
        elif op == "cache_fold":
            kda.kda_cache_fold(s["codes"], s["scale"], s["window"], s["n_win"])
        else:
            kda.kda_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], token=s["token"],
                           probs=s["probs"])
    elif op == "cache_load":
        return _plain_load(s)
    else:
        {"cache_store": _plain_store, "cache_decode": _plain_decode, "cache_fold": _plain_fold, "sample": _plain_sample}[op](s)
    if op == "sample":
        return s["token"] if s["probs"] is None else (s["token"], s["probs"])
    if op == "cache_decode":
        return (s["o"],) + s["window"]
    return _values(s["codes"], s["scale"]), s["scale"]


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "sample":
        # the logits once, the probabilities once
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["R"] * case["V"] * e * (2 if case["probs"] else 1) + case["R"] * 24, "flops": case["R"] * case["V"] * 4}
    units, packed, values = case["B"] * case["H"], D * D + 4 * D, 2 * D * D
    if op == "cache_store":
        return {"bytes": units * (4 * D * D + packed + values), "flops": units * 3 * D * D}
    W, e = case["W"], 4 if case["dtype"] == "f32" else 2
    if op == "cache_load":
        n = W / 2 if case["window"] else 0
        return {"bytes": units * (packed + 4 * D * D + n * 3 * D * e), "flops": units * (1 + 2 * n) * D * D}
    if op == "cache_fold":
        n = W / 2 if case["ragged"] else W
        return {"bytes": units * (2 * packed + values + n * 3 * D * e), "flops": units * (4 + 2 * n) * D * D}
    n = (W - 1) / 2 if case["ragged"] else W // 2
    return {"bytes": units * (packed + n * 3 * D * e + (8 * D + 1) * e), "flops": units * (4 * D * D + n * 8 * D)}


# ---- the definition, in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    """States step by step through the window's tokens; samples row by row on the host."""
    op, s = case["op"], prepare(case, seed)
    if op == "sample":
        R, V = case["R"], case["V"]
        if R * V > 192 * 160000:
            return None
        host = lambda x, none: np.full(R, none) if x is None else x.cpu().numpy().astype(np.float64)  # noqa: E731
        l = s["logits"].float().cpu().numpy().astype(np.float64)
        u, T, k, p, m = host(s["u"], 0.0), host(s["temperature"], 1.0), host(s["top_k"], 0.0), host(s["top_p"], 1.0), host(s["min_p"], 0.0)
        token, probs = np.zeros(R, np.int32), np.zeros((R, V) if case["probs"] else 0)
        for r in range(R):
            first = np.argsort(-l[r], kind="stable")
            w = np.exp((l[r, first] - l[r, first[0]]) / (T[r] if T[r] > 0 else 1.0))
            n = 1 if T[r] == 0 else V if k[r] < 1 else min(V, int(k[r]))
            if p[r] < 1:
                n = min(n, 1 + int(np.searchsorted(np.cumsum(w[:n]), p[r] * w[:n].sum())))
            kept = np.zeros(V)
            kept[first[:n]] = np.where(w[:n] >= m[r], w[:n], 0.0)
            cum = np.cumsum(kept)
            token[r] = np.searchsorted(cum, u[r] * cum[-1], side="right")
            if case["probs"]:
                probs[r] = kept / cum[-1]
        return (token, probs) if case["probs"] else token

    f = lambda x: x.to(torch.float64)  # noqa: E731
    B, H = case["B"], case["H"]
    S = f(s["codes"]).transpose(-1, -2) * f(s["scale"])[..., None] if op != "cache_store" else None

    def through(S, n, window, t, b):
        """States S of the places b whose windows hold a token t."""
        i = torch.nonzero(n > t).flatten().tolist()
        k, la, u = (f(x[b[i], :, t]) for x in window)
        S[i] = S[i] * torch.exp(la)[..., None] + k[..., None] * u[:, :, None]

    if op == "cache_load":
        page = torch.arange(B, device="cuda") if s["page"] is None else s["page"].long()
        got = S[page.clamp(min=0)].clone()
        if case["window"]:
            for t in range(case["W"]):
                through(got, s["n_win"], s["window"], t, page.clamp(min=0))
        got[page < 0] = f(s["S"])[page < 0]
        return got
    every = torch.arange(B, device="cuda")
    if op == "cache_decode":
        for t in range(case["W"]):
            through(S, s["n_win"], s["window"], t, every)
        S = S * torch.exp(f(s["log_alpha"]))[..., None]
        u = f(s["beta"])[..., None] * (f(s["v"]) - (S * f(s["k"])[..., None]).sum(-2))
        # (the update is held, and read, in the type of the inputs)
        u = f(u.to(s["v"].dtype))
        S = S + f(s["k"])[..., None] * u[:, :, None]
        ok = (s["n_win"] >= 0)[:, None, None]
        got = [torch.where(ok, (S * f(s["q"])[..., None]).sum(-2), f(s["o"]))]
        at = torch.nonzero(s["n_win"] >= 0).flatten()
        for x, new in zip(s["window"], (f(s["k"]), f(s["log_alpha"]), u)):
            x = f(x).clone()
            x[at, :, s["n_win"][at].long()] = new[at]
            got.append(x)
        return tuple(got)
    if op == "cache_fold":
        old = S.clone()
        for t in range(case["W"]):
            through(S, s["n_win"], s["window"], t, every)
    else:
        S = f(s["S"])
    top = S.abs().amax(-1, keepdim=True)
    scale = torch.where(top >= TINY, top / 127.0, 0.0 * top)
    S = torch.where(top >= TINY, torch.round(S / torch.where(top >= TINY, scale, 1.0)) * scale, 0.0 * S)
    S, scale = S.transpose(-1, -2).contiguous(), scale[..., 0]
    if op == "cache_fold":
        idle = s["n_win"] <= 0
        S[idle], scale[idle] = old[idle].transpose(-1, -2), f(s["scale"])[idle]
        return S, scale
    if s["page"] is None:
        return S, scale
    pool, pool_scale = f(s["codes"]), f(s["scale"])
    at = torch.nonzero(s["page"] >= 0).flatten()
    pool[s["page"][at].long()], pool_scale[s["page"][at].long()] = S[at], scale[at]
    return pool, pool_scale
