"""Speculative decoding with a tree of drafted tokens over cached KDA states: what is measured, and in plain form.

A serving step of a KDA model drafts a tree of tokens per sequence (node 0 the pending token, every other node a
continuation of an earlier one), runs the layers over all nodes at once from the cached state, accepts one path against
the target's probabilities, and moves the state along that path alone:

  tree_prologue  the layer's short convolution, Swish, norms and gates, each node convolving over its own ancestors
  tree_decode    the KDA outputs of all nodes from one read of the cached state, which stays as it is
  tree_accept    the accepted path and the next token, from target and draft probabilities and given random numbers
  tree_commit    the cached state and convolution history moved along the accepted path, in place

Where `own` is false the operators are computed by elementary torch operations in 32 bits (the sums of tree_accept in
64), where it is true by the framework's entry points.
"""
import math

import torch

own = False

D = 128        # channels of a head (keys and values)
TAPS = 4       # width of the short convolution
L2_EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- the cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one user's draft of 8 nodes through one layer of 96 heads: latency
        dict(name="prologue B1 N8", op="tree_prologue", B=1, N=8, H=96, dtype="bf16", tree=True, ragged=False),
        # a serving batch of 256 requests, the batch of the decode benchmark, 16 nodes each
        dict(name="prologue B256 N16", op="tree_prologue", B=256, N=16, H=96, dtype="bf16", tree=True, ragged=False),
        # one user again: one read of 96 states
        dict(name="decode B1 N8", op="tree_decode", B=1, N=8, H=96, dtype="bf16", tree=True, ragged=False),
        # few heads, odd sizes, node counts that differ by request (some idle), fp32
        dict(name="decode B23 N21 ragged f32", op="tree_decode", B=23, N=21, H=31, dtype="f32", tree=True, ragged=True),
        # the decode benchmark's 256 x 96 states, a chain of the pending token and a 7-token draft
        dict(name="decode B256 chain 8", op="tree_decode", B=256, N=8, H=96, dtype="bf16", tree=False, ragged=False),
        # wide trees: the most nodes of a call
        dict(name="decode B64 N64", op="tree_decode", B=64, N=64, H=96, dtype="bf16", tree=True, ragged=False),
        # one user, a chain of 3 drafts with their draft probabilities: latency
        dict(name="accept B1 chain 4", op="tree_accept", B=1, N=4, V=32000, dtype="f32", tree=False, ragged=False, drafts=True),
        # a serving batch, a 7-token draft with its probabilities over a large vocabulary
        dict(name="accept B256 chain 8", op="tree_accept", B=256, N=8, V=160000, dtype="f32", tree=False, ragged=False, drafts=True),
        # drafts without probabilities (the most probable continuations), an odd vocabulary, bf16 probabilities
        dict(name="accept B48 N48 fixed bf16", op="tree_accept", B=48, N=48, V=50021, dtype="bf16", tree=True, ragged=True, drafts=False),
        # one user's accepted path
        dict(name="commit B1 N8", op="tree_commit", B=1, N=8, P=8, H=96, dtype="bf16", ragged=True, conv=True),
        # odd sizes, long paths out of large trees, fp32
        dict(name="commit B17 N40 f32", op="tree_commit", B=17, N=40, P=23, H=13, dtype="f32", ragged=True, conv=False),
        # the serving batch
        dict(name="commit B256 N8", op="tree_commit", B=256, N=8, P=8, H=96, dtype="bf16", ragged=True, conv=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree_prologue", "tree_decode", "tree_accept", "tree_commit"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype, N=_spread(rng, 1, 64), ragged=rng.random() < 0.5)
    if op == "tree_accept":
        c.update(V=_spread(rng, 500, 160000), tree=rng.random() < 0.6, drafts=rng.random() < 0.6)
        most = 256 * 8 * 160000 // (c["N"] * c["V"])      # the largest listed case's probabilities
        c["B"] = _spread(rng, 1, max(1, min(256, most)))
        return c
    c["H"] = _spread(rng, 1, 96)
    most = {"tree_prologue": 256 * 16 * 96, "tree_decode": 64 * 64 * 96}.get(op, 256 * 16 * 96) // (c["N"] * c["H"])
    c["B"] = _spread(rng, 1, max(1, min(256, most)))
    if op == "tree_commit":
        c["P"] = _spread(rng, 1, min(c["N"], 16))
        c["conv"] = rng.random() < 0.5
    else:
        c["tree"] = rng.random() < 0.7
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _tree(gen, B, N, tree):
    """Parents [B, N] of drafted trees: node 0 the root, every later node under an earlier one; a chain where `tree` is
    false.  The larger of two draws: trees of a few levels."""
    i = torch.arange(N, device="cuda")
    if not tree:
        return (i - 1).to(torch.int32).expand(B, N).contiguous()
    x = torch.rand((2, B, N), generator=gen, device="cuda").amax(0)
    return torch.minimum((x * i).long(), (i - 1).clamp(min=0)).masked_fill(i == 0, -1).to(torch.int32)


def _counts(gen, B, most, ragged):
    if not ragged:
        return None
    n = torch.randint(0, most + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = most
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    B, N, dt, op = case["B"], case["N"], DTYPES[case["dtype"]], case["op"]
    s = dict(op=op, B=B, N=N)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    if op == "tree_accept":
        V = case["V"]
        s["parent"] = _tree(gen, B, N, case["tree"])
        s["n_node"] = _counts(gen, B, N, case["ragged"])
        s["u"] = torch.rand((B, N), generator=gen, device="cuda")
        # a draft model near its target: the same logits with some noise
        p = torch.empty((B, N, V), dtype=dt, device="cuda")
        q = torch.empty((B, max(N - 1, 0), V), dtype=dt, device="cuda") if case["drafts"] else None
        tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        above = s["parent"].clamp(min=0).long()
        step = max(1, (1 << 27) // (N * V))
        for b in range(0, B, step):
            lt = normal(min(step, B - b), N, V, std=3.0)
            p[b:b + step] = torch.softmax(lt, -1).to(dt)
            a = above[b:b + step]
            if q is not None:
                lt = (lt + normal(*lt.shape, std=0.7))[:, :N - 1]
                q[b:b + step] = torch.softmax(lt, -1).to(dt)
            # a node's token: drawn from its parent's distribution (the Gumbel maximum), so siblings may coincide
            for i in range(1, N):
                row = lt[torch.arange(a.shape[0], device="cuda"), a[:, i].clamp(max=lt.shape[1] - 1)]
                g = torch.rand(row.shape, generator=gen, device="cuda").clamp(min=1e-20)
                tokens[b:b + step, i] = (row - torch.log(-torch.log(g))).argmax(-1).to(torch.int32)
        s.update(p=p, q=q, tokens=tokens)
        if not case["tree"]:
            s["parent"] = None
        return s

    H = case["H"]
    if op == "tree_commit":
        P = case["P"]
        s["P"] = P
        s["n_path"] = _counts(gen, B, P, case["ragged"])
        # distinct nodes in ascending order, as a path has them
        order = torch.rand((B, N), generator=gen, device="cuda").argsort(-1)[:, :P]
        s["path"] = order.sort(-1).values.to(torch.int32)
    else:
        s["parent"] = _tree(gen, B, N, case["tree"])
        s["n_node"] = _counts(gen, B, N, case["ragged"])
        if not case["tree"]:
            s["parent"] = None
    if op == "tree_prologue" or case.get("conv"):
        for name in ("xq", "xk", "xv"):
            s[name] = normal(B, N, H, D).to(dt)
        s["conv_state"] = normal(B, 3, TAPS - 1, H, D).to(dt)
    if op == "tree_prologue":
        s["a_raw"], s["b_raw"] = normal(B, N, H, D).to(dt), normal(B, N, H).to(dt)
        s["conv_w"], s["a_bias"] = normal(3, H, D, TAPS, std=0.5), normal(H, D)
        # (rows past a sequence's node count stay as they are)
        s["out"] = tuple(torch.zeros((B, N, H, D), dtype=dt, device="cuda") for _ in range(4)) + (
            torch.zeros((B, N, H), dtype=dt, device="cuda"),)
        return s
    for name in ("q", "k"):
        x = normal(B, N, H, D)
        s[name] = (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)).to(dt)
    s["v"] = normal(B, N, H, D).to(dt)
    # retention from almost all to almost nothing
    s["log_alpha"] = (-5.0 * torch.sigmoid(normal(B, N, H, D) - 2.0)).to(dt)
    s["beta"] = torch.sigmoid(normal(B, N, H)).to(dt)
    # a state as a running sequence has it: of the order of the values it holds
    s["S"] = torch.empty((B, H, D, D), device="cuda")
    for b in range(0, B, 32):
        s["S"][b:b + 32] = normal(min(32, B - b), H, D, D, std=0.1)
    if op == "tree_decode":
        s["o"] = torch.zeros((B, N, H, D), dtype=dt, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------

def _valid(n, B, N):
    """[B, N]: which of the N rows of a sequence count."""
    i = torch.arange(N, device="cuda")
    return (i < N).expand(B, N) if n is None else i < n[:, None]


def _parents(s):
    i = torch.arange(s["N"], device="cuda")
    p = (i - 1).expand(s["B"], s["N"]) if s["parent"] is None else s["parent"].long()
    return torch.where((p >= 0) & (p < i), p, torch.full_like(p, -1))


def _ancestors(parent):
    """[B, N, N] fp32, 1 where column j is row i itself or an ancestor of it."""
    N = parent.shape[1]
    a = torch.eye(N, device="cuda") + (parent[..., None] == torch.arange(N, device="cuda")).float()
    for _ in range(max(1, math.ceil(math.log2(max(2, N))))):
        a = (torch.matmul(a, a) > 0).float()
    return a


def _plain_prologue(s):
    B, N = s["B"], s["N"]
    parent = _parents(s)
    bi = torch.arange(B, device="cuda")[:, None]
    # ancestors 1, 2, 3 levels up; -1, -2, -3: that many inputs back in the history
    up = [torch.arange(N, device="cuda").expand(B, N)]
    for _ in range(TAPS - 1):
        a = up[-1]
        up.append(torch.where(a >= 0, parent.gather(1, a.clamp(min=0)), a - 1))
    got = []
    for t, x in enumerate((s["xq"], s["xk"], s["xv"])):
        x, w, y = x.float(), s["conv_w"][t], 0.0
        for j, a in enumerate(up):
            row = torch.where((a >= 0)[..., None, None], x[bi, a.clamp(min=0)],
                              s["conv_state"][:, t].float()[bi, (TAPS - 1 + a).clamp(0, TAPS - 2)])
            y = y + w[..., TAPS - 1 - j] * row
        y = y * torch.sigmoid(y)
        if t < 2:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) + L2_EPS)
        got.append(y)
    got.append(-5.0 * torch.sigmoid(s["a_raw"].float() + s["a_bias"]))
    got.append(torch.sigmoid(s["b_raw"].float()))
    ok = _valid(s["n_node"], B, N)
    return tuple(torch.where(ok.reshape(ok.shape + (1,) * (o.dim() - 2)), y.to(o.dtype), o) for y, o in zip(got, s["out"]))


def _plain_decode(s):
    B, N = s["B"], s["N"]
    H = s["q"].shape[2]
    heads = lambda x: x.float().transpose(1, 2).contiguous()  # noqa: E731  [B, H, N, D]
    anc = _ancestors(_parents(s))
    G = torch.matmul(anc, s["log_alpha"].float().reshape(B, N, H * D)).reshape(B, N, H, D).transpose(1, 2).contiguous()
    q, k, v, beta = heads(s["q"]), heads(s["k"]), heads(s["v"]), s["beta"].float().transpose(1, 2)
    decay = torch.exp(G)
    held, read = torch.matmul(k * decay, s["S"]), torch.matmul(q * decay, s["S"])
    U, O = torch.zeros_like(v), torch.empty_like(v)
    for i in range(N):
        # the decay from each ancestor j to node i, and what i finds of what j wrote
        kd = k * torch.exp((G[:, :, i:i + 1] - G).clamp(max=0.0)) * anc[:, None, i, :, None]
        found = (kd * k[:, :, i:i + 1]).sum(-1, keepdim=True)
        U[:, :, i] = beta[:, :, i, None] * (v[:, :, i] - held[:, :, i] - (found * U).sum(2))
        O[:, :, i] = read[:, :, i] + ((kd * q[:, :, i:i + 1]).sum(-1, keepdim=True) * U).sum(2)
    return torch.where(_valid(s["n_node"], B, N)[..., None, None], O.transpose(1, 2).to(s["o"].dtype), s["o"])


def _plain_accept(s):
    B, N, p, q = s["B"], s["N"], s["p"], s["q"]
    bi = torch.arange(B, device="cuda")
    n = torch.full((B,), N, device="cuda") if s["n_node"] is None else s["n_node"].long()
    parent, tokens, u = _parents(s), s["tokens"].long(), s["u"].double()
    at = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = torch.where(n > 0, 0, -1).int()
    m = (n > 0).long()
    # the residual at node `at`: max(p - c q, 0) of mass Z; without q, p with the refused tokens' weights gone
    c, Z = torch.zeros(B, device="cuda", dtype=torch.float64), torch.ones(B, device="cuda", dtype=torch.float64)
    gone = torch.zeros((B, p.shape[-1]), dtype=torch.bool, device="cuda") if q is None else None
    last = max(N - 2, 0)
    for i in range(1, N):
        here = (parent[:, i] == at) & (i < n)
        t = tokens[:, i]
        if q is None:
            w = p[bi, at, t].double().masked_fill(gone[bi, t], 0.0)
            ok = here & (u[:, i] * Z < w)
            gone[bi, t] |= here & ~ok
            Z = torch.where(here & ~ok, Z - w, Z)
            gone &= ~ok[:, None]
        else:
            qr = at.clamp(max=last)
            qt = q[bi, qr, t].double()
            w = (p[bi, at, t].double() - c * qt).clamp(min=0.0)
            ok = here & (u[:, i] * qt * Z < w)
            c = torch.where(here & ~ok, c + Z, c)
            Z = torch.where(here & ~ok, (p[bi, at].double() - c[:, None] * q[bi, qr].double()).clamp(min=0.0).sum(-1), Z)
        c, Z = torch.where(ok, 0.0, c), torch.where(ok, 1.0, Z)
        at = torch.where(ok, i, at)
        path[bi, m.clamp(max=N - 1)] = torch.where(ok, i, path[bi, m.clamp(max=N - 1)]).int()
        m = m + ok
    row = p[bi, at].double()
    if q is None:
        w = row.masked_fill(gone, 0.0)
    elif N > 1:
        w = (row - c[:, None] * q[bi, at.clamp(max=last)].double()).clamp(min=0.0)
        w = torch.where((c > 0)[:, None], w, row)
    else:
        w = row
    w = torch.where((w.sum(-1) > 0)[:, None], w, row)
    cum = w.cumsum(-1)
    token = (cum <= u[:, :1] * cum[:, -1:]).sum(-1)
    return path, m.int(), torch.where(n > 0, token, -1).int()


def _plain_commit(s):
    B, N, P = s["B"], s["N"], s["P"]
    bi = torch.arange(B, device="cuda")
    S, go = s["S"], _valid(s["n_path"], B, P)
    k, v, la, beta = (s[x].float() for x in ("k", "v", "log_alpha", "beta"))
    for t in range(P):
        i = s["path"][:, t].long()
        kt = k[bi, i]
        held = torch.exp(la[bi, i])[..., None] * S
        u = beta[bi, i][..., None] * (v[bi, i] - (held * kt[..., None]).sum(-2))
        S = torch.where(go[:, t, None, None, None], held + kt[..., None] * u[..., None, :], S)
    s["S"].copy_(S)
    if "conv_state" not in s:
        return s["S"]
    # the last three inputs of the history followed by the path's
    m = go.sum(-1)
    at = m[:, None] + torch.arange(TAPS - 1, device="cuda")
    node = s["path"].long().gather(1, (at - (TAPS - 1)).clamp(0, P - 1))
    for t, x in enumerate((s["xq"], s["xk"], s["xv"])):
        old = s["conv_state"][:, t]
        new = torch.where((at >= TAPS - 1)[..., None, None], x[bi[:, None], node], old[bi[:, None], at.clamp(max=TAPS - 2)])
        s["conv_state"][:, t] = new
    return s["S"], s["conv_state"]


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if not own:
        return {"tree_prologue": _plain_prologue, "tree_decode": _plain_decode, "tree_accept": _plain_accept,
                "tree_commit": _plain_commit}[op](s)
    import gated_delta_rule_27_amd as kda
    if op == "tree_prologue":
        return kda.kda_tree_prologue(s["xq"], s["xk"], s["xv"], s["a_raw"], s["b_raw"], s["conv_w"], s["a_bias"],
                                     s["parent"], s["n_node"], s["conv_state"], l2_eps=L2_EPS, out=s["out"])
    if op == "tree_decode":
        return kda.kda_tree_decode(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S"], s["parent"], s["n_node"],
                                   o=s["o"])
    if op == "tree_accept":
        return kda.kda_tree_accept(s["p"], s["q"], s["tokens"], s["u"], s["parent"], s["n_node"])
    conv = (s["xq"], s["xk"], s["xv"], s["conv_state"]) if "conv_state" in s else None
    kda.kda_tree_commit(s["k"], s["v"], s["log_alpha"], s["beta"], s["S"], s["path"], s["n_path"], conv=conv)
    return s["S"] if conv is None else (s["S"], s["conv_state"])


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    B, N, e = case["B"], case["N"], 4 if case["dtype"] == "f32" else 2
    if case["ragged"]:      # counts are uniform over 0 .. N, one sequence has them all
        N = 1 + (N - 1) / 2 if B > 1 else N
    if case["op"] == "tree_accept":
        # the one row that the next token is drawn from, and its draft row
        return {"bytes": B * case["V"] * e * (2 if case["drafts"] else 1) + B * case["N"] * 20, "flops": 3 * B * case["V"]}
    H = case["H"]
    if case["op"] == "tree_prologue":
        return {"bytes": B * N * H * (8 * D + 2) * e + B * 9 * H * D * e + 3 * H * D * 20,
                "flops": B * N * H * D * (3 * 2 * TAPS + 20)}
    if case["op"] == "tree_decode":
        return {"bytes": B * H * D * D * 4 + B * N * H * (5 * D + 1) * e,
                "flops": B * H * (N * 4 * D * D + N * (N + 1) / 2 * 2 * D if not case["tree"] else N * 4 * D * D)}
    P = 1 + (case["P"] - 1) / 2 if case["ragged"] and B > 1 else case["P"]
    conv = B * 3 * (TAPS - 1) * H * D * e * 2 if case["conv"] else 0
    return {"bytes": 2 * B * H * D * D * 4 + B * P * H * (3 * D + 1) * e + conv, "flops": B * P * H * 5 * D * D}


# ---- the definition, in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    """Token by token from the recurrence and the convolution as they are defined, each node from its parent's state."""
    op = case["op"]
    if op == "tree_accept":
        return None     # whole numbers only
    s = prepare(case, seed)
    B, N, H = s["B"], s["N"], case["H"]
    f = lambda x: x.to(torch.float64)  # noqa: E731
    if op == "tree_prologue":
        got = [f(o).clone() for o in s["out"]]
        n = [N] * B if s["n_node"] is None else s["n_node"].tolist()
        up = [[i - 1 for i in range(N)]] * B if s["parent"] is None else s["parent"].tolist()
        # rows of inputs by their place: the three of the history, then the nodes; each node's window of four
        window = torch.zeros((B, N, TAPS), dtype=torch.long)
        for b in range(B):
            before = {-1: [0, 1, 2]}
            for i in range(N):
                window[b, i] = torch.tensor(before[up[b][i]] + [3 + i])
                before[i] = window[b, i, 1:].tolist()
        window = window.cuda()
        for b in range(B):
            m = n[b]
            if m == 0:
                continue
            for t, x in enumerate((s["xq"], s["xk"], s["xv"])):
                rows = torch.cat([f(s["conv_state"][b, t]), f(x[b])])[window[b, :m]]       # [m, 4, H, D]
                y = (rows * f(s["conv_w"][t]).movedim(-1, 0)).sum(1)
                y = y / (1 + torch.exp(-y))
                got[t][b, :m] = y / torch.sqrt(y.square().sum(-1, keepdim=True) + L2_EPS) if t < 2 else y
            got[3][b, :m] = -5 / (1 + torch.exp(-(f(s["a_raw"][b, :m]) + f(s["a_bias"]))))
            got[4][b, :m] = 1 / (1 + torch.exp(-f(s["b_raw"][b, :m])))
        return tuple(got)

    def step(S, k, v, la, beta):
        S = torch.exp(la)[..., None] * S
        u = beta[..., None] * (v - (k[..., None] * S).sum(-2))
        return S + k[..., None] * u[..., None, :]

    if op == "tree_decode":
        if B * N * H > 256 * 16 * 96:
            return None
        o = f(s["o"]).clone()
        parent = _parents(s)
        group = max(1, (1 << 32) // ((N + 1) * H * D * D * 8))
        for b in range(0, B, group):
            g = slice(b, min(B, b + group))
            j = torch.arange(g.stop - g.start, device="cuda")
            held = torch.empty((N + 1, len(j), H, D, D), dtype=torch.float64, device="cuda")
            held[N] = s["S"][g]                     # (place -1: the cached state)
            for i in range(N):
                row = lambda x: f(x[g, i])  # noqa: E731
                held[i] = step(held[parent[g, i], j], row(s["k"]), row(s["v"]), row(s["log_alpha"]), row(s["beta"]))
                out = (held[i] * row(s["q"])[..., None]).sum(-2)
                ok = _valid(s["n_node"], B, N)[g, i, None, None]
                o[g, i] = torch.where(ok, out, o[g, i])
        return o

    S = torch.empty((B, H, D, D), dtype=torch.float64, device="cuda")
    n = [s["P"]] * B if s["n_path"] is None else s["n_path"].tolist()
    new = f(s["conv_state"]) if "conv_state" in s else None
    for b in range(B):
        Sb, way = f(s["S"][b]), s["path"][b, :n[b]].long()
        for i in way.tolist():
            Sb = step(Sb, f(s["k"][b, i]), f(s["v"][b, i]), f(s["log_alpha"][b, i]), f(s["beta"][b, i]))
        S[b] = Sb
        if new is not None:
            for t, x in enumerate((s["xq"], s["xk"], s["xv"])):
                new[b, t] = torch.cat([new[b, t], f(x[b])[way]])[-(TAPS - 1):]
    return S if new is None else (S, new)
