"""The calls of tree speculative decoding as a serving step makes them: one
layer's prologue, decode, epilogue, acceptance and commit in a row, in a
captured graph, on two streams at once; and their refusals and largest sizes.

Tolerances.  Committed states against token-by-token steps from the same
bits: fp32 on both sides, 1e-4 normwise as for every fp32 result here.
Outputs: both sides are rounded once to the output type (half a step each),
2 * (eps / 2) + 1e-4.
"""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import tree as otree
from gpu_util import case, nerr, need_gpu, np_
from tree_util import SENTINEL, i32, node_inputs, random_trees

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Step:
    """The buffers and weights of one layer over B trees of N nodes, its
    cached state, and the calls of one step on them."""

    def __init__(self, kda, B, N, H, V, dtype, seed):
        self.kda, self.B, self.N, self.H, self.V = kda, B, N, H, V
        d = kda_inputs.layer_inputs(B * N, H, dtype=dtype, device="cuda", seed=seed, lengths=[N] * B,
                                    conv_state=True)
        self.conv_w, self.a_bias, self.hist = d["conv_w"], d["a_bias"], d["conv_state"]
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.S = rand(B, H, 128, 128) * 0.1
        self.norm_w = 1 + 0.1 * rand(H, 128)
        # a token's inputs of the layer, and what its output says of the next token
        self.table = {n: (rand(V, H, 128) * s).to(DT[dtype]) for n, s in
                      (("xq", 1), ("xk", 1), ("xv", 1), ("a", 2), ("g", 1))}
        self.table["b"] = rand(V, H).to(DT[dtype])
        self.head = rand(H * 128, V) * (2.0 / (H * 128) ** 0.5)
        self.x = {n: torch.zeros((B, N) + t.shape[1:], dtype=t.dtype, device="cuda")
                  for n, t in self.table.items()}
        self.tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        self.parent = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        self.count = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.u = torch.zeros((B, N), device="cuda")
        self.q = torch.zeros((B, N - 1, V), device="cuda")
        # (rows past a sequence's nodes stay as they are here)
        self.out = tuple(torch.zeros_like(self.x["xq"]) for _ in range(4)) + (torch.zeros_like(self.x["b"]),)
        self.o = torch.zeros_like(self.x["xq"])
        self.y = torch.zeros_like(self.x["xq"])
        self.p = torch.zeros((B, N, V), device="cuda")
        self.path = torch.empty_like(self.tokens)
        self.m = torch.empty_like(self.count)
        self.next = torch.empty_like(self.count)

    def draft(self, seed, pending):
        """A tree per sequence: parents, counts, tokens drawn from q, u."""
        rng = np.random.default_rng(seed)
        B, N, V = self.B, self.N, self.V
        par = random_trees(B, N, seed)
        count = rng.integers(1, N + 1, size=B)
        count[0] = N
        q = rng.dirichlet(np.full(V, 0.3), size=(B, N - 1)).astype(np.float32)
        tok = np.zeros((B, N), dtype=np.int32)
        tok[:, 0] = pending
        for b in range(B):
            for i in range(1, N):
                tok[b, i] = rng.choice(V, p=q[b, par[b, i]].astype(np.float64) / q[b, par[b, i]].sum(dtype=np.float64))
        self.host = par, count, tok, q, rng.random((B, N)).astype(np.float32)
        self.parent.copy_(i32(par))
        self.count.copy_(i32(count))
        self.tokens.copy_(i32(tok))
        self.q.copy_(torch.from_numpy(q))
        self.u.copy_(torch.from_numpy(self.host[4]))
        for n, t in self.table.items():
            self.x[n].copy_(t[self.tokens.long()])

    def layer(self):
        x, kda, T = self.x, self.kda, (self.B * self.N, self.H, 128)
        kda.kda_tree_prologue(x["xq"], x["xk"], x["xv"], x["a"], x["b"], self.conv_w, self.a_bias, self.parent,
                              self.count, self.hist, out=self.out)
        kda.kda_tree_decode(*self.out, self.S, self.parent, self.count, o=self.o)
        kda.kda_epilogue(self.o.view(T), x["g"].view(T), self.norm_w, y=self.y.view(T))

    def predict(self):
        z = self.y.float().view(self.B, self.N, -1) @ self.head
        self.p.copy_(torch.softmax(z.double(), -1))

    def finish(self):
        x, kda = self.x, self.kda
        kda.kda_tree_accept(self.p, self.q, self.tokens, self.u, self.parent, self.count, path=self.path,
                            n_path=self.m, next_token=self.next)
        kda.kda_tree_commit(*self.out[1:], self.S, self.path, self.m,
                            conv=(x["xq"], x["xk"], x["xv"], self.hist))


@pytest.mark.parametrize("dtype,B,N,H,V", [("f32", 4, 7, 2, 50), ("bf16", 3, 13, 3, 33), ("bf16", 2, 40, 2, 200)])
def test_steps_follow_the_tokens_one_by_one(dtype, B, N, H, V):
    """Three steps; after each, states and histories are those of the emitted
    tokens run one by one, the accepted nodes' outputs theirs, and the walk
    the oracle's on the same probabilities."""
    kda = need_gpu()
    case(f"tree steps {dtype} B={B} N={N} H={H} V={V}")
    t = Step(kda, B, N, H, V, dtype, 5)
    ref_S, ref_hist = t.S.clone(), t.hist.clone()
    pending, taken = np.arange(B) % V, 0
    tol = torch.finfo(DT[dtype]).eps + 1e-4
    for step in range(3):
        t.draft(60 + step, pending)
        par, count, tok, q, u = t.host
        t.layer()
        t.predict()
        t.finish()
        torch.cuda.synchronize()
        path, m, nxt = t.path.cpu().numpy(), t.m.cpu().numpy(), t.next.cpu().numpy()
        p = np_(t.p)
        for b in range(B):
            way, token, margin = otree.accept(p[b], q[b], tok[b], u[b], par[b], int(count[b]))
            assert margin > 1e-12, "the case has no answer to compare"
            assert path[b, :m[b]].tolist() == way and nxt[b] == token, b
            for i in way:   # the layer, a token at a time
                one = {n: x[b, i:i + 1].contiguous() for n, x in t.x.items()}
                q1, k1, v1, la1, b1, h1 = kda.kda_prologue(
                    one["xq"], one["xk"], one["xv"], one["a"], one["b"], t.conv_w, t.a_bias,
                    conv_state=ref_hist[b:b + 1].contiguous())
                ref_hist[b] = h1[0]
                S1 = ref_S[b:b + 1].contiguous()
                o1 = kda.kda_decode_step(q1, k1, v1, la1, b1, S1)
                ref_S[b] = S1[0]
                assert nerr(np_(t.o[b, i]), np_(o1[0])) <= tol, (step, b, i)
            taken += len(way)
        torch.cuda.synchronize()
        assert torch.equal(t.hist, ref_hist), "the histories are copies of inputs"
        assert nerr(np_(t.S), np_(ref_S)) <= 1e-4, step
        pending = nxt
    print(f"    {taken} tokens in 3 steps of {B} sequences", flush=True)
    assert taken > 3 * B   # (some drafts were accepted)


def _snapshot(t):
    torch.cuda.synchronize()
    return [x.clone() for x in (t.o, t.y, t.S, t.hist, t.path, t.m, t.next, *t.out)]


@pytest.mark.parametrize("dtype,N", [("bf16", 8), ("f32", 20), ("bf16", 64)])
def test_captured_steps_replay_as_eager_ones(dtype, N):
    """The five calls in one graph, replayed on new drafts; the state moves on
    with every replay.  The same steps made eagerly in between give the same
    bits."""
    kda = need_gpu()
    B, H, V = 5, 3, 70
    case(f"captured tree step {dtype} N={N}")
    t, e = Step(kda, B, N, H, V, dtype, 8), Step(kda, B, N, H, V, dtype, 8)
    # the probabilities are an input of the recorded step
    g = torch.Generator(device="cuda").manual_seed(1)
    probs = [torch.softmax(torch.randn((B, N, V), generator=g, device="cuda"), -1) for _ in range(4)]

    def run(s):
        s.layer()
        s.finish()

    t.draft(0, 1)
    e.draft(0, 1)
    for s in (t, e):
        s.p.copy_(probs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(t)
    torch.cuda.current_stream().wait_stream(side)
    run(e)
    for a, b in zip(_snapshot(t), _snapshot(e)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(t)
    torch.cuda.synchronize()
    for r in range(4):
        print(f"  replay {r}", flush=True)
        for s in (t, e):
            s.draft(10 + r, r)
            s.p.copy_(probs[r])
        graph.replay()
        run(e)
        for i, (a, b) in enumerate(zip(_snapshot(t), _snapshot(e))):
            assert torch.equal(a, b), (r, i)


def test_steps_on_two_streams_at_once():
    """Two steps on two streams, neither the default one, several times: each
    gives the bits it gives alone."""
    kda = need_gpu()
    B, N, H, V = 24, 16, 4, 900
    case("tree steps on two streams")
    alone = []
    for seed in (21, 22):
        t = Step(kda, B, N, H, V, "bf16", seed)
        t.draft(seed, 3)
        for _ in range(4):
            t.layer()
            t.predict()
            t.finish()
        alone.append(_snapshot(t))
    two = [Step(kda, B, N, H, V, "bf16", seed) for seed in (21, 22)]
    for t, seed in zip(two, (21, 22)):
        t.draft(seed, 3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for t, s in zip(two, streams):
            with torch.cuda.stream(s):
                t.layer()
                t.predict()
                t.finish()
    for t, ref in zip(two, alone):
        for i, (a, b) in enumerate(zip(_snapshot(t), ref)):
            assert torch.equal(a, b), i


def test_no_sequences():
    kda = need_gpu()
    case("tree calls with B = 0")
    x, b = torch.empty((0, 4, 2, 128), device="cuda"), torch.empty((0, 4, 2), device="cuda")
    S = torch.empty((0, 2, 128, 128), device="cuda")
    w, bias = torch.empty((3, 2, 128, 4), device="cuda"), torch.empty((2, 128), device="cuda")
    out = kda.kda_tree_prologue(x, x, x, x, b, w, bias)
    assert [t.shape for t in out] == [x.shape] * 4 + [b.shape]
    assert kda.kda_tree_decode(x, x, x, x, b, S).shape == x.shape
    path, m, nxt = kda.kda_tree_accept(torch.empty((0, 4, 9), device="cuda"), None,
                                       torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                                       torch.empty((0, 4), device="cuda"))
    assert (path.shape, m.shape, nxt.shape) == ((0, 4), (0,), (0,))
    assert kda.kda_tree_commit(x, x, x, b, S, path) is S
    torch.cuda.synchronize()


def test_binding_refuses_and_writes_nothing():
    kda = need_gpu()
    case("tree calls: wrong shapes, types, strides, places")
    B, N, H, V = 2, 4, 2, 9
    w = node_inputs(B, N, H, "f32", seed=3)
    five = [w[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    par = i32(random_trees(B, N, 1))
    o = torch.full_like(w["v"], SENTINEL)
    S0 = w["S"].clone()

    def no(error, match, fn, *a, **kw):
        with pytest.raises(error, match=match):
            fn(*a, **kw)

    def put(args, i, x):
        return [x if j == i else a for j, a in enumerate(args)]

    dec = five + [w["S"], par, None]
    D = kda.kda_tree_decode
    no(ValueError, "k must be contiguous", D, *put(dec, 1, w["k"].transpose(1, 2).contiguous().transpose(1, 2)), o=o)
    no(TypeError, "v must be torch.float32", D, *put(dec, 2, w["v"].bfloat16()), o=o)
    no(ValueError, "log_alpha must have shape", D, *put(dec, 3, w["log_alpha"][:, :3].contiguous()), o=o)
    no(ValueError, "beta must be on cuda", D, *put(dec, 4, w["beta"].cpu()), o=o)
    no(TypeError, "S must be torch.float32", D, *put(dec, 5, w["S"].bfloat16()), o=o)
    no(TypeError, "parent must be torch.int32", D, *put(dec, 6, par.long()), o=o)
    no(ValueError, "n_node must have shape", D, *put(dec, 7, i32([1, 2, 3])), o=o)
    no(ValueError, "o must have shape", D, *dec, o=o[:1])
    no(kda.KDAError, None, D, *dec, o=w["q"])                      # overlap
    wide = torch.zeros((B, 65, H, 128), device="cuda")
    no(kda.KDAError, None, D, wide, wide, wide, wide, wide[..., 0].contiguous(), w["S"])
    no(TypeError, None, D, *[x.half() for x in five], w["S"], par)

    p = torch.full((B, N, V), 1.0 / V, device="cuda")
    tok, u = torch.zeros((B, N), dtype=torch.int32, device="cuda"), torch.zeros((B, N), device="cuda")
    A = kda.kda_tree_accept
    path = torch.full((B, N), 77, dtype=torch.int32, device="cuda")
    no(ValueError, "q must have shape", A, p, p, tok, u, path=path)
    no(TypeError, "tokens must be torch.int32", A, p, None, tok.long(), u, path=path)
    no(TypeError, "u must be torch.float32", A, p, None, tok, u.double(), path=path)
    no(ValueError, "p must be|contiguous", A, p.transpose(0, 1), None, tok, u, path=path)
    no(kda.KDAError, None, A, p, None, path, u, path=path)         # overlap

    com = five[1:] + [w["S"], path]
    C = kda.kda_tree_commit
    no(ValueError, "path must be an int32 tensor", C, *put(com, 5, path[0]))
    no(TypeError, "path must be torch.int32", C, *put(com, 5, path.long()))
    no(ValueError, "conv must be", C, *com, conv=(w["q"], w["k"], w["v"]))
    no(ValueError, "conv_state must have shape", C, *com, conv=(w["q"], w["k"], w["v"], w["S"]))
    no(kda.KDAError, None, C, *put(com, 0, w["S"].view(-1)[:B * N * H * 128].view(B, N, H, 128)))
    no(ValueError, "out must be", kda.kda_tree_prologue, *five, torch.zeros((3, H, 128, 4), device="cuda"),
       torch.zeros((H, 128), device="cuda"), out=five[:4])
    torch.cuda.synchronize()
    assert torch.all(o == SENTINEL) and torch.all(path == 77) and torch.equal(w["S"], S0)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements (states of 4 * 2^30 too): the last
    sequences give the bits they give by themselves."""
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free memory")
    B, N, H = 2740, 64, 96
    case(f"tree prologue, decode, commit with B={B} N={N} H={H}")
    assert B * N * H * 128 > 2 ** 31 and B * H * 128 * 128 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    # one tensor for every input: its values are fit for k and for log alpha
    x = torch.empty((B, N, H, 128), dtype=torch.bfloat16, device="cuda").uniform_(-0.08, 0.0, generator=g)
    beta = torch.empty((B, N, H), dtype=torch.bfloat16, device="cuda").uniform_(0.0, 1.0, generator=g)
    S = torch.empty((B, H, 128, 128), device="cuda").uniform_(-1.0, 1.0, generator=g)
    par = i32(random_trees(1, N, 5)).expand(B, N).contiguous()
    count = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    path = torch.sort(torch.randint(0, N, (B, 8), generator=g, device="cuda", dtype=torch.int32), 1)[0].contiguous()
    last = slice(B - 2, B)
    count[last] = N
    some = lambda t: t[last].clone()
    o = kda.kda_tree_decode(x, x, x, x, beta, S, par, count)
    one = kda.kda_tree_decode(some(x), some(x), some(x), some(x), some(beta), some(S), some(par))
    assert torch.equal(o[last], one)
    del o
    print("  decode", flush=True)
    before = some(S)
    kda.kda_tree_commit(x, x, x, beta, S, path)
    assert torch.equal(S[last], kda.kda_tree_commit(some(x), some(x), some(x), some(beta), before, some(path)))
    assert not torch.equal(S[last], before.new_zeros(()).expand_as(before))
    del S, before
    print("  commit", flush=True)
    w = torch.empty((3, H, 128, 4), device="cuda").uniform_(-1, 1, generator=g)
    bias = torch.zeros((H, 128), device="cuda")
    got = kda.kda_tree_prologue(x, x, x, x, beta, w, bias, par, count)
    ref = kda.kda_tree_prologue(some(x), some(x), some(x), some(x), some(beta), w, bias, some(par))
    for a, r in zip(got, ref):
        assert torch.equal(a[last], r)
    del got, ref, x
    print("  prologue", flush=True)
    B, V = 9, 1 << 22
    p = torch.empty((B, N, V), dtype=torch.bfloat16, device="cuda").uniform_(0.0, 1.0 / V, generator=g)
    q = p.view(-1)[:B * (N - 1) * V].view(B, N - 1, V)
    tok = torch.randint(0, V, (B, N), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand((B, N), generator=g, device="cuda")
    par = i32(random_trees(B, N, 6))
    got = kda.kda_tree_accept(p, q, tok, u, par)
    ref = kda.kda_tree_accept(_tail(p, B), _tail(q, B), _tail(tok, B), _tail(u, B), _tail(par, B))
    for a, r in zip(got, ref):
        assert torch.equal(a[B - 2:], r)


def _tail(t, B):
    return t[B - 2:].clone()


def test_commit_of_nodes_far_into_a_sequence():
    """Without a limit on N: a path through a sequence of more than 2^31
    channels' values, against the same nodes gathered."""
    kda = need_gpu()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free memory")
    N, H = 180000, 96
    case(f"tree_commit with N={N} H={H}")
    assert N * H * 128 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty((1, N, H, 128), dtype=torch.bfloat16, device="cuda").uniform_(-0.08, 0.0, generator=g)
    beta = torch.empty((1, N, H), dtype=torch.bfloat16, device="cuda").uniform_(0.0, 1.0, generator=g)
    S = torch.empty((1, H, 128, 128), device="cuda").uniform_(-1.0, 1.0, generator=g)
    hist = torch.zeros((1, 3, 3, H, 128), dtype=torch.bfloat16, device="cuda")
    way = [0, 3, N - 1, 175000, 175000, 9, N - 2]
    ix = torch.tensor(way, device="cuda")
    few, fbeta = x[:, ix].contiguous(), beta[:, ix].contiguous()
    ref, rhist = S.clone(), hist.clone()
    kda.kda_tree_commit(few, few, few, fbeta, ref, i32([list(range(len(way)))]), conv=(few, few, few, rhist))
    kda.kda_tree_commit(x, x, x, beta, S, i32([way]), conv=(x, x, x, hist))
    torch.cuda.synchronize()
    assert torch.equal(S, ref) and torch.equal(hist, rhist)
