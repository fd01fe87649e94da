"""A serving loop of all of it: a prompt's prefill, its states into the 8-bit cache, drafts
decoded and sampled from there (folds where the windows are full), verified against the fp32
states of the target, accepted, and both moved on: eagerly against the oracles, and captured
against eager calls."""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import cache as oc
from oracle import sample as osamp
from oracle import tree as otree
from cache_util import D, DT, i32
from gpu_util import case, need_gpu, np_

pytestmark = pytest.mark.gpu


class Serving:
    """B sequences of H heads, N - 1 drafts a step, windows of W; a vocabulary of V whose rows are a token's inputs."""

    def __init__(self, kda, dtype, seed, B=3, H=2, N=4, W=10, V=3000):
        self.kda, self.B, self.H, self.N, self.W, self.V = kda, B, H, N, W, V
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        unit = lambda *s: torch.nn.functional.normalize(rand(*s, D), dim=-1) * 0.99  # noqa: E731
        self.table = [x.to(DT[dtype]) for x in (unit(V, H), unit(V, H), rand(V, H, D), -5 * torch.sigmoid(rand(V, H, D) - 2),
                                                torch.sigmoid(rand(V, H)))]
        self.head = rand(H * D, V) * 0.8
        d = kda_inputs.prefill_inputs(60, H, dtype=dtype, device="cuda", seed=seed, lengths=[20, 7, 33])
        _, self.S = kda.kda_chunk_fwd(*(d[x] for x in ("q", "k", "v", "log_alpha", "beta")), cu_seqlens=d["cu_seqlens"])
        # the prompts' states go to pages of a pool, the batch is read from there
        pool = (torch.zeros((B + 4, H, D, D), dtype=torch.int8, device="cuda"), torch.zeros((B + 4, H, D), device="cuda"))
        page = i32([5, 0, 3])
        kda.kda_cache_store(self.S, *pool, page)
        self.codes, self.scale = kda.kda_cache_store(kda.kda_cache_load(*pool, page))
        self.win = tuple(torch.zeros((B, H, W, D), dtype=DT[dtype], device="cuda") for _ in range(3))
        self.n = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pending = torch.arange(B, device="cuda", dtype=torch.int32) * 7
        self.u_draft, self.u = torch.zeros((N - 1, B), device="cuda"), torch.zeros((B, N), device="cuda")
        # requests of their own: greedy, by k, by p and m
        self.ask = [torch.tensor([0.0, 0.9, 1.2], device="cuda"), i32([0, 40, 0]), torch.tensor([1.0, 0.95, 0.9], device="cuda"),
                    torch.tensor([0.0, 0.0, 0.01], device="cuda")]
        self.tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        self.q = torch.zeros((N - 1, B, V), device="cuda")
        self.logits = torch.zeros((N - 1, B, V), device="cuda")

    def random(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.u_draft.copy_(torch.rand(self.u_draft.shape, generator=g, device="cuda"))
        self.u.copy_(torch.rand(self.u.shape, generator=g, device="cuda"))

    def predict(self, o):
        return o.float().reshape(-1, self.H * D) @ self.head

    def step(self):
        kda, B, N, V = self.kda, self.B, self.N, self.V
        self.tokens[:, 0].copy_(self.pending)
        for i in range(N):
            x = [t[self.tokens[:, i].long()] for t in self.table]
            o = kda.kda_cache_decode(*x, self.codes, self.scale, self.win, self.n + i)
            if i + 1 < N:
                self.logits[i].copy_(self.predict(o))
                token, _ = kda.kda_sample(self.logits[i], self.u_draft[i], *self.ask, probs=self.q[i])
                self.tokens[:, i + 1].copy_(token)
        x = [t[self.tokens.long()] for t in self.table]
        self.target = self.predict(kda.kda_tree_decode(*x, self.S)).view(B, N, V)
        _, self.p = kda.kda_sample(self.target, None, *(a[:, None].expand(B, N).contiguous() for a in self.ask), probs=True)
        self.path, self.m, nxt = kda.kda_tree_accept(self.p, self.q.transpose(0, 1).contiguous(), self.tokens, self.u)
        kda.kda_tree_commit(*x[1:], self.S, self.path, self.m)
        # the window's places past the accepted tokens are written anew by the next step
        self.n += self.m
        full = torch.where(self.n + N > self.W, self.n, torch.zeros_like(self.n))
        kda.kda_cache_fold(self.codes, self.scale, self.win, full)
        self.n -= full
        self.full, self.pending = full, self.pending.copy_(nxt)

    def everything(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.tokens, self.q, self.p, self.path, self.m, self.pending, self.n, self.S, self.codes,
                                    self.scale, *self.win)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_serving_loop_from_prefill_to_accepted_tokens(dtype):
    kda = need_gpu()
    case(f"prefill, store, draft, sample, verify, accept, commit, fold {dtype}")
    s = Serving(kda, dtype, 1)
    half = oc.HALF[dtype]
    # half a step everywhere, of the pool's pages and once more of the batch's (see the conversation's test)
    halves = lambda: (np_(s.scale).astype(np.float64) ** 2).sum(-1) ** 0.5 * 0.501 * np.sqrt(D)  # noqa: E731
    drift = 2 * halves()
    taken = folds = 0
    for step in range(6):
        s.random(50 + step)
        n0 = s.n.cpu().numpy()
        s.step()
        torch.cuda.synchronize()
        tok, q, p, m = s.tokens.cpu().numpy(), np_(s.q), np_(s.p), s.m.cpu().numpy()
        ask = [a.cpu().numpy() for a in s.ask]
        for b in range(s.B):
            for i in range(s.N - 1):
                t, pr, margin = osamp.row(np_(s.logits[i, b]), float(s.u_draft[i, b]), *(float(a[b]) if a.dtype.kind == "f" else int(a[b]) for a in ask))
                assert margin < 1e-9 or tok[b, i + 1] == t, (step, b, i, margin)
                # (as in the sampling tests)
                assert (np.abs(q[i, b] - pr) <= 5.5 * 2.0 ** -24 * pr + 2.0 ** -126).all()
            way, nxt, margin = otree.accept(p[b], q[:, b], tok[b], np_(s.u[b]), otree.chain(s.N), s.N)
            assert margin < 1e-6 or (s.path[b, :m[b]].tolist() == way and int(s.pending[b]) == nxt), (step, b, margin)
            for j in range(m[b]):
                u = np.linalg.norm(np_(s.win[2][b, :, n0[b] + j]).astype(np.float64), axis=-1)
                drift[b] += half * u        # (keys are shorter than 1: no more of it)
        f = s.full.cpu().numpy()
        folds += int((f > 0).sum())
        drift += np.where(f > 0, 1, 0)[:, None] * halves()
        S, S8 = np_(s.S).astype(np.float64), np_(kda.kda_cache_load(s.codes, s.scale, None, s.win, s.n)).astype(np.float64)
        far = np.linalg.norm((S8 - S).reshape(s.B, s.H, -1), axis=-1)
        size = np.linalg.norm(S.reshape(s.B, s.H, -1), axis=-1)
        # (and the roundings of up to four tokens a step on both sides in fp32, 1e-5: 40 of 2^-24 a token)
        assert (far <= drift + 1e-5 * (step + 1) * size).all(), (step, far / drift)
        taken += int(m.sum())
    print(f"    {taken} tokens, {folds} folds", flush=True)
    assert taken > 6 * s.B and folds >= s.B


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_captured_loop_replays_as_eager_steps(dtype):
    kda = need_gpu()
    case(f"captured serving step {dtype}")
    a, b, warm = (Serving(kda, dtype, 2) for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for r in range(5):
        a.random(80 + r)
        b.random(80 + r)
        graph.replay()
        b.step()
        for i, (x, y) in enumerate(zip(a.everything(), b.everything())):
            assert torch.equal(x, y), (r, i)
