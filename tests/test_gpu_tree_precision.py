"""What kda_tree_decode holds between its inputs and the one rounding of its
outputs: 24 bits, for bf16 inputs as for fp32 ones.

Every number of these cases is a whole number, no token decays (log alpha =
0), and every partial sum stays below 2^24: a 32-bit evaluation is exact in
whatever order it sums, and the outputs, at most 256, are exact in bf16.  So
nothing is tolerated.  Fewer bits in an operand (a state of 19 bits held in
16, say) show as whole units.
"""
import pytest
import torch

from gpu_util import case, need_gpu
from tree_util import i32

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = 2
SIZES = [2, 8, 10, 16, 24, 32, 40, 48, 64]


class Nodes:
    """Zeros for every input of B = 1 sequences of N nodes, filled in by the
    cases below; `part[i]` continues node i - 1, other nodes the state."""

    def __init__(self, N, dtype, seed):
        self.N, self.dt = N, DT[dtype]
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.q, self.k, self.v, self.la = (torch.zeros((1, N, H, 128), device="cuda") for _ in range(4))
        self.beta = torch.zeros((1, N, H), device="cuda")
        self.S = torch.zeros((1, H, 128, 128), device="cuda")

    def ints(self, lo, hi, *shape):
        """Whole numbers of [lo, hi]."""
        return torch.randint(lo, hi + 1, shape, generator=self.g, device="cuda").float()

    def near_pairs(self, pairs):
        """State rows 2 c and 2 c + 1 of 19 bits that differ by at most 4;
        returns, for every node, 12 of those pairs entered with +1 and -1 (or
        the reverse): [N, H, 128]."""
        a = self.ints(1 << 18, (1 << 19) - 5, H, pairs, 1, 128)
        near = torch.cat([a, a + self.ints(-4, 4, H, pairs, 1, 128)], 2)
        self.S[0, :, :2 * pairs] = near.reshape(H, 2 * pairs, 128)
        x = torch.zeros((self.N, H, 128), device="cuda")
        for i in range(self.N):
            for h in range(H):
                c = torch.randperm(pairs, generator=self.g, device="cuda")[:12]
                s = 2 * self.ints(0, 1, 12) - 1
                x[i, h, 2 * c], x[i, h, 2 * c + 1] = s, -s
        return x

    def outputs(self, kda, parent):
        a = [x.to(self.dt) for x in (self.q, self.k, self.v, self.la, self.beta)]
        for x, y in zip(a, (self.q, self.k, self.v)):
            assert torch.equal(x.float(), y), "an input is not exact in its type"
        o = kda.kda_tree_decode(*a, self.S, i32([parent]))
        torch.cuda.synchronize()
        return o[0].double()

    def from_state(self, x):
        """x [N, H, 128] times the states, in 64 bits."""
        return torch.matmul(x.double().transpose(0, 1), self.S[0].double()).transpose(0, 1)


def _equal(o, ref):
    assert ref.abs().max() <= 256 and (ref != 0).any()
    off = (o - ref).abs()
    print(f"    off by at most {off.max().item():g} of {ref.abs().max().item():g}, "
          f"{(off > 0).double().mean().item():.1%} of the outputs", flush=True)
    assert torch.equal(o, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", SIZES)
def test_what_is_read_keeps_the_state_whole(dtype, N):
    """o = S^T q alone (beta = 0)."""
    kda = need_gpu()
    case(f"tree_decode, exact reads, {dtype} N={N}")
    t = Nodes(N, dtype, N)
    x = t.near_pairs(64)
    t.q[0] = x
    _equal(t.outputs(kda, [-1] * N), t.from_state(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", SIZES)
def test_what_is_held_keeps_the_state_whole(dtype, N):
    """o = u = v - S^T k: q and k share a channel whose state row is 0."""
    kda = need_gpu()
    case(f"tree_decode, exact pseudo-values, {dtype} N={N}")
    t = Nodes(N, dtype, 100 + N)
    x = t.near_pairs(63)
    t.k[0] = x
    t.k[..., 127] = t.q[..., 127] = 1
    t.beta.fill_(1)
    t.v[0] = t.ints(-100, 100, N, H, 128)
    _equal(t.outputs(kda, [-1] * N), t.v[0].double() - t.from_state(x))


def _pairs(N):
    """Node 2 m continues the state, node 2 m + 1 node 2 m."""
    return [i - 1 if i % 2 else -1 for i in range(N)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", SIZES)
def test_pseudo_values_keep_their_bits(dtype, N):
    """u of a node is -(S_0 + S_1), 22 bits; its child reads S_0 + S_2 + u
    with S_2 - S_1 small."""
    kda = need_gpu()
    case(f"tree_decode, pseudo-values of 22 bits, {dtype} N={N}")
    t = Nodes(N, dtype, 200 + N)
    a, c, r = (t.ints(lo, hi, H, 128) for lo, hi in ((1 << 20, (1 << 21) - 1),) * 2 + ((-60, 60),))
    t.S[0, :, 0], t.S[0, :, 1], t.S[0, :, 2] = a, c, c + r
    t.k[0, 0::2, :, :2] = 1
    t.beta[0, 0::2] = 1
    t.q[0, 1::2, :, 0] = t.q[0, 1::2, :, 2] = 1
    ref = torch.zeros((N, H, 128), dtype=torch.float64, device="cuda")
    ref[1::2] = r.double()
    _equal(t.outputs(kda, _pairs(N)), ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", SIZES)
@pytest.mark.parametrize("of", ["q", "k"])
def test_couplings_keep_their_bits(dtype, N, of):
    """<q, k> (and <k, k>) of a node and its child are whole numbers M of up
    to 20 bits; a state row r - M takes all but r away again."""
    kda = need_gpu()
    case(f"tree_decode, couplings of 20 bits of {of}, {dtype} N={N}")
    t = Nodes(N, dtype, 300 + N)
    half = N // 2
    a, c = t.ints(1, 127, half, H, 64), t.ints(1, 127, half, H, 64)   # channels 0 .. 63
    M = (a.double() * c.double()).sum(-1)                             # [half, H]
    assert M.max() > 1 << 17 and M.max() < 1 << 20
    r = t.ints(-100, 100, half, H, 128)
    z = 64 + torch.arange(half, device="cuda")                        # a channel for every pair
    t.S[0, :, 64:64 + half] = (r.double() - M[..., None]).float().transpose(0, 1)
    t.k[0, 0:2 * half:2, :, :64] = a
    t.v[0, 0::2] = 1
    t.beta[0, 0::2] = 1
    child = torch.arange(half, device="cuda") * 2 + 1
    x = t.q if of == "q" else t.k
    x[0, child, :, :64] = c
    x[0, child, :, z] = 1
    ref = torch.zeros((N, H, 128), dtype=torch.float64, device="cuda")
    if of == "q":      # o = S^T q + M u, u = 1
        ref[child] = r.double()
    else:              # o = u of the child = v - S^T k - M
        t.q[0, child, :, 127] = t.k[0, child, :, 127] = 1
        t.beta[0, child] = 1
        t.v[0, child] = t.ints(-100, 100, half, H, 128)
        ref[child] = t.v[0, child].double() - r.double()
    _equal(t.outputs(kda, _pairs(N)), ref)
