"""Inputs and comparisons of the 8-bit state cache's tests."""
import numpy as np
import torch

import kda_inputs

D = 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SENTINEL = 77


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def states(n, H, seed, spread=1.0):
    """fp32 states whose key channels differ in size by factors of e^spread."""
    g = gen(seed)
    S = torch.randn((n, H, D, D), generator=g, device="cuda")
    return S * 0.1 * torch.exp(spread * torch.randn((n, H, D, 1), generator=g, device="cuda"))


def window(P, H, W, dtype, seed, mu=-2.0):
    g = gen(seed)
    shape = (P, H, W, D)
    k = torch.nn.functional.normalize(torch.randn(shape, generator=g, device="cuda"), dim=-1)
    la = -5.0 * torch.sigmoid(torch.randn(shape, generator=g, device="cuda") + mu)
    u = 0.5 * torch.randn(shape, generator=g, device="cuda")
    return tuple(x.to(DT[dtype]).contiguous() for x in (k, la, u))


def token(B, H, dtype, seed, mu=-2.0):
    d = kda_inputs.decode_inputs(B, H, dtype=dtype, device="cuda", seed=seed)
    g = gen(seed)
    la = -5.0 * torch.sigmoid(torch.randn((B, H, D), generator=g, device="cuda") + mu)
    return d["q"], d["k"], d["v"], la.to(DT[dtype]), d["beta"]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def within(name, got, ref, bound):
    """Every element within its bound."""
    got, ref, bound = (np.asarray(x, np.float64) for x in (got, ref, bound))
    assert np.isfinite(got).all(), f"{name}: non-finite"
    off = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    print(f"    {name}: at most {np.max(off / np.maximum(bound, 1e-300)):.3f} of the bound", flush=True)
    assert (off <= bound).all(), f"{name}: {got[worst]} at {worst}, {ref[worst]} +- {bound[worst]}"
