"""Inputs of the tree speculative decoding tests."""
import numpy as np
import torch

import kda_inputs

SENTINEL = 1024.0   # exact in bf16 and fp32


def random_trees(B, N, seed, shape="tree"):
    """Parents [B, N] (numpy int32): "tree" random, "chain", "star" (every
    node under the root), "forest" (some nodes start at the cached state
    again, by values outside [0, i) of every kind)."""
    rng = np.random.default_rng(seed)
    par = np.full((B, N), -1, dtype=np.int32)
    for i in range(1, N):
        if shape == "chain":
            par[:, i] = i - 1
        elif shape == "star":
            par[:, i] = 0
        else:
            par[:, i] = rng.integers(0, i, size=B)
        if shape == "forest":
            bad = np.array([-1, i, i + 1, 1 << 30, -(1 << 31), N], dtype=np.int64)[
                rng.integers(0, 6, size=B)].astype(np.int32)
            par[:, i] = np.where(rng.random(B) < 0.3, bad, par[:, i])
    return par


def node_inputs(B, N, H, dtype, seed, decay_mu=-2.0, state_std=0.1):
    """q, k, v, log_alpha [B, N, H, 128], beta [B, N, H], S [B, H, 128, 128]."""
    d = kda_inputs.prefill_inputs(B * N, H, dtype=dtype, device="cuda", seed=seed,
                                  lengths=[N] * B, h0_std=state_std, decay_mu=decay_mu)
    w = {x: d[x].view(B, N, *d[x].shape[1:]) for x in ("q", "k", "v", "log_alpha", "beta")}
    w["S"] = d["h0"]
    return w


def i32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
