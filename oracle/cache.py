"""CPU oracle for the 8-bit state cache -- TEST INFRASTRUCTURE ONLY (same rule
as the rest of ``oracle``).

``quantise`` is the rounding of a state to codes and scales, operation by
operation in float32 as it is defined; everything else goes through the
window token by token in float64.  Beside each result stands a bound on what
an evaluation in 32 bits may be off: 2^-24 times the sum of the magnitudes
that are added up, each with the roundings that its factors have seen.
"""
import numpy as np

EPS = 2.0 ** -24          # half a step of fp32, relative
TINY = np.float32(2.0 ** -100)
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of the type (24 and 8 bits), relative


def quantise(S):
    """float32 states [.., 128 (key), 128 (value)] -> codes [.., value, key]
    int8 and scales [.., key] float32.  (The product of two 24-bit numbers is
    exact in float64.)"""
    S = np.asarray(S, dtype=np.float32)
    top = np.abs(S).max(-1)
    held = top >= TINY
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inverse = np.where(held, np.float32(127) / top, np.float32(0)).astype(np.float32)
        scale = np.where(held, top / np.float32(127), np.float32(0)).astype(np.float32)
        codes = np.rint(S.astype(np.float64) * inverse[..., None]).astype(np.int8)
    return np.swapaxes(codes, -1, -2), scale


def values(codes, scale):
    """float64 states [.., key, value] of codes and scales."""
    return np.swapaxes(np.asarray(codes, np.float64), -1, -2) * np.asarray(scale, np.float64)[..., None]


def state(codes, scale, k, la, u, n):
    """One head's state after the first n tokens of its window (k, la, u [W,
    128] float64) and the bound of its entries."""
    S = values(codes, scale)
    # a decay's sum of log alpha is exact, its exponential off by two steps at the most (four roundings)
    terms = [S]
    for t in range(n):
        terms = [x * np.exp(la[t])[:, None] for x in terms] + [k[t][:, None] * u[t][None, :]]
    total = sum(terms)
    bound = EPS * (n + 8) * sum(np.abs(x) for x in terms)
    return total, bound


def decode(q, k, v, la, beta, codes, scale, wk, wla, wu, n):
    """One head's token: the update before it is rounded, its bound; and a
    function of the update as it is held that gives the output and its bound."""
    S, off = state(codes, scale, wk, wla, wu, n)
    d = np.exp(la)[:, None]
    S, off = d * S, d * (off + 4 * EPS * np.abs(S))

    def read(x):
        # a vector times 128 terms: a sum of as many roundings as its depth, 16 at the most
        return x @ S, np.abs(x) @ off + 16 * EPS * (np.abs(x) @ np.abs(S))

    sk, bk = read(k)
    u = beta * (v - sk)
    bu = np.abs(beta) * (bk + 4 * EPS * (np.abs(v) + np.abs(sk)))

    def output(held):
        sq, bq = read(q)
        kq = float(k @ q)
        return sq + kq * held, bq + EPS * (16 * (np.abs(k) @ np.abs(q)) * np.abs(held) + 4 * np.abs(sq))

    return u, bu, output
