"""CPU oracle for speculative decoding with a tree of drafted tokens -- TEST
INFRASTRUCTURE ONLY (same rule as the rest of ``oracle``).

Every node of a tree is the end of one path from the root; a node's outputs
are those of that path run as an ordinary sequence: through the token-by-token
recurrence (``oracle.fwd``) and the layer prologue (``oracle.layer``).  No
ancestor masks, no Gram matrices.  The verification of the drafts is the
rejection walk written on normalised distributions, one residual after the
other.  All in float64.
"""
import numpy as np

import oracle
from oracle import layer


def paths(parent, n):
    """The path from the root to every node i < n: lists of node indices.
    parent[i] outside [0, i): node i continues the cached state."""
    out = []
    for i in range(n):
        p = int(parent[i])
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def chain(N):
    return np.arange(N) - 1


def _rows(x, ways):
    return np.concatenate([np.asarray(x, dtype=np.float64)[w] for w in ways])


def _cu(ways):
    return np.concatenate([[0], np.cumsum([len(w) for w in ways])])


def decode(q, k, v, log_alpha, beta, S, parent, n):
    """One sequence: q, k, v, log_alpha [N, H, 128], beta [N, H], S [H, 128,
    128]; returns o [n, H, 128] of the first n nodes."""
    ways = paths(parent, n)
    cu = _cu(ways)
    h0 = np.broadcast_to(np.asarray(S, dtype=np.float64), (n,) + S.shape)
    o, _ = oracle.fwd(*[_rows(x, ways) for x in (q, k, v, log_alpha, beta)], h0=h0, cu_seqlens=cu,
                      store_state=False)
    return o[cu[1:] - 1]


def prologue(xq, xk, xv, a, b, conv_w, a_bias, parent, n, conv_state=None, l2_eps=1e-6):
    """One sequence: x, a [N, H, 128], b [N, H], conv_state [3, 3, H, 128] or
    None; returns (q, k, v, log_alpha, beta) of the first n nodes."""
    ways = paths(parent, n)
    cu = _cu(ways)
    cs = None if conv_state is None else np.broadcast_to(
        np.asarray(conv_state, dtype=np.float64), (n,) + conv_state.shape)
    got = layer.prologue(*[_rows(x, ways) for x in (xq, xk, xv, a, b)], conv_w, a_bias,
                         cu_seqlens=cu, conv_state=cs, l2_eps=l2_eps)
    return tuple(x[cu[1:] - 1] for x in got[:5])


def commit(k, v, log_alpha, beta, S, way, x=None, conv_state=None):
    """One sequence moved along the nodes `way`: (state, history or None).
    x: the three convolution inputs [N, H, 128]."""
    way = list(way)
    if not way:
        return np.asarray(S, dtype=np.float64), conv_state
    kk = _rows(k, [way])
    _, hT = oracle.fwd(kk, kk, *[_rows(t, [way]) for t in (v, log_alpha, beta)],
                       h0=np.asarray(S, dtype=np.float64)[None])
    hist = None
    if conv_state is not None:
        hist = np.stack([np.concatenate([conv_state[t], x[t][way]])[-3:] for t in range(3)])
    return hT[0], hist


def accept(p, q, tokens, u, parent, n):
    """One sequence: p [N, V], q [N - 1, V] or None, tokens, u [N]; returns
    (accepted nodes, next token, margin): the margin is the smallest distance
    of a decision from its border, in probability."""
    V = p.shape[1]
    if n == 0:
        return [], -1, np.inf
    p = np.asarray(p, dtype=np.float64)
    way, margin = [0], np.inf
    while True:
        r = way[-1]
        left = p[r].copy()          # what the next child is tested against, of mass 1
        for x in range(r + 1, n):
            if int(parent[x]) != r:
                continue
            t = int(tokens[x])
            if not 0 <= t < V:
                continue
            draft = np.zeros(V) if q is None else np.asarray(q[r], dtype=np.float64)
            if q is None:
                draft[t] = 1.0
            margin = min(margin, abs(u[x] * draft[t] - left[t]))
            if float(u[x]) * draft[t] < left[t]:
                way.append(x)
                break
            left = np.maximum(left - draft, 0.0) if q is not None else np.where(
                np.arange(V) == t, 0.0, left)
            mass = left.sum()
            left = left / mass if mass > 0 else left
        else:
            break
    w = left if left.sum() > 0 else p[r]
    cum = np.cumsum(w)
    target = float(u[0]) * cum[-1]
    nxt = int(np.argmax(cum > target)) if (cum > target).any() else 0
    margin = min(margin, np.abs(cum - target)[w > 0].min() if (w > 0).any() else np.inf)
    return way, nxt, margin
