"""CPU oracle for sampling -- TEST INFRASTRUCTURE ONLY (same rule as the rest of
``oracle``).  One row at a time, by sorting it, in extended precision."""
import numpy as np


def row(logits, u=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probabilities [V], margin): margin is how far the nearest border
    between two tokens lies from u, and the nearest leading set's share from
    top_p, relative to the sums."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    V = len(l)
    probs = np.zeros(V)
    top = l.max()
    if top == -np.inf:
        return -1, probs, np.inf
    order = np.lexsort((np.arange(V), -l))
    margin = np.inf
    if not temperature > 0:
        probs[order[0]] = 1.0
        return int(order[0]), probs, margin
    x = l[order]
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(x == top, 0.0, (x - top).astype(np.longdouble) / np.longdouble(temperature))
    w = np.where(x == -np.inf, np.longdouble(0), np.exp(np.where(np.isnan(d), -np.inf, d)))   # (infinite top: nothing else weighs)
    n = int((x > -np.inf).sum())
    if 1 <= top_k < V:
        n = min(n, int(top_k))
    if top_p < 1:
        cum = np.cumsum(w[:n])
        goal = np.longdouble(max(top_p, 0.0)) * cum[-1]
        keep = max(1, int((cum < goal).sum()) + 1)
        away = np.abs(cum - goal) / cum[-1]
        away[cum == goal] = np.inf              # (met exactly: sums of whole numbers)
        if top_p > 0:
            margin = min(margin, away.min())
        n = min(n, keep)
    kept = w[:n] >= (min(min_p, 1.0) if min_p > 0 else 0.0)
    held = np.zeros(V, np.longdouble)
    held[order[:n]] = np.where(kept, w[:n], 0)
    cum = np.cumsum(held)
    probs = (held / cum[-1]).astype(np.float64)
    if u is None:
        return -1, probs, margin
    u = 0.0 if not u > 0 else float(u)
    goal = np.longdouble(u) * cum[-1]
    if u >= 1:
        return int(np.nonzero(held > 0)[0][-1]), probs, margin
    token = int((cum <= goal).sum())
    border = np.unique(cum[held > 0])
    away = np.abs(border - goal) / cum[-1]
    away[border == goal] = np.inf
    return token, probs, float(min(margin, away.min()))
