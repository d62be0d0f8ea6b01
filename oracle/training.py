"""Oracle: the router's training steps in fp64 (test infrastructure only).

gate           softmax over the experts, the k largest (ties to the lower id),
               their weights, tokens per expert, the balance loss
gate_backward  the gradient of sum(dw * w) + dloss * loss into the logits
router_backward  dx = dz W, dW = dz^T x

Pins (tests/test_oracle_training.py): gate_backward against central
differences of gate, every convention and mask; the loss of a uniform router
is 1 and of a router that always picks the same k experts E / k; the counts
sum to k per routed token.
"""

import numpy as np


def gate(z, k, renorm=False, mask=None):
    """z [T, E] fp64 (-inf: not available), mask [T] bool or None.
    Returns dict ids [T, k] (-1: none), w, p, counts [E + 1], loss, routed [T]."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    routed = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool).copy()
    routed &= ~np.all(np.isneginf(z), axis=1)
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    p = np.zeros((T, E))
    for t in np.nonzero(routed)[0]:
        e = np.exp(z[t] - np.max(z[t]))
        p[t] = e / e.sum()
        order = [i for i in np.lexsort((np.arange(E), -z[t])) if z[t, i] > -np.inf][:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order] / (p[t, order].sum() if renorm else 1.0)
    counts = np.array([np.sum(ids == e) for e in range(E)] + [routed.sum()], dtype=np.int64)
    n = int(routed.sum())
    loss = float(E / (k * n * n) * np.sum(counts[:E] * p.sum(axis=0))) if n else 0.0
    return dict(ids=ids, w=w, p=p, counts=counts, loss=loss, routed=routed)


def gate_backward(z, ids, renorm=False, dw=None, counts=None, dloss=None):
    """dlogits [T, E] from the definition: d p_a / d z_b = p_a ([a = b] - p_b)."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    b = np.zeros(E)
    if dloss is not None and counts[E] > 0:
        b = dloss * E * np.asarray(counts[:E], dtype=np.float64) / (k * float(counts[E]) ** 2)
    for t in range(T):
        if ids[t, 0] < 0:
            continue
        e = np.exp(z[t] - np.max(z[t]))
        p = e / e.sum()
        dp = b.copy()
        if dw is not None:
            live = (ids[t] >= 0) & (ids[t] < E)
            c = ids[t][live]
            g = np.asarray(dw, dtype=np.float64)[t][live]
            if renorm:
                s = p[c].sum()
                g = (g - np.sum(g * p[c]) / s) / s
            np.add.at(dp, c, g)
        out[t] = p * (dp - np.sum(p * dp))
    return out


def router_backward(x, w_router, dz):
    """(dx [T, H], dW [E, H])"""
    x, w, dz = (np.asarray(a, dtype=np.float64) for a in (x, w_router, dz))
    return dz @ w, dz.T @ x
