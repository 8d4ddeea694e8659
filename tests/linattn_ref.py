"""Linear attention with decay and token sampling in 64 bits, from their
definitions, on the host: the recurrence token by token, its gradient as the
reversed recurrence, and a row of logits sorted and summed."""
import numpy as np


def _heads(x, heads):
    """[N, Hx, D] with the rows of shared heads repeated."""
    return np.repeat(x, heads // x.shape[1], axis=1)


def forward(q, k, v, g, scale, lens, state=None):
    """Packed rows [N, H*, D] of sequences `lens` long: (out, last states)."""
    h, dk, dv = len(g), q.shape[2], v.shape[2]
    q, k, v = (_heads(np.asarray(x, np.float64), h) for x in (q, k, v))
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    out = np.zeros((q.shape[0], h, dv))
    last = np.zeros((len(lens), h, dk, dv))
    at = 0
    for s, n in enumerate(lens):
        z = np.zeros((h, dk, dv)) if state is None else np.array(state[s], np.float64)
        for t in range(at, at + n):
            z = lam * z + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * np.matmul(q[t][:, None, :], z)[:, 0]
        last[s] = z
        at += n
    return out, last


def backward(do, q, k, v, g, scale, lens, state=None, dlast=None):
    """(dq, dk, dv, dstate) with the gradients of shared heads summed."""
    h, dk, dv = len(g), q.shape[2], v.shape[2]
    shared = [h // x.shape[1] for x in (q, k, v)]
    q, k, v, do = (_heads(np.asarray(x, np.float64), h) for x in (q, k, v, do))
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    grads = [np.zeros_like(x) for x in (q, k, v)]
    dstate = np.zeros((len(lens), h, dk, dv))
    at = 0
    for s, n in enumerate(lens):
        z = np.zeros((h, dk, dv)) if state is None else np.array(state[s], np.float64)
        for t in range(at, at + n):
            z = lam * z + k[t][:, :, None] * v[t][:, None, :]
            grads[0][t] = scale * np.matmul(z, do[t][:, :, None])[:, :, 0]
        r = np.zeros((h, dk, dv)) if dlast is None else np.array(dlast[s], np.float64)
        for t in range(at + n - 1, at - 1, -1):
            r = r + scale * q[t][:, :, None] * do[t][:, None, :]
            grads[1][t] = np.matmul(r, v[t][:, :, None])[:, :, 0]
            grads[2][t] = np.matmul(k[t][:, None, :], r)[:, 0]
            r = lam * r
        dstate[s] = r
        at += n
    grads = [x.reshape(x.shape[0], x.shape[1] // m, m, x.shape[2]).sum(2)
             for x, m in zip(grads, shared)]
    return grads + [dstate]


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, kept) of one row of logits."""
    x = np.asarray(x, np.float64)
    live = np.flatnonzero(x > -np.inf)
    if live.size == 0:
        return -1, -np.inf, 0
    top = x[live].max()
    if not temperature > 0:
        return int(np.flatnonzero(x == top)[0]), 0.0, 1
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x[live] == top, 1.0, np.exp((x[live] - top) / np.float64(temperature)))
    order = np.argsort(-x[live], kind="stable")
    if top_k > 0:
        order = order[:top_k]
    if min_p > 0:
        order = order[w[order] >= min(float(min_p), 1.0)]
    if top_p < 1:
        sums = np.cumsum(w[order])
        order = order[:max(1, int(np.searchsorted(sums, top_p * sums[-1])) + 1)]
    keep = np.sort(order)
    sums = np.cumsum(w[keep])
    u = min(max(float(u), 0.0), 1.0) if u == u else 0.0
    passed = np.flatnonzero(sums > u * sums[-1])
    j = int(passed[0]) if passed.size else int(np.flatnonzero(w[keep] > 0)[-1])
    return int(live[keep[j]]), float(np.log(w[keep[j]] / sums[-1])), int(keep.size)
