"""The gated recurrence in 64 bits, from its definition, on the host: token by
token, and its gradient as the reversed recurrence."""
import numpy as np


def gates(g, form):
    """(a, 1 - a)."""
    g = np.asarray(g, np.float64)
    if form == "decay":
        return g, 1 - g
    if form == "log":
        return np.exp(g), -np.expm1(g)
    e = np.exp(-np.abs(g))
    small, large = e / (1 + e), 1 / (1 + e)
    return np.where(g < 0, small, large), np.where(g < 0, large, small)


def forward(a, b, lens, state=None):
    """h over packed rows [N, D] of sequences `lens` long: (out, last states)."""
    out = np.zeros(b.shape)
    last = np.zeros((len(lens), b.shape[1]))
    at = 0
    for s, n in enumerate(lens):
        h = np.zeros(b.shape[1]) if state is None else np.array(state[s], np.float64)
        for t in range(at, at + n):
            h = a[t] * h + b[t]
            out[t] = h
        last[s] = h
        at += n
    return out, last


def before(out, lens, state=None):
    """h(t - 1) of each token."""
    prev = np.zeros(out.shape)
    at = 0
    for s, n in enumerate(lens):
        if n:
            prev[at] = 0 if state is None else state[s]
            prev[at + 1:at + n] = out[at:at + n - 1]
        at += n
    return prev


def backward(dout, a, lens, dlast=None):
    """(dh, the initial states' gradient)."""
    dh = np.zeros(dout.shape)
    first = np.zeros((len(lens), dout.shape[1]))
    at = 0
    for s, n in enumerate(lens):
        g = np.zeros(dout.shape[1]) if dlast is None else np.array(dlast[s], np.float64)
        for t in range(at + n - 1, at - 1, -1):
            dh[t] = dout[t] + g
            g = a[t] * dh[t]
        first[s] = g
        at += n
    return dh, first


def slope(a, rest, form):
    return {"decay": np.ones_like(a), "log": a, "sigmoid": a * rest}[form]
