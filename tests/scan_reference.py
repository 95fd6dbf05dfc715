"""The recurrence over whole sequences and its gradients, token by token in 64 bits (numpy).

    D = diag(gate);  w = v (mamba2) or beta (v - (D S)^T k);  S <- D S + k w^T;  y = S^T q

Inputs of one sequence and all heads: q, k [T][H][dk], v [T][H][dv], gate [T][H] or
[T][H][dk], beta [T][H] or None, S [H][dk][dv].
"""
import numpy as np


def _gate(gate, t):
    return gate[t][:, None, None] if gate.ndim == 2 else gate[t][:, :, None]


def forward(q, k, v, gate, beta, S, keep=None):
    """(y [T][H][dv], final state). keep: a list that receives D S of every token."""
    S = S.astype(np.float64).copy()
    y = np.zeros(v.shape, np.float64)
    for t in range(len(q)):
        DS = _gate(gate, t) * S
        w = v[t]
        if beta is not None:
            w = beta[t][:, None] * (v[t] - np.einsum("hdv,hd->hv", DS, k[t]))
        S = DS + k[t][:, :, None] * w[:, None, :]
        y[t] = np.einsum("hdv,hd->hv", S, q[t])
        if keep is not None:
            keep.append((DS, S))
    return y, S


def backward(q, k, v, gate, beta, S0, dy, dS):
    """Gradients, and the size of the terms that cancel in dlog (for its tolerance)."""
    kept = []
    forward(q, k, v, gate, beta, S0, kept)
    G = dS.astype(np.float64).copy()
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog", gate))}
    if beta is not None:
        out["dbeta"] = np.zeros(beta.shape)
    size = np.zeros(k.shape)
    run = None
    for t in range(len(q) - 1, -1, -1):
        DS, S = kept[t]
        if run is None or t % 64 == 63:  # the 64-token chunk's end: its product of state and gradient
            run = np.abs(S * G).sum(-1)
        G = G + q[t][:, :, None] * dy[t][:, None, :]
        out["dq"][t] = np.einsum("hdv,hv->hd", S, dy[t])
        r, w = None, v[t]
        if beta is not None:
            r = v[t] - np.einsum("hdv,hd->hv", DS, k[t])
            w = beta[t][:, None] * r
        writer = np.einsum("hdv,hv->hd", G, w)
        dw = np.einsum("hdv,hd->hv", G, k[t])
        reader = np.zeros_like(writer)
        if beta is not None:
            out["dbeta"][t] = (dw * r).sum(-1)
            dw = beta[t][:, None] * dw
            reader = -np.einsum("hdv,hv->hd", DS, dw)
            G = G - k[t][:, :, None] * dw[:, None, :]
        out["dk"][t] = writer + reader
        out["dv"][t] = dw
        through = (G * DS).sum(-1)
        out["dlog"][t] = through if gate.ndim == 3 else through.sum(-1)
        run = run + np.abs(q[t] * out["dq"][t]) + np.abs(k[t] * reader) + np.abs(k[t] * writer)
        size[t] = run
        G = _gate(gate, t) * G
    out["dS0"] = G
    return out, size if gate.ndim == 3 else size.sum(-1)
