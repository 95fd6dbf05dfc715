"""What a layer does around its recurrence, in 64 bits (numpy): the short convolution, the selective
recurrence token by token, the output norm, their gradients by formula, and first-order bounds of
what fp32 arithmetic may be off by.

A bound is in units of u = 2^-24: every operation adds its result once, a factor's relative error
carries over, sums of n terms add n times the sum of the terms' sizes. Functions: sigmoid and silu
of z are off by (|z| + 8) u (the exponent's rounding, exp2, a sum, a reciprocal and a product, with
room for two units each), softplus by (|v| + 8) u of itself, exp2 by 3 u beside its exponent's error.
A sigmoid or a decay below 2^-126, the smallest normal number of fp32 (an exponent below -87.3), is 0: up to
2^-126 off whatever its own size, TINY units of u.
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126 / U


def sigmoid(x):
    return 1 / (1 + np.exp(-x))


def softplus(x):
    return np.logaddexp(0, x)


# ---------------------------------------------------------------------------------
# convolution: one sequence; x [L][C], w [C][K], b [C] or None, kept [K-1][C]
# parts: (channels, norm, scale)
# ---------------------------------------------------------------------------------
def conv(x, w, b, kept, parts, silu=True, eps=1e-6, dy=None, dend=None):
    """(outputs, bounds): y and end, or with dy the gradients dx, dw, db, dkept."""
    L, C = x.shape
    K = w.shape[1]
    long = np.concatenate([kept, x])
    b = np.zeros(C) if b is None else b
    u = b + sum(w[:, j] * long[j:j + L] for j in range(K))
    eu = (K + 1) * (np.abs(b) + sum(np.abs(w[:, j] * long[j:j + L]) for j in range(K)))
    s = sigmoid(u) if silu else np.ones_like(u)
    a = u * s
    slope = s * (1 + u * (1 - s)) if silu else np.ones_like(u)
    ea = 1.1 * eu + np.abs(a) * (np.abs(u) + 8) + TINY * np.abs(u) if silu else eu
    eslope = 0.5 * eu + (1 + np.abs(u)) * (s * (np.abs(u) + 10) + TINY) if silu else 0 * eu
    y, ey = a.copy(), ea.copy()
    g = None if dy is None else dy.copy()
    eg = None if dy is None else 0 * dy
    c = 0
    for width, n, scale in parts:
        if n:
            cols = slice(c, c + width)
            A, EA = a[:, cols].reshape(L, width // n, n), ea[:, cols].reshape(L, width // n, n)
            S = (A * A).sum(-1, keepdims=True) + eps
            r = 1 / np.sqrt(S)
            er = r * ((np.abs(A) * EA).sum(-1, keepdims=True) / S + n / 2 + 4)
            y[:, cols] = (scale * A * r).reshape(L, width)
            ey[:, cols] = (scale * (EA * r + np.abs(A) * er + 2 * np.abs(A) * r)).reshape(L, width)
            if dy is not None:
                d = dy[:, cols].reshape(L, width // n, n)
                dot = (d * A).sum(-1, keepdims=True)
                edot = (np.abs(d) * EA).sum(-1, keepdims=True) + (n + 2) * np.abs(d * A).sum(-1, keepdims=True)
                inner = d - A * dot * r * r
                einner = (EA * np.abs(dot) * r * r + np.abs(A) * (edot * r * r + np.abs(dot) * 2 * r * er)
                          + 4 * (np.abs(d) + np.abs(A * dot) * r * r))
                g[:, cols] = (scale * r * inner).reshape(L, width)
                eg[:, cols] = (scale * (r * einner + er * np.abs(inner) + 2 * r * np.abs(inner))).reshape(L, width)
        c += width
    if dy is None:
        return {"y": y, "end": long[L:]}, {"y": ey}
    eg = eg * np.abs(slope) + np.abs(g) * eslope + np.abs(g * slope)
    g = g * slope
    d, ed = np.zeros_like(long), np.zeros_like(long)
    if dend is not None:
        d[L:] += dend
        ed[L:] += (K + 1) * np.abs(dend)
    dw, edw = np.zeros_like(w), np.zeros_like(w)
    for j in range(K):
        d[j:j + L] += w[:, j] * g
        ed[j:j + L] += np.abs(w[:, j]) * (eg + (K + 1) * np.abs(g))
        dw[:, j] = (g * long[j:j + L]).sum(0)
        edw[:, j] = ((eg + (L + 2) * np.abs(g)) * np.abs(long[j:j + L])).sum(0)
    return ({"dx": d[K - 1:], "dkept": d[:K - 1], "dw": dw, "db": g.sum(0)},
            {"dx": ed[K - 1:], "dkept": ed[:K - 1], "dw": edw, "db": (eg + (L + 2) * np.abs(g)).sum(0)})


# ---------------------------------------------------------------------------------
# selective recurrence: one sequence; x, dt, z [L][D], A [D][N], B, C [L][G][N], h0 [D][N]
# ---------------------------------------------------------------------------------
def selective(x, dt, A, B, C, h0, D=None, z=None, bias=None, soft=True, dout=None, dend=None):
    """(outputs, bounds): out and end, or with dout the gradients."""
    L, ch = x.shape
    G, N = B.shape[1:]
    spread = lambda m: np.repeat(m, ch // G, axis=0)  # [G][N] -> [D][N]
    raw = dt + (0 if bias is None else bias)
    v = np.abs(raw)
    delta = softplus(raw) if soft else raw
    ed = np.abs(delta) * (v + 8) if soft else np.abs(delta)
    skip = np.zeros(ch) if D is None else D
    h, eh = h0.copy(), np.zeros_like(h0)
    keep, y, ey = [], np.zeros((L, ch)), np.zeros((L, ch))
    for t in range(L):
        Bt, Ct = spread(B[t]), spread(C[t])
        a = np.exp(delta[t][:, None] * A)
        ea = a * (np.abs(A) * (ed[t] + 4 * np.abs(delta[t]))[:, None] + 3) + TINY
        w = (delta[t] * x[t])[:, None] * Bt
        ew = np.abs(w) * ((ed[t] / np.maximum(np.abs(delta[t]), 1e-300))[:, None] + 3)
        old, eold = h, eh
        h = a * old + w
        eh = a * eold + ea * np.abs(old) + ew + np.abs(h) + np.abs(a * old)
        y[t] = (Ct * h).sum(-1) + skip * x[t]
        ey[t] = (np.abs(Ct) * (eh + (N + 2) * np.abs(h))).sum(-1) + 2 * np.abs(skip * x[t])
        keep.append((a, ea, old, eold, h, eh))
    gate = np.ones_like(x) if z is None else z * sigmoid(z)
    eg = np.zeros_like(x) if z is None else np.abs(gate) * (np.abs(z) + 8) + TINY * np.abs(z)
    if dout is None:
        return {"out": y * gate, "end": h}, {"out": ey * np.abs(gate) + np.abs(y) * (eg + np.abs(gate)), "end": eh}
    dy = dout * gate
    edy = np.abs(dout) * (eg + np.abs(gate))
    o = {"dx": np.zeros_like(x), "ddt": np.zeros_like(x), "dB": np.zeros_like(B), "dC": np.zeros_like(C),
         "dA": np.zeros_like(A)}
    e = {k: np.zeros_like(val) for k, val in o.items()}
    g = np.zeros_like(h0) if dend is None else dend.copy()
    egr = np.zeros_like(g)
    per = ch // G
    group = lambda m: m.reshape(G, per, N).sum(1)
    for t in range(L - 1, -1, -1):
        a, ea, old, eold, h, eh = keep[t]
        Bt, Ct = spread(B[t]), spread(C[t])
        d, edt, dl = dy[t][:, None], edy[t][:, None], delta[t][:, None]
        edl = ed[t][:, None]
        g2 = g + Ct * d
        egr = egr + np.abs(Ct) * (edt + np.abs(d)) + np.abs(g2)
        g = g2
        dx_ = dl * x[t][:, None]
        edx_ = np.abs(x[t][:, None]) * (edl + np.abs(dl))
        o["dC"][t] = group(d * h)
        e["dC"][t] = group(edt * np.abs(h) + np.abs(d) * eh + (per + 2) * np.abs(d * h))
        o["dB"][t] = group(g * dx_)
        e["dB"][t] = group(egr * np.abs(dx_) + np.abs(g) * edx_ + (per + 2) * np.abs(g * dx_))
        s = (g * Bt).sum(-1)
        es = (egr * np.abs(Bt) + (N + 2) * np.abs(g * Bt)).sum(-1)
        ah, eah = a * old, ea * np.abs(old) + a * eold + np.abs(a * old)
        p = g * ah
        ep = egr * np.abs(ah) + np.abs(g) * eah + np.abs(p)
        f = (A * p).sum(-1)
        ef = (np.abs(A) * (ep + (N + 2) * np.abs(p))).sum(-1)
        o["dx"][t] = delta[t] * s + skip * dy[t]
        e["dx"][t] = (np.abs(delta[t]) * es + ed[t] * np.abs(s) + 2 * np.abs(delta[t] * s)
                      + np.abs(skip) * (edy[t] + 3 * np.abs(dy[t])))
        sig = sigmoid(raw[t]) if soft else np.ones(ch)
        o["ddt"][t] = (x[t] * s + f) * sig
        e["ddt"][t] = ((np.abs(x[t]) * es + ef + 2 * (np.abs(x[t] * s) + np.abs(f))) * sig
                       + np.abs(o["ddt"][t]) * (v[t] + 8) + np.abs(x[t] * s + f) * TINY)
        o["dA"] += dl * p
        e["dA"] += np.abs(dl) * ep + (edl + (L + 2) * np.abs(dl)) * np.abs(p)
        egr = a * egr + np.abs(g) * (ea + a)
        g = a * g
    o["dend"], e["dend"] = g, egr
    o["dD"] = (dy * x).sum(0)
    e["dD"] = ((edy + (L + 2) * np.abs(dy)) * np.abs(x)).sum(0)
    o["dbias"] = o["ddt"].sum(0)
    e["dbias"] = (e["ddt"] + (L + 2) * np.abs(o["ddt"])).sum(0)
    if z is not None:
        sig = sigmoid(z)
        slope = sig * (1 + z * (1 - sig))
        o["dz"] = dout * y * slope
        e["dz"] = np.abs(dout) * (ey * np.abs(slope) + np.abs(y) * (1 + np.abs(z)) * (sig * (np.abs(z) + 12) + TINY))
    return o, e


# ---------------------------------------------------------------------------------
# norm: x, z [rows][G][W], weight, bias [G or 1][W]
# ---------------------------------------------------------------------------------
def norm(x, z, w, b, gate="after", sig_gate=False, centred=False, eps=1e-5, dout=None):
    W = x.shape[-1]
    mean = lambda m: m.mean(-1, keepdims=True)
    n_sum = 48  # roundings of a group's sum: 32 values a lane and the steps between lanes
    if z is None:
        gt, eg, slope, eslope = np.ones_like(x), 0 * x, 0 * x, 0 * x
    else:
        s = sigmoid(z)
        gt = s if sig_gate else z * s
        eg = np.abs(gt) * (np.abs(z) + 8) + TINY * (1 + np.abs(z))
        slope = s * (1 - s) if sig_gate else s * (1 + z * (1 - s))
        eslope = (1 + np.abs(z)) * (s * (np.abs(z) + 12) + TINY)
    before = gate == "before"
    u = x * gt if before else x
    eu = np.abs(x) * (eg + np.abs(gt)) if before else 0 * x
    m = mean(u) if centred else 0 * mean(u)
    em = mean(eu) + (n_sum + 2) * mean(np.abs(u)) if centred else 0 * m
    v = u - m
    ev = eu + em + np.abs(v)
    var = mean(v * v) + eps
    r = 1 / np.sqrt(var)
    rel = mean(np.abs(v) * ev) / var + n_sum / 2 + 4
    n = v * r
    en = r * ev + np.abs(n) * (rel + 1)
    bb = 0 if b is None else b
    o = n * w + bb
    eo = np.abs(w) * en + 2 * (np.abs(n * w) + np.abs(bb))
    if dout is None:
        if before or z is None:
            return {"out": o}, {"out": eo}
        return {"out": o * gt}, {"out": eo * np.abs(gt) + np.abs(o) * (eg + np.abs(gt))}
    after = gate == "after" and z is not None
    do = dout * gt if after else dout
    edo = np.abs(dout) * (eg + np.abs(gt)) if after else 0 * dout
    dn = do * w
    edn = np.abs(w) * edo + np.abs(dn)
    sn = mean(dn * n)
    esn = mean(edn * np.abs(n) + np.abs(dn) * en + (n_sum + 2) * np.abs(dn * n))
    s1 = mean(dn) if centred else 0 * sn
    es1 = mean(edn + (n_sum + 2) * np.abs(dn)) if centred else 0 * sn
    du = r * (dn - n * sn - s1)
    edu = (r * (edn + en * np.abs(sn) + np.abs(n) * esn + es1 + 3 * (np.abs(dn) + np.abs(n * sn) + np.abs(s1)))
           + np.abs(du) * (rel + 1))
    rows = x.shape[0] * (x.shape[1] if w.shape[0] == 1 else 1)
    over = (0, 1) if w.shape[0] == 1 else (0,)
    keep = w.shape
    res = {"dx": du * gt if before else du, "dw": (do * n).sum(over).reshape(keep),
           "db": do.sum(over).reshape(keep)}
    err = {"dx": edu * np.abs(gt) + np.abs(du) * (eg + np.abs(gt)) if before else edu,
           "dw": (edo * np.abs(n) + np.abs(do) * en + (rows + 2) * np.abs(do * n)).sum(over).reshape(keep),
           "db": (edo + (rows + 2) * np.abs(do)).sum(over).reshape(keep)}
    if z is not None:
        k = du * x if before else dout * o
        ek = (edu + np.abs(du)) * np.abs(x) if before else np.abs(dout) * (eo + np.abs(o))
        res["dz"] = k * slope
        err["dz"] = ek * np.abs(slope) + np.abs(k) * eslope
    return res, err
