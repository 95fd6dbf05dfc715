"""Cases of the sequence-scan and serving-plan operators: what each reads, computes and returns.

  scan_forward   a packed batch of prompts through the layer's recurrence: every
                 token's output and each sequence's final state
  scan_backward  the gradients of the same for training
  scan_plan      request lengths -> sequence starts, chunk starts and the chunk table
  window_plan    decode lengths -> window positions, sketch parities, rows to update

The recurrence, per (sequence, head), with g the gate (a scalar per token, or one
value per key channel), is
    S_t = Diag(g_t) S_{t-1} + k_t w_t^T,   y_t = S_t^T q_t,
    w_t = v_t (mamba2)  or  beta_t (v_t - (Diag(g_t) S_{t-1})^T k_t) (gdn, kda).
The gates' gradient is returned for ln g, that is g * dL/dg.
"""
import random

import torch

own = False

RULES = {"mamba2": 0, "gdn": 1, "kda": 2}
CHUNK = 64    # tokens of one entry of the chunk table
PLAIN = 16    # tokens the plain form takes at once


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def _scan(op, rule, dtype, seqs, tokens, heads, d_k, d_v, ragged, carried):
    return {"op": op, "rule": rule, "dtype": dtype, "seqs": seqs, "tokens": tokens,
            "heads": heads, "d_k": d_k, "d_v": d_v, "ragged": ragged, "carried": carried}


def listed():
    return [
        # the tiny fp32 layer: two 16-token prompts, where only latency counts
        {"name": "forward mamba2 tiny", **_scan("forward", "mamba2", "f32", 2, 32, 4, 16, 32, False, True)},
        # one long prompt through a Gated DeltaNet layer, from an empty state
        {"name": "forward gdn long", **_scan("forward", "gdn", "bf16", 1, 8192, 32, 128, 128, False, False)},
        # a prefill batch of many requests of unlike lengths, continuing kept states
        {"name": "forward gdn ragged", **_scan("forward", "gdn", "bf16", 41, 8003, 32, 128, 128, True, True)},
        # the Mamba-2 layer (80 heads, 128 x 64), a few prompts
        {"name": "forward mamba2 batch", **_scan("forward", "mamba2", "bf16", 5, 5120, 80, 128, 64, True, False)},
        # the KDA layer, per-channel gates
        {"name": "forward kda batch", **_scan("forward", "kda", "bf16", 2, 4096, 32, 128, 128, False, True)},
        # one training step's backward through a Gated DeltaNet layer
        {"name": "backward gdn", **_scan("backward", "gdn", "bf16", 2, 4096, 32, 128, 128, False, False)},
        # packed documents of odd lengths through the Mamba-2 layer, with carried states
        {"name": "backward mamba2 ragged", **_scan("backward", "mamba2", "bf16", 6, 2011, 80, 128, 64, True, True)},
        # a small fp32 KDA layer, as in a gradient check
        {"name": "backward kda f32", **_scan("backward", "kda", "f32", 3, 777, 8, 64, 64, True, True)},
        # one serving batch of prompts
        {"name": "scan plan batch", "op": "scan_plan", "seqs": 37, "tokens": 9001},
        # a large offline batch
        {"name": "scan plan large", "op": "scan_plan", "seqs": 20000, "tokens": 4000000},
        # the serving step's batch of 256 rows, window 8
        {"name": "window plan batch", "op": "window_plan", "rows": 256, "window": 8},
        # the largest pools
        {"name": "window plan large", "op": "window_plan", "rows": 200000, "window": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "scan_plan", "window_plan"])
    if op == "scan_plan":
        seqs = _log_int(rng, 4, 20000)
        return {"op": op, "seqs": seqs, "tokens": _log_int(rng, 16 * seqs, min(4000000, 2000 * seqs))}
    if op == "window_plan":
        return {"op": op, "rows": _log_int(rng, 16, 200000), "window": rng.randint(1, 16)}
    rule = rng.choice(["mamba2", "gdn", "kda"])
    heads = rng.choice([1, 4, 5, 16, 32]) if rule != "mamba2" else rng.choice([1, 4, 16, 32, 80])
    d_k, d_v = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 128, 128])
    most = 8192 * 32 if op == "forward" else 4096 * 32
    if rule == "kda":
        most //= 2
    tokens = _log_int(rng, 1, min(8192, most // heads, 4096 if op == "backward" else 8192))
    seqs = _log_int(rng, 1, max(1, min(64 if op == "forward" else 6, tokens)))
    return _scan(op, rule, rng.choice(["bf16", "bf16", "f32"]), seqs, tokens, heads, d_k, d_v,
                 rng.random() < 0.7, rng.random() < 0.5)


def _lengths(case):
    """The case's request lengths: equal, or unlike (some of them zero)."""
    n, total = case["seqs"], case["tokens"]
    if case["op"] != "scan_plan" and not case["ragged"]:
        return [total // n + (i < total % n) for i in range(n)]
    rng = random.Random("%d %d" % (n, total))
    w = [0.0 if n > 2 and rng.random() < 0.05 else 0.05 + rng.random() ** 2 for _ in range(n)]
    w[rng.randrange(n)] += 1.0
    got = [int(total * x / sum(w)) for x in w]
    got[max(range(n), key=lambda i: got[i])] += total - sum(got)
    return got


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    if case["op"] == "scan_plan":
        # the arrays are sized for `tokens`; a batch fills them to a varying degree
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        lens = (lens * (0.8 + 0.2 * uniform(lens.numel()))).int()
        return {"case": case, "lengths": lens[torch.randperm(lens.numel(), generator=gen, device=dev)]}
    if case["op"] == "window_plan":
        lens = torch.randint(0, 100000, (case["rows"],), generator=gen, device=dev, dtype=torch.int32)
        idle = uniform(case["rows"]) < 0.03  # padding rows of the batch
        return {"case": case, "lengths": torch.where(idle, -1, lens)}

    n, T, H, dk, dv = (case[x] for x in ("seqs", "tokens", "heads", "d_k", "d_v"))
    t_in = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    q, k, v = normal(T, H, dk), normal(T, H, dk), normal(T, H, dv)
    if case["rule"] == "mamba2":
        q, k, v = (x / dk ** 0.5 for x in (q, k, v))
        rate = 1.0 + 15.0 * uniform(H)
        decay = torch.exp(-torch.nn.functional.softplus(-3.0 + 0.5 * normal(T, H)) * rate)
    else:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
        decay = (0.90 + 0.099 * uniform(T, H) if case["rule"] == "gdn"
                 else 0.85 + 0.149 * uniform(T, H, dk))
    s = {"case": case, "lens": _lengths(case), "q": q.to(t_in), "k": k.to(t_in), "v": v.to(t_in), "decay": decay,
         "beta": torch.sigmoid(normal(T, H)) if case["rule"] != "mamba2" else None,
         "state_in": 0.1 * normal(n, H, dk, dv) if case["carried"] else None}
    if case["op"] == "backward":
        s["dy"] = normal(T, H, dv)
        s["dstate"] = normal(n, H, dk, dv) if case["carried"] else None
    s["lengths"] = torch.tensor(s["lens"], dtype=torch.int32, device=dev)
    s["plan"] = _plain_scan_plan(s["lengths"], T)
    return s


# ---------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------
def _plain_scan_plan(lengths, total):
    """[seq_start (n + 1) | chunk_start (n + 1) | chunk_seq (total // 64 + n, -1 past the last chunk)]"""
    n = lengths.numel()
    start = torch.zeros(n + 1, dtype=torch.int64, device=lengths.device)
    start[1:] = lengths.clamp(min=0).long().cumsum(0).clamp(max=total)
    chunk = torch.zeros_like(start)
    chunk[1:] = ((start[1:] - start[:-1] + CHUNK - 1) // CHUNK).cumsum(0)
    entry = torch.arange(total // CHUNK + n, device=lengths.device)
    owner = (torch.searchsorted(chunk, entry, right=True) - 1).clamp(max=n - 1)
    owner = torch.where(entry < chunk[-1], owner, -1)
    return torch.cat([start, chunk, owner]).int()


def _plain_window_plan(lengths, window):
    n = lengths.numel()
    row = torch.arange(n, device=lengths.device)
    live = lengths >= 0
    tau = torch.where(live, lengths % window + 1, 0)
    parity = torch.where(live, lengths // window % 2, 0)
    full = tau == window
    place = torch.where(full, full.cumsum(0) - 1, n)
    rows = torch.full((n + 1,), -1, dtype=torch.int64, device=lengths.device)
    rows[place] = torch.where(full, row, -1)
    return {"tau": tau.int(), "parity": parity.int(), "update_rows": rows[:n].int(),
            "n_update": full.sum().int().reshape(1)}


def _token_places(s, width):
    """[sequences, padded length] of token indices, and which of them hold a token; padded to `width` tokens."""
    n, T = s["case"]["seqs"], s["case"]["tokens"]
    longest = -(-max(max(s["lens"]), 1) // width) * width
    start = s["plan"][:n].long()
    at = torch.arange(longest, device=start.device)
    holds = at < s["lengths"].long()[:, None]
    return torch.where(holds, start[:, None] + at, T), holds


def _spread(x, place, fill):
    """[tokens, ...] -> [sequences, padded length, ...], `fill` where there is no token."""
    return torch.cat([x, torch.full_like(x[:1], fill)])[place]


def _chunked(x, width):
    """[n, length, H, ...] -> [n, H, chunks, width, ...]"""
    return x.unflatten(1, (-1, width)).movedim(3, 1)


def _pairs(a, b, ratio):
    """sum_d a_id b_jd ratio_ij[d]; a ratio shared by all channels leaves a plain product."""
    if ratio.shape[-1] == 1:
        return (a @ b.transpose(-1, -2)) * ratio[..., 0]
    return (a[..., :, None, :] * b[..., None, :, :] * ratio).sum(-1)


def _plain_forward(q, k, v, log_g, beta, S):
    """Padded inputs in 32 bits ([n, H, chunks, PLAIN, ...]; log_g in 64) -> outputs in the same layout, final state.

    Within a chunk, with G_ij = g_{j+1} .. g_i: K_ij = k_i G_ij k_j (j < i), P_ij = q_i G_ij k_j (j <= i); the
    writes w solve (I + beta K) w = beta (v - G k S), the outputs are G q S + P w. The inverse of the unit lower
    triangular I + X is the product of I + (-X)^(2^m)."""
    c = log_g.cumsum(3)
    low = torch.ones(PLAIN, PLAIN, dtype=torch.bool, device=q.device).tril()
    ratio = torch.where(low[..., None], c[..., :, None, :] - c[..., None, :, :], -torch.inf).exp().float()
    P = _pairs(q, k, ratio)
    into, out, whole = c.exp().float(), (c[..., -1:, :] - c).exp().float(), c[..., -1, :].exp().float()
    qh, kt = into * q, (out * k).transpose(-1, -2)
    if beta is not None:
        kh = into * k
        X = -beta[..., None] * _pairs(k, k, ratio).tril(-1)
        eye = torch.eye(PLAIN, device=q.device)
        inv = eye + X
        X = X @ X
        inv = inv + inv @ X
        X = X @ X
        inv = inv + inv @ X
        X = X @ X
        inv = inv + inv @ X
    y = []
    for i in range(q.shape[2]):
        w = v[:, :, i]
        if beta is not None:
            w = inv[:, :, i] @ (beta[:, :, i, :, None] * (w - kh[:, :, i] @ S))
        y.append(qh[:, :, i] @ S + P[:, :, i] @ w)
        S = whole[:, :, i, :, None] * S + kt[:, :, i] @ w
    return torch.stack(y, 2), S


def _plain_scan(s):
    case = s["case"]
    place, holds = _token_places(s, PLAIN)
    q, k, v = (_chunked(_spread(s[x].float(), place, 0.0), PLAIN) for x in "qkv")
    log_g = _spread(s["decay"].double(), place, 1.0).log()
    log_g = _chunked(log_g if case["rule"] == "kda" else log_g[..., None], PLAIN)
    beta = _chunked(_spread(s["beta"], place, 0.0), PLAIN) if s["beta"] is not None else None
    S = s["state_in"]
    if S is None:
        S = torch.zeros(case["seqs"], case["heads"], case["d_k"], case["d_v"], device="cuda")

    def packed(x):
        return x.movedim(1, 3).flatten(1, 2)[holds]

    if case["op"] == "forward":
        y, last = _plain_forward(q, k, v, log_g, beta, S)
        return {"y": packed(y), "state": last}
    leaves = [x.detach().requires_grad_() for x in (q, k, v, log_g, S)]
    leaves += [beta.detach().requires_grad_()] if beta is not None else []
    with torch.enable_grad():
        y, last = _plain_forward(*leaves[:4], leaves[5] if beta is not None else None, leaves[4])
        dy = _chunked(_spread(s["dy"], place, 0.0), PLAIN)
        total = (y * dy).sum()
        if s["dstate"] is not None:
            total = total + (last * s["dstate"]).sum()
    got = torch.autograd.grad(total, leaves)
    t_in = s["q"].dtype
    dlog = packed(got[3]).float()
    out = {"dq": packed(got[0]).to(t_in), "dk": packed(got[1]).to(t_in), "dv": packed(got[2]).to(t_in),
           "dlog_decay": dlog if case["rule"] == "kda" else dlog[..., 0], "dstate_in": got[4]}
    if beta is not None:
        out["dbeta"] = packed(got[5])
    return out


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "scan_plan":
        return _plain_scan_plan(state["lengths"], case["tokens"])
    if case["op"] == "window_plan":
        return _plain_window_plan(state["lengths"], case["window"])
    return _plain_scan(state)


def _own(s):
    import sketched_recurrent_state_amd as ssm
    case = s["case"]
    if case["op"] == "scan_plan":
        plan = torch.empty(2 * (case["seqs"] + 1) + case["tokens"] // CHUNK + case["seqs"],
                           dtype=torch.int32, device="cuda")
        ssm.scan_plan(s["lengths"], case["tokens"], plan)
        return plan
    if case["op"] == "window_plan":
        d = ssm.Dims.make("gdn", "bf16", case["rows"], 1, 128, 128, case["window"], 8)
        tau, parity, rows = torch.empty(3, case["rows"], dtype=torch.int32, device="cuda")
        count = torch.empty(1, dtype=torch.int32, device="cuda")
        ssm.window_plan(d, s["lengths"], tau, parity, rows, count)
        return {"tau": tau, "parity": parity, "update_rows": rows, "n_update": count}
    d = ssm.Dims.make(case["rule"], case["dtype"], case["seqs"], case["heads"], case["d_k"], case["d_v"], 8, 8)
    tokens = (case["tokens"], s["plan"], s["q"], s["k"], s["v"], s["decay"], s["beta"])
    shape = (case["seqs"], case["heads"], case["d_k"], case["d_v"])
    if case["op"] == "forward":
        y = torch.empty(case["tokens"], case["heads"], case["d_v"], device="cuda")
        last = torch.empty(shape, device="cuda")
        ssm.scan_forward(d, *tokens, last, y, state_in=s["state_in"])
        return {"y": y, "state": last}
    out = {"dq": torch.empty_like(s["q"]), "dk": torch.empty_like(s["k"]), "dv": torch.empty_like(s["v"]),
           "dlog_decay": torch.empty_like(s["decay"]), "dstate_in": torch.empty(shape, device="cuda")}
    if s["beta"] is not None:
        out["dbeta"] = torch.empty_like(s["beta"])
    ssm.scan_backward(d, *tokens, s["dy"], out["dq"], out["dk"], out["dv"], out["dlog_decay"], out.get("dbeta"),
                      state_in=s["state_in"], dstate=s["dstate"], dstate_in=out["dstate_in"])
    return out


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------
def work(case):
    if case["op"] == "scan_plan":
        n, entries = case["seqs"], case["tokens"] // CHUNK + case["seqs"]
        return {"bytes": 4 * (n + 2 * (n + 1) + entries), "flops": 4 * n + entries}
    if case["op"] == "window_plan":
        return {"bytes": 16 * case["rows"], "flops": 4 * case["rows"]}
    n, T, H, dk, dv = (case[x] for x in ("seqs", "tokens", "heads", "d_k", "d_v"))
    delta = case["rule"] != "mamba2"
    e = 2 if case["dtype"] == "bf16" else 4
    gates = 4 * ((dk if case["rule"] == "kda" else 1) + delta)
    inputs, states = (2 * dk + dv) * e + gates, 4 * n * H * dk * dv
    product = 2 * T * H * dk * dv  # one token's product with the state, over all tokens
    if case["op"] == "forward":
        return {"bytes": T * H * (inputs + 4 * dv) + states * (1 + case["carried"]), "flops": product * (2 + delta)}
    # the states again, then their gradients: outputs and writes against both
    return {"bytes": T * H * (2 * inputs + 4 * dv) + states * (1 + 2 * case["carried"]),
            "flops": product * (5 + 3 * delta)}


# ---------------------------------------------------------------------------------
# the definition, token by token in 64 bits
# ---------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] not in ("forward", "backward"):
        return None
    s = prepare(case, seed)
    n, H, dk, dv = (case[x] for x in ("seqs", "heads", "d_k", "d_v"))
    lens, first = s["lens"], [sum(s["lens"][:i]) for i in range(n)]
    steps = max(lens)
    back = case["op"] == "backward"
    if back and 8.0 * steps * n * H * dk * dv > 1e11:
        return None
    delta, f64 = case["rule"] != "mamba2", torch.float64
    S = torch.zeros(n, H, dk, dv, dtype=f64, device="cuda") if s["state_in"] is None else s["state_in"].to(f64)
    names = ["q", "k", "v", "decay"] + (["beta"] if delta else []) + (["dy"] if back else [])
    wide = {x: s[x].to(f64) for x in names}
    wide["decay"] = wide["decay"].reshape(case["tokens"], H, -1)

    def at(t):
        """The sequences that still have a token at step t, and those tokens."""
        rows = [i for i in range(n) if t < lens[i]]
        here = torch.tensor([first[i] + t for i in rows], device="cuda")
        return torch.tensor(rows, device="cuda"), here

    y = torch.zeros(case["tokens"], H, dv, dtype=f64, device="cuda")
    kept = []
    for t in range(steps):
        rows, here = at(t)
        old = S if rows.numel() == n else S[rows]
        k, w = wide["k"][here], wide["v"][here]
        decayed = wide["decay"][here].unsqueeze(-1) * old
        if delta:
            w = wide["beta"][here].unsqueeze(-1) * (w - (decayed * k.unsqueeze(-1)).sum(2))
        new = decayed + k.unsqueeze(-1) * w.unsqueeze(2)
        y[here] = (new * wide["q"][here].unsqueeze(-1)).sum(2)
        if back:
            kept.append((rows, here, decayed))
        if rows.numel() == n:
            S = new
        else:
            S[rows] = new
    if not back:
        return {"y": y, "state": S}
    G = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].to(f64)
    out = {"d" + x: torch.zeros_like(wide[x]) for x in ("q", "k", "v")}
    out["dlog_decay"] = torch.zeros_like(wide["decay"])
    if delta:
        out["dbeta"] = torch.zeros_like(wide["beta"])
    while kept:
        rows, here, decayed = kept.pop()
        q, k, v, dy = (wide[x][here] for x in ("q", "k", "v", "dy"))
        g = G[rows] + q.unsqueeze(-1) * dy.unsqueeze(2)
        w = v
        if delta:
            beta = wide["beta"][here].unsqueeze(-1)
            missed = v - (decayed * k.unsqueeze(-1)).sum(2)
            w = beta * missed
        out["dq"][here] = (decayed * dy.unsqueeze(2)).sum(-1) + k * (w * dy).sum(-1, keepdim=True)
        from_write = (g * w.unsqueeze(2)).sum(-1)
        dw = (g * k.unsqueeze(-1)).sum(2)
        if delta:
            out["dbeta"][here] = (dw * missed).sum(-1)
            dw = beta * dw
            from_write = from_write - (decayed * dw.unsqueeze(2)).sum(-1)
            g = g - k.unsqueeze(-1) * dw.unsqueeze(2)
        out["dk"][here], out["dv"][here] = from_write, dw
        through = (g * decayed).sum(-1)
        out["dlog_decay"][here] = through if case["rule"] == "kda" else through.sum(-1, keepdim=True)
        G[rows] = wide["decay"][here].unsqueeze(-1) * g
    if case["rule"] != "kda":
        out["dlog_decay"] = out["dlog_decay"][..., 0]
    out["dstate_in"] = G
    return out
