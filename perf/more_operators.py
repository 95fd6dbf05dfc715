"""Cases of the operators around a layer's recurrence: what each reads, computes and returns.

  conv       the short causal convolution of a layer's inputs (per channel, 2 to 4 taps) with its
             activation and the l2 norm of queries and keys per head: packed prompts (forward),
             their gradients (backward), a batch of single tokens (step)
  selective  the selective state space recurrence (a decay per channel and state): packed prompts,
             their gradients, a batch of single tokens
  norm       the norm of groups of channels with a gate, over a layer's outputs: forward, backward

Convolution, for token t of a sequence and channel c, x before the sequence from the kept state
(its last K - 1 inputs) or zero:
    u_t = bias + sum_j w_j x_{t-(K-1)+j},  a = silu(u),  y = a  or  scale a / sqrt(sum_head a^2 + eps).
Selective recurrence, for channel d and state n, with B and C shared by a group of channels:
    delta = softplus(dt + dt_bias),  h <- exp(delta A) h + delta x B,
    y = sum_n C h + D x,  out = y silu(z).
Norm, per token and group: u = x (or x silu(z)), n = (u - mean) / sqrt(var + eps), the mean taken as
zero without centring; o = n w + b; out = o silu(z) (or o).
"""
import functools
import random

import torch

own = False

CHUNK = 64        # tokens of one entry of the chunk table
NORM_EPS = 1e-6   # of the queries' and keys' l2 norm
EPS = 1e-5        # of the output norm


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def _conv(way, dtype, seqs, tokens, taps, heads, d_k, d_v, plain, normed, bias, ragged, carried):
    """heads > 0: queries, keys and values of heads channels each; else `plain` channels."""
    return {"op": "conv", "way": way, "dtype": dtype, "seqs": seqs, "tokens": tokens, "taps": taps, "heads": heads,
            "d_k": d_k, "d_v": d_v, "plain": plain, "normed": normed, "bias": bias, "ragged": ragged,
            "carried": carried}


def _selective(way, dtype, seqs, tokens, channels, states, groups, gated, ragged, carried):
    return {"op": "selective", "way": way, "dtype": dtype, "seqs": seqs, "tokens": tokens, "channels": channels,
            "states": states, "groups": groups, "gated": gated, "ragged": ragged, "carried": carried}


def _norm(way, x_dtype, dtype, rows, groups, width, gate, shared, centred, bias):
    """gate: "after" the norm, "before" it, or "none"."""
    return {"op": "norm", "way": way, "x_dtype": x_dtype, "dtype": dtype, "rows": rows, "groups": groups,
            "width": width, "gate": gate, "shared": shared, "centred": centred, "bias": bias}


def listed():
    return [
        # the tiny fp32 layer's decode step: two rows, where only latency counts
        {"name": "conv step tiny", **_conv("step", "f32", 2, 2, 4, 4, 16, 32, 0, True, False, False, True)},
        # one decode step of a serving batch before a Gated DeltaNet layer (32 heads, 128 x 128)
        {"name": "conv step batch", **_conv("step", "bf16", 256, 256, 4, 32, 128, 128, 0, True, False, False, True)},
        # one long prompt before that layer: queries and keys normalised per head
        {"name": "conv forward gdn", **_conv("forward", "bf16", 1, 8192, 4, 32, 128, 128, 0, True, False, False, False)},
        # a prefill batch of many requests of unlike lengths, 80 heads of 64 as plain channels, kept inputs
        {"name": "conv forward ragged", **_conv("forward", "bf16", 41, 8003, 4, 0, 0, 0, 5120, False, True, True, True)},
        # one training step's backward before the Gated DeltaNet layer
        {"name": "conv backward gdn", **_conv("backward", "bf16", 2, 8192, 4, 32, 128, 128, 0, True, False, False, False)},
        # one long prompt through a selective layer
        {"name": "selective forward", **_selective("forward", "bf16", 1, 8192, 5120, 16, 1, True, False, False)},
        # a prefill batch of many requests of unlike lengths, continuing kept states
        {"name": "selective forward ragged", **_selective("forward", "bf16", 41, 8003, 5120, 16, 1, True, True, True)},
        # one training step's backward through a selective layer
        {"name": "selective backward", **_selective("backward", "bf16", 2, 4096, 5120, 16, 1, True, False, False)},
        # a small fp32 layer with two groups, as in a gradient check
        {"name": "selective backward f32", **_selective("backward", "f32", 3, 777, 512, 16, 2, False, True, True)},
        # one decode step of a serving batch through a selective layer
        {"name": "selective step batch", **_selective("step", "bf16", 256, 256, 5120, 16, 1, True, False, True)},
        # a prompt's outputs of the Gated DeltaNet layer, normalised per head, gated after
        {"name": "norm forward gdn", **_norm("forward", "f32", "bf16", 8192, 32, 128, "after", True, False, False)},
        # training: the Mamba-2 layer's outputs (80 heads of 64), one group, gated before
        {"name": "norm backward mamba2", **_norm("backward", "f32", "bf16", 4096, 1, 5120, "before", False, False, False)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv", "conv", "selective", "selective", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        width = 8 * _log_int(rng, 2, 640)
        groups = _log_int(rng, 1, max(1, 5120 // width))
        way = rng.choice(["forward", "backward"])
        most = (8192 * 4096 if way == "forward" else 4096 * 5120) // (2 if dtype == "f32" else 1)
        return _norm(way, rng.choice(["f32", dtype]), dtype, _log_int(rng, 1, max(1, most // (groups * width))), groups,
                     width, rng.choice(["after", "before", "none"]), rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.5)
    way = rng.choice(["forward", "backward", "step"])
    if op == "conv":
        heads, d_k, d_v, plain = 0, 0, 0, 0
        if rng.random() < 0.6:
            heads = rng.choice([1, 3, 4, 16, 32])
            d_k, d_v = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 128, 128])
        else:
            plain = 8 * _log_int(rng, 2, 1024)
        channels = heads * (2 * d_k + d_v) + plain
        most = min(8192, (8192 if way != "step" else 256) * 12288 // channels)
        tokens = _log_int(rng, 1, (most if way != "step" else min(most, 512)) // (2 if dtype == "f32" else 1))
        seqs = tokens if way == "step" else _log_int(rng, 1, min(64, tokens))
        return _conv(way, dtype, seqs, tokens, rng.choice([2, 3, 4, 4]), heads, d_k, d_v, plain,
                     heads > 0 and rng.random() < 0.7, rng.random() < 0.5, way != "step" and rng.random() < 0.7,
                     way == "step" or rng.random() < 0.5)
    groups, states = rng.choice([1, 1, 2, 4]), rng.choice([8, 16, 16, 16, 32, 64])
    channels = 16 * groups * _log_int(rng, 2, 320 // groups)
    most = {"forward": 8192, "backward": 4096, "step": 256}[way] * 5120 * 16 // (channels * states)
    most = max(1, min(8192 if way != "step" else 512, most // (2 if dtype == "f32" else 1)))
    tokens = _log_int(rng, 1, most)
    seqs = tokens if way == "step" else _log_int(rng, 1, min(64, tokens))
    return _selective(way, dtype, seqs, tokens, channels, states, groups, rng.random() < 0.7,
                      way != "step" and rng.random() < 0.7, way == "step" or rng.random() < 0.5)


def _lengths(case):
    """The case's request lengths: equal, or unlike (some of them zero)."""
    n, total = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [total // n + (i < total % n) for i in range(n)]
    rng = random.Random("%d %d" % (n, total))
    w = [0.0 if n > 2 and rng.random() < 0.05 else 0.05 + rng.random() ** 2 for _ in range(n)]
    w[rng.randrange(n)] += 1.0
    got = [int(total * x / sum(w)) for x in w]
    got[max(range(n), key=lambda i: got[i])] += total - sum(got)
    return got


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _parts(case):
    """(channels, channels of a head to normalise over or 0, scale) of each array that is convolved."""
    if not case["heads"]:
        return [(case["plain"], 0, 1.0)]
    keys = case["heads"] * case["d_k"]
    over = case["d_k"] if case["normed"] else 0
    return [(keys, over, case["d_k"] ** -0.5 if over else 1.0), (keys, over, 1.0),
            (case["heads"] * case["d_v"], 0, 1.0)]


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

    t_in = _type(case["dtype"])
    s = {"case": case}
    if case["op"] == "norm":
        rows, groups, width = case["rows"], case["groups"], case["width"]
        own_weights = 1 if case["shared"] else groups
        s["x"] = normal(rows, groups, width).to(_type(case["x_dtype"]))
        # the gate is a column range of the layer's input projection
        s["z"] = (normal(rows, groups * width + 64).to(t_in)[:, :groups * width] if case["gate"] != "none" else None)
        s["weight"] = 1.0 + 0.2 * normal(own_weights, width)
        s["bias"] = 0.2 * normal(own_weights, width) if case["bias"] else None
        if case["way"] == "backward":
            s["dout"] = normal(rows, groups, width).to(t_in)
        return s
    n, T = case["seqs"], case["tokens"]
    if case["way"] != "step":
        s["lens"] = _lengths(case)
        s["plan"] = _plain_plan(torch.tensor(s["lens"], dtype=torch.int32, device=dev), T)
    pool = n
    if case["way"] == "step":  # the batch's rows are somewhere in a larger pool
        pool = n + n // 4 + 1
        s["slot"] = torch.randperm(pool, generator=gen, device=dev)[:n].int()
    if case["op"] == "conv":
        parts = _parts(case)
        C, K = sum(p[0] for p in parts), case["taps"]
        # the parts are column ranges of one input projection, which holds other columns too
        projected = normal(T, C + 64).to(t_in)
        s["x"] = list(projected[:, :C].split([p[0] for p in parts], 1))
        s["weight"] = normal(C, K) / K ** 0.5
        s["bias"] = 0.1 * normal(C) if case["bias"] else None
        s["state"] = normal(pool, K - 1, C).to(t_in) if case["carried"] else None
        if case["way"] == "backward":
            s["dy"] = [normal(T, p[0]).to(t_in) for p in parts]
            s["dstate"] = normal(n, K - 1, C).to(t_in) if case["carried"] else None
        return s
    D, N, G = case["channels"], case["states"], case["groups"]
    s["x"] = normal(T, D).to(t_in)
    s["dt"] = normal(T, D).to(t_in)
    # steps of 0.001 to 0.1 about the bias, as layers start out
    step = torch.exp(uniform(D) * (torch.tensor(0.1).log() - torch.tensor(0.001).log()).item() - 6.907755)
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32).repeat(D, 1) * (0.8 + 0.4 * uniform(D, N))
    s["B"], s["C"] = normal(T, 48 + 2 * G * N).to(t_in)[:, 48:].reshape(T, 2, G, N).unbind(1)
    s["D"] = 1.0 + 0.1 * normal(D)
    s["z"] = normal(T, D + 64).to(t_in)[:, :D] if case["gated"] else None
    s["state"] = 0.3 * normal(pool, D, N) if case["carried"] else None
    if case["way"] == "backward":
        s["dy"] = normal(T, D).to(t_in)
        s["dstate"] = normal(n, D, N) if case["carried"] else None
    return s


# ---------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------
def _plain_plan(lengths, total):
    """[seq_start (n + 1) | chunk_start (n + 1) | chunk_seq (total // 64 + n, -1 past the last chunk)]"""
    n = lengths.numel()
    start = torch.zeros(n + 1, dtype=torch.int64, device=lengths.device)
    start[1:] = lengths.long().cumsum(0)
    chunk = torch.zeros_like(start)
    chunk[1:] = ((start[1:] - start[:-1] + CHUNK - 1) // CHUNK).cumsum(0)
    entry = torch.arange(total // CHUNK + n, device=lengths.device)
    owner = (torch.searchsorted(chunk, entry, right=True) - 1).clamp(max=n - 1)
    return torch.cat([start, chunk, torch.where(entry < chunk[-1], owner, -1)]).int()


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _sequence_starts(s):
    """Sequence starts (n + 1), and each token's sequence."""
    n, T = s["case"]["seqs"], s["case"]["tokens"]
    start = s["plan"][:n + 1].long()
    token = torch.arange(T, device=start.device)
    return start, torch.searchsorted(start[1:], token, right=True)


def _plain_conv(rows, at, weight, bias, case):
    """rows[at] [tokens, taps, channels] with the taps -> the parts' outputs."""
    u = (rows[at] * weight.t()).sum(1)
    a = _silu(u if bias is None else u + bias)
    parts = _parts(case)
    split = a.split([p[0] for p in parts], 1)

    def normed(x, over, scale):
        if not over:
            return x
        x = x.unflatten(1, (-1, over))
        return (scale * x / (x.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()).flatten(1)

    return [normed(x, over, scale) for x, (_, over, scale) in zip(split, parts)]


def _plain_conv_prompts(s):
    case = s["case"]
    n, T, K = case["seqs"], case["tokens"], case["taps"]
    t_in = _type(case["dtype"])
    start, seq = _sequence_starts(s)
    back = torch.arange(1 - K, 1, device="cuda")  # taps, oldest first

    def places(first_token, sequence):
        """Rows of [tokens | kept states | zeros] for tokens first_token + back of their sequences."""
        token = first_token[:, None] + back
        kept = T + sequence[:, None] * (K - 1) + (token - start[sequence][:, None] + K - 1)
        return torch.where(token >= start[sequence][:, None], token, kept)

    at = places(torch.arange(T, device="cuda"), seq)
    every = torch.arange(n, device="cuda")
    last = places(start[1:] - 1, every)[:, 1:]
    x = torch.cat([x.float() for x in s["x"]], 1)
    C = x.shape[1]
    state = torch.zeros(n, K - 1, C, device="cuda") if s["state"] is None else s["state"].float()
    if case["way"] == "forward":
        rows = torch.cat([x, state.flatten(0, 1)])
        y = _plain_conv(rows, at, s["weight"], s["bias"], case)
        return {"y": [v.to(t_in) for v in y], "state": rows[last].to(t_in)}
    leaves = [v.detach().requires_grad_() for v in (x, state, s["weight"])]
    leaves += [s["bias"].detach().requires_grad_()] if s["bias"] is not None else []
    with torch.enable_grad():
        rows = torch.cat([leaves[0], leaves[1].flatten(0, 1)])
        y = torch.cat(_plain_conv(rows, at, leaves[2], leaves[3] if s["bias"] is not None else None, case), 1)
        total = (y * torch.cat([v.float() for v in s["dy"]], 1)).sum()
        if s["dstate"] is not None:
            total = total + (rows[last] * s["dstate"].float()).sum()
    got = torch.autograd.grad(total, leaves)
    out = {"dx": [v.contiguous().to(t_in) for v in got[0].split([p[0] for p in _parts(case)], 1)], "dweight": got[2]}
    if s["bias"] is not None:
        out["dbias"] = got[3]
    if s["state"] is not None:
        out["dstate_in"] = got[1].to(t_in)
    return out


def _plain_conv_step(s):
    case = s["case"]
    t_in, slot = _type(case["dtype"]), s["slot"].long()
    rows = torch.cat([s["state"][slot], torch.cat(s["x"], 1)[:, None]], 1)  # [rows, taps, channels]
    n, K, C = rows.shape
    at = torch.arange(n * K, device="cuda").reshape(n, K)
    y = _plain_conv(rows.float().reshape(n * K, C), at, s["weight"], s["bias"], case)
    s["state"][slot] = rows[:, 1:]
    return {"y": [v.to(t_in) for v in y], "state": s["state"]}


def _per_channel(x, channels):
    """[tokens, groups, states] -> [tokens, channels, states]"""
    return x.repeat_interleave(channels // x.shape[1], 1)


def _plain_selective(x, delta, A, B, C, D, z, h0, first, longest):
    """Outputs and every token's state. first: the first tokens of the sequences that hold any, whose
    states before are h0. Pairs (decay, state) are joined over twice as many tokens at a time."""
    D_ch = x.shape[1]
    a = torch.exp(delta[..., None] * A)
    h = (delta * x)[..., None] * _per_channel(B, D_ch)
    if h0 is not None:
        h = h.index_add(0, first, a[first] * h0)
    a = a.index_fill(0, first, 0.0)
    k = 1
    while k < longest:
        h = torch.cat([h[:k], h[k:] + a[k:] * h[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    y = (h * _per_channel(C, D_ch)).sum(-1) + D * x
    return (y if z is None else y * _silu(z)), h


def _plain_selective_prompts(s):
    case = s["case"]
    n, t_in = case["seqs"], _type(case["dtype"])
    start, _ = _sequence_starts(s)
    holds = torch.tensor([length > 0 for length in s["lens"]], device="cuda")
    first, last, longest = start[:-1][holds], start[1:][holds] - 1, max(s["lens"])
    wide = [s[k].float() for k in ("x", "dt", "B", "C", "A", "D", "dt_bias")]
    z = None if s["z"] is None else s["z"].float()

    def through(x, dt, B, C, A, D, dt_bias, z, state):
        out, h = _plain_selective(x, _softplus(dt + dt_bias), A, B, C, D, z,
                                  None if state is None else state[holds], first, longest)
        end = torch.zeros(n, *h.shape[1:], device="cuda") if state is None else state
        return out, end.index_put((holds.nonzero()[:, 0],), h[last])

    if case["way"] == "forward":
        out, end = through(*wide, z, s["state"])
        return {"y": out.to(t_in), "state": end}
    leaves = [v.detach().requires_grad_() for v in wide]
    gate = None if z is None else z.detach().requires_grad_()
    state = None if s["state"] is None else s["state"].detach().requires_grad_()
    with torch.enable_grad():
        out, end = through(*leaves, gate, state)
        total = (out * s["dy"].float()).sum()
        if s["dstate"] is not None:
            total = total + (end * s["dstate"]).sum()
    more = [v for v in (gate, state) if v is not None]
    got = torch.autograd.grad(total, leaves + more)
    out = {"dx": got[0].to(t_in), "ddt": got[1].to(t_in), "dB": got[2].to(t_in), "dC": got[3].to(t_in),
           "dA": got[4], "dD": got[5], "ddt_bias": got[6]}
    if gate is not None:
        out["dz"] = got[7].to(t_in)
    if state is not None:
        out["dstate_in"] = got[-1]
    return out


def _plain_selective_step(s):
    case = s["case"]
    D, slot, t_in = case["channels"], s["slot"].long(), _type(case["dtype"])
    x = s["x"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["A"]) * s["state"][slot] + (delta * x)[..., None] * _per_channel(s["B"].float(), D)
    s["state"][slot] = h
    y = (h * _per_channel(s["C"].float(), D)).sum(-1) + s["D"] * x
    return {"y": (y if s["z"] is None else y * _silu(s["z"].float())).to(t_in), "state": s["state"]}


def _plain_norm(x, z, weight, bias, case):
    gate = None if z is None else _silu(z).reshape(x.shape)
    u = x * gate if case["gate"] == "before" else x
    if case["centred"]:
        u = u - u.mean(-1, keepdim=True)
    o = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * weight
    if bias is not None:
        o = o + bias
    return o * gate if case["gate"] == "after" else o


def _plain_norms(s):
    case = s["case"]
    t_in = _type(case["dtype"])
    z = None if s["z"] is None else s["z"].float()
    if case["way"] == "forward":
        return _plain_norm(s["x"].float(), z, s["weight"], s["bias"], case).to(t_in)
    given = {"dx": s["x"].float(), "dweight": s["weight"], "dbias": s["bias"], "dz": z}
    leaves = {k: v.detach().requires_grad_() for k, v in given.items() if v is not None}
    with torch.enable_grad():
        out = _plain_norm(leaves["dx"], leaves.get("dz"), leaves["dweight"], leaves.get("dbias"), case)
    got = dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), s["dout"].float())))
    got["dx"] = got["dx"].to(_type(case["x_dtype"]))
    if z is not None:
        got["dz"] = got["dz"].to(t_in)
    return got


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "norm":
        return _plain_norms(state)
    if case["op"] == "conv":
        return _plain_conv_step(state) if case["way"] == "step" else _plain_conv_prompts(state)
    return _plain_selective_step(state) if case["way"] == "step" else _plain_selective_prompts(state)


@functools.lru_cache(None)
def _dims(items):
    """The dimensions that a user's program keeps beside its weights."""
    import sketched_recurrent_state_amd as ssm
    case = dict(items)
    if case["op"] == "norm":
        return ssm.NormDims.make(case["x_dtype"], case["dtype"], case["groups"], case["width"], gate=case["gate"],
                                 activation="silu", shared=case["shared"], centred=case["centred"], eps=EPS)
    if case["op"] == "conv":
        parts = _parts(case)
        return ssm.ConvDims.make(case["dtype"], case["seqs"], case["taps"], [p[0] for p in parts],
                                 norm=[p[1] for p in parts], scale=[p[2] for p in parts], activation="silu",
                                 eps=NORM_EPS)
    return ssm.SelectiveDims.make(case["dtype"], case["seqs"], case["channels"], case["states"],
                                  groups=case["groups"], softplus=True)


def _own(s):
    import sketched_recurrent_state_amd as ssm
    case = s["case"]
    d = _dims(tuple(case.items()))
    t_in, T, n = _type(case["dtype"]), case["tokens"] if "tokens" in case else 0, case.get("seqs")
    if case["op"] == "norm":
        if case["way"] == "forward":
            out = torch.empty(s["x"].shape, dtype=t_in, device="cuda")
            ssm.gated_norm(d, case["rows"], s["x"], s["z"], s["weight"], s["bias"], out)
            return out
        got = {"dx": torch.empty_like(s["x"]), "dweight": torch.empty_like(s["weight"])}
        if s["bias"] is not None:
            got["dbias"] = torch.empty_like(s["bias"])
        if s["z"] is not None:
            got["dz"] = torch.empty(s["z"].shape, dtype=t_in, device="cuda")
        ssm.gated_norm_backward(d, case["rows"], s["x"], s["z"], s["weight"], s["bias"], s["dout"], got["dx"],
                                got.get("dz"), got["dweight"], got.get("dbias"))
        return got
    if case["op"] == "conv":
        K, C = case["taps"], s["weight"].shape[0]
        like = [torch.empty(x.shape, dtype=t_in, device="cuda") for x in s["x"]]
        if case["way"] == "step":
            ssm.conv_step(d, s["x"], s["weight"], s["bias"], s["state"], like, slot=s["slot"],
                          num_slots=s["state"].shape[0])
            return {"y": like, "state": s["state"]}
        if case["way"] == "forward":
            last = torch.empty(n, K - 1, C, dtype=t_in, device="cuda")
            ssm.conv_forward(d, T, s["plan"], s["x"], s["weight"], s["bias"], like, last, state_in=s["state"])
            return {"y": like, "state": last}
        out = {"dx": like, "dweight": torch.empty_like(s["weight"])}
        if s["bias"] is not None:
            out["dbias"] = torch.empty_like(s["bias"])
        if s["state"] is not None:
            out["dstate_in"] = torch.empty_like(s["state"])
        ssm.conv_backward(d, T, s["plan"], s["x"], s["weight"], s["bias"], s["dy"], like, out["dweight"],
                          out.get("dbias"), state_in=s["state"], dstate=s["dstate"], dstate_in=out.get("dstate_in"))
        return out
    inputs = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"]}
    y = torch.empty(s["x"].shape, dtype=t_in, device="cuda")
    if case["way"] == "step":
        ssm.selective_step(d, *inputs, s["state"], y, **more, slot=s["slot"], num_slots=s["state"].shape[0])
        return {"y": y, "state": s["state"]}
    if case["way"] == "forward":
        last = torch.empty(n, case["channels"], case["states"], device="cuda")
        ssm.selective_forward(d, T, s["plan"], *inputs, last, y, **more, state_in=s["state"])
        return {"y": y, "state": last}
    shape = (T, case["groups"], case["states"])
    out = {"dx": y, "ddt": torch.empty_like(y), "dA": torch.empty_like(s["A"]),
           "dB": torch.empty(shape, dtype=t_in, device="cuda"), "dC": torch.empty(shape, dtype=t_in, device="cuda"),
           "dD": torch.empty_like(s["D"]), "ddt_bias": torch.empty_like(s["dt_bias"])}
    if s["z"] is not None:
        out["dz"] = torch.empty_like(y)
    if s["state"] is not None:
        out["dstate_in"] = torch.empty_like(s["state"])
    ssm.selective_backward(d, T, s["plan"], *inputs, s["dy"], out["dx"], out["ddt"], out["dA"], out["dB"], out["dC"],
                           **more, dD=out["dD"], dz=out.get("dz"), ddt_bias=out["ddt_bias"], state_in=s["state"],
                           dstate=s["dstate"], dstate_in=out.get("dstate_in"))
    return out


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------
def work(case):
    back = case["way"] == "backward"
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        size, weights = case["rows"] * case["groups"] * case["width"], (1 if case["shared"] else case["groups"]) * case["width"]
        ex, gate = 2 if case["x_dtype"] == "bf16" else 4, case["gate"] != "none"
        weights *= 4 * (1 + case["bias"])
        if back:
            return {"bytes": size * (2 * ex + e + 2 * e * gate) + 2 * weights, "flops": size * (14 + 10 * gate)}
        return {"bytes": size * (ex + e + e * gate) + weights, "flops": size * (5 + 5 * gate)}
    n, T = case["seqs"], case["tokens"]
    if case["op"] == "conv":
        K, parts = case["taps"], _parts(case)
        C, normed = sum(p[0] for p in parts), sum(p[0] for p in parts if p[1])
        weights = C * 4 * (K + case["bias"])
        states = n * (K - 1) * C * e
        if back:
            return {"bytes": 3 * T * C * e + 2 * weights + states * 3 * case["carried"],
                    "flops": T * (C * (6 * K + 10) + 8 * normed)}
        return {"bytes": 2 * T * C * e + weights + states * (1 + case["carried"]),
                "flops": T * (C * (2 * K + 5) + 3 * normed)}
    D, N, G = case["channels"], case["states"], case["groups"]
    weights, states = 4 * D * (N + 2), 4 * n * D * N
    if back:
        return {"bytes": T * (D * e * (5 + 2 * case["gated"]) + 4 * G * N * e) + 2 * weights + states * 3 * case["carried"],
                "flops": T * D * (22 * N + 20)}
    return {"bytes": T * (D * e * (3 + case["gated"]) + 2 * G * N * e) + weights + states * (1 + case["carried"]),
            "flops": T * D * (7 * N + 12)}


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "selective": _exact_selective}[case["op"]](case, s)


def _exact_norm(case, s):
    """Every gradient by its formula."""
    x, w = s["x"].double(), s["weight"].double()
    gate, slope = 1.0, 0.0
    if s["z"] is not None:
        z = s["z"].double().reshape(x.shape)
        sig = torch.sigmoid(z)
        gate, slope = z * sig, sig * (1 + z * (1 - sig))
    before = case["gate"] == "before"
    u = x * gate if before else x
    m = u.mean(-1, keepdim=True) if case["centred"] else torch.zeros_like(u[..., :1])
    r = ((u - m).pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    n = (u - m) * r
    o = n * w + (s["bias"].double() if s["bias"] is not None else 0.0)
    if case["way"] == "forward":
        return o * gate if case["gate"] == "after" else o
    g = s["dout"].double()
    do = g * gate if case["gate"] == "after" else g
    dn = do * w
    du = r * (dn - n * (dn * n).mean(-1, keepdim=True) - (dn.mean(-1, keepdim=True) if case["centred"] else 0.0))
    over = (0, 1) if case["shared"] else (0,)
    out = {"dx": du * gate if before else du, "dweight": (do * n).sum(over).reshape(w.shape)}
    if s["bias"] is not None:
        out["dbias"] = do.sum(over).reshape(w.shape)
    if s["z"] is not None:
        out["dz"] = ((du * x if before else g * o) * slope).reshape(s["z"].shape)
    return out


def _exact_conv(case, s):
    """Sequence by sequence, tap by tap; every gradient by its formula."""
    K, parts, f64 = case["taps"], _parts(case), torch.float64
    widths = [p[0] for p in parts]
    x, w = torch.cat(s["x"], 1).to(f64), s["weight"].to(f64)
    C, back = x.shape[1], case["way"] == "backward"
    b = torch.zeros(C, dtype=f64, device="cuda") if s["bias"] is None else s["bias"].to(f64)
    if case["way"] == "step":
        pool, slot = s["state"].to(f64), s["slot"].long()
        lens, kept = [1] * case["seqs"], pool[slot]
    else:
        lens = s["lens"]
        kept = torch.zeros(len(lens), K - 1, C, dtype=f64, device="cuda") if s["state"] is None else s["state"].to(f64)
    y, ends = torch.empty_like(x), torch.empty_like(kept)
    dx, dw, db, dkept = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(b), torch.empty_like(kept)
    dy = torch.cat(s["dy"], 1).to(f64) if back else None
    at = 0
    for i, n in enumerate(lens):
        mine = slice(at, at + n)
        at += n
        long = torch.cat([kept[i], x[mine]])
        ends[i] = long[n:]
        u = b.repeat(n, 1)
        for j in range(K):
            u = u + w[:, j] * long[j:j + n]
        sig = torch.sigmoid(u)
        a, g, c = u * sig, torch.empty_like(u), 0
        for width, over, scale in parts:
            cols = slice(c, c + width)
            c += width
            v = a[:, cols]
            if over:
                v = v.unflatten(1, (-1, over))
                r = (v.pow(2).sum(-1, keepdim=True) + NORM_EPS).rsqrt()
                y[mine, cols] = (scale * v * r).flatten(1)
                if back:
                    d = scale * dy[mine, cols].unflatten(1, (-1, over))
                    g[:, cols] = (r * d - v * r.pow(3) * (d * v).sum(-1, keepdim=True)).flatten(1)
            else:
                y[mine, cols] = v
                if back:
                    g[:, cols] = dy[mine, cols]
        if back:
            g = g * sig * (1 + u * (1 - sig))
            d_long = torch.zeros_like(long)
            if s["dstate"] is not None:
                d_long[n:] += s["dstate"][i].to(f64)
            for j in range(K):
                d_long[j:j + n] += w[:, j] * g
                dw[:, j] += (g * long[j:j + n]).sum(0)
            db += g.sum(0)
            dkept[i], dx[mine] = d_long[:K - 1], d_long[K - 1:]
    if not back:
        if case["way"] == "step":
            pool[slot] = ends
            ends = pool
        return {"y": list(y.split(widths, 1)), "state": ends}
    out = {"dx": list(dx.split(widths, 1)), "dweight": dw}
    if s["bias"] is not None:
        out["dbias"] = db
    if s["state"] is not None:
        out["dstate_in"] = dkept
    return out


def _exact_selective(case, s):
    """Token by token, then back."""
    D, N, G, f64 = case["channels"], case["states"], case["groups"], torch.float64
    n, T, back = case["seqs"], case["tokens"], case["way"] == "backward"
    step = case["way"] == "step"
    lens = [1] * n if step else s["lens"]
    first = [sum(lens[:i]) for i in range(n)]
    wide = {k: s[k].to(f64) for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")}
    raw = wide["dt"] + wide["dt_bias"]
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    z = None if s["z"] is None else s["z"].to(f64)
    if s["state"] is None:
        h = torch.zeros(n, D, N, dtype=f64, device="cuda")
    else:
        h = s["state"][s["slot"].long()].to(f64) if step else s["state"].to(f64)

    def spread(m):  # [rows, groups, states] -> [rows, groups, channels of a group, states], as channels
        return m.unsqueeze(2).expand(-1, -1, D // G, -1).reshape(-1, D, N)

    y, kept = torch.zeros(T, D, dtype=f64, device="cuda"), []
    for t in range(max(lens)):
        rows = torch.tensor([i for i in range(n) if t < lens[i]], device="cuda")
        here = torch.tensor([first[i] + t for i in range(n) if t < lens[i]], device="cuda")
        dl, xs, old = delta[here], wide["x"][here], h[rows]
        a = torch.exp(dl.unsqueeze(-1) * wide["A"])
        new = a * old + (dl * xs).unsqueeze(-1) * spread(wide["B"][here])
        h = h.index_copy(0, rows, new) if rows.numel() < n else new
        y[here] = (new * spread(wide["C"][here])).sum(-1) + wide["D"] * xs
        if back:
            kept.append((rows, here, a, old, new))
    if not back:
        if step:
            pool = s["state"].to(f64)
            pool[s["slot"].long()] = h
            h = pool
        return {"y": y if z is None else y * z * torch.sigmoid(z), "state": h}
    dy = s["dy"].to(f64)
    out = {}
    if z is not None:
        sig = torch.sigmoid(z)
        out["dz"] = dy * y * sig * (1 + z * (1 - sig))
        dy = dy * z * sig
    g = torch.zeros(n, D, N, dtype=f64, device="cuda") if s["dstate"] is None else s["dstate"].to(f64)
    for k in ("dx", "ddelta"):
        out[k] = torch.zeros(T, D, dtype=f64, device="cuda")
    for k in ("dB", "dC"):
        out[k] = torch.zeros(T, G, N, dtype=f64, device="cuda")
    out["dA"] = torch.zeros(D, N, dtype=f64, device="cuda")
    while kept:
        rows, here, a, old, new = kept.pop()
        dl, xs, d = delta[here], wide["x"][here], dy[here]
        B = spread(wide["B"][here])
        now = g[rows] + d.unsqueeze(-1) * spread(wide["C"][here])
        out["dC"][here] = (d.unsqueeze(-1) * new).unflatten(1, (G, -1)).sum(2)
        out["dB"][here] = ((dl * xs).unsqueeze(-1) * now).unflatten(1, (G, -1)).sum(2)
        through = (now * B).sum(-1)
        decay = now * a * old  # with respect to delta A
        out["dx"][here] = dl * through
        out["ddelta"][here] = xs * through + (decay * wide["A"]).sum(-1)
        out["dA"] += (decay * dl.unsqueeze(-1)).sum(0)
        g = g.index_copy(0, rows, a * now) if rows.numel() < n else a * now
    out["dx"] += wide["D"] * dy
    out["dD"] = (dy * wide["x"]).sum(0)
    out["ddt"] = out.pop("ddelta") * torch.sigmoid(raw)
    out["ddt_bias"] = out["ddt"].sum(0)
    if s["state"] is not None:
        out["dstate_in"] = g
    return out
