"""Whole-sequence scan (forward, backward) and the serving plans on the GPU, against the
token-by-token recurrence in 64 bits (tests/scan_reference.py).

Tolerances, relative to the norm of each (sequence's) result, with u = 2^-24 the unit
roundoff of fp32:
  * forward: a value's path through a block of 16 tokens has one contraction over d_k, two
    over 16 tokens and a few scalings, each product and sum rounded once: at most d_k + 48
    roundings, of which those of earlier blocks have decayed. (d_k + 48) u.
  * backward: the path meets the forward values (d_k + 48), contractions over d_v and over
    16 tokens, and the reverse recurrence (d_k + 48) again: (2 d_k + d_v + 160) u. bf16
    gradients are rounded once more, by at most 2^-8 of the value.
  * d ln(decay) is a sum of terms that cancel: its error is measured against the sum of the
    terms' sizes (the same for each element), over at most 64 tokens and d_k channels more:
    (2 d_k + d_v + 160 + 64 + d_k) u.
"""
import numpy as np
import pytest

from tests import scan_reference as ref

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def dev_f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


class Batch:
    """A packed batch: host values in 64 bits (exactly what the device holds) and device tensors."""

    def __init__(self, rule, dtype, lens, H, dk, dv, seed=0, spare=0, gates=None, carried=True):
        rng = np.random.default_rng([seed, dk, dv, len(lens)])
        self.rule, self.lens, self.H, self.dk, self.dv = rule, list(lens), H, dk, dv
        self.n, self.T = len(lens), sum(lens) + spare
        T, n = self.T, self.n
        tin = torch.bfloat16 if dtype == "bf16" else torch.float32
        unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
        q, k = unit(rng.standard_normal((T, H, dk))), unit(rng.standard_normal((T, H, dk)))
        v = rng.standard_normal((T, H, dv))
        gshape = (T, H, dk) if rule == "kda" else (T, H)
        gate = rng.uniform(0.85, 0.999, gshape) if gates is None else gates(rng, gshape)
        beta = None if rule == "mamba2" else 1 / (1 + np.exp(-rng.standard_normal((T, H))))
        self.t = {"q": dev_f32(q).to(tin), "k": dev_f32(k).to(tin), "v": dev_f32(v).to(tin),
                  "decay": dev_f32(gate), "beta": None if beta is None else dev_f32(beta),
                  "state_in": dev_f32(0.3 * rng.standard_normal((n, H, dk, dv))) if carried else None,
                  "dy": dev_f32(rng.standard_normal((T, H, dv))),
                  "dstate": dev_f32(rng.standard_normal((n, H, dk, dv))) if carried else None}
        self.tin = tin
        self.d = ssm.Dims.make(rule, dtype, n, H, dk, dv, 4, 4)
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.plan = torch.empty(ssm.scan_sizes(self.d, T)[0], dtype=torch.int32, device="cuda")
        ssm.scan_plan(self.lengths, T, self.plan)

    def host(self, name):
        x = self.t[name]
        return None if x is None else x.double().cpu().numpy()

    def args(self):
        return (self.d, self.T, self.plan) + tuple(self.t[x] for x in ("q", "k", "v", "decay", "beta"))

    def parts(self):
        at = 0
        for i, l in enumerate(self.lens):
            yield i, slice(at, at + l)
            at += l

    def seq(self, i, s):
        h = {x: self.host(x) for x in ("q", "k", "v", "decay", "beta")}
        S = self.host("state_in")
        S = np.zeros((self.H, self.dk, self.dv)) if S is None else S[i]
        return [None if h[x] is None else h[x][s] for x in ("q", "k", "v", "decay", "beta")] + [S]

    def forward(self, **kw):
        y = torch.full((self.T, self.H, self.dv), 7.0, device="cuda")
        state = torch.full((self.n, self.H, self.dk, self.dv), 7.0, device="cuda")
        ssm.scan_forward(*self.args(), state, y, state_in=self.t["state_in"], **kw)
        return y, state

    def backward(self, **kw):
        t = self.t
        o = {"dq": torch.full_like(t["q"], 7), "dk": torch.full_like(t["k"], 7),
             "dv": torch.full_like(t["v"], 7), "dlog": torch.full_like(t["decay"], 7),
             "dbeta": None if t["beta"] is None else torch.full_like(t["beta"], 7),
             "dS0": torch.full((self.n, self.H, self.dk, self.dv), 7.0, device="cuda")}
        ssm.scan_backward(*self.args(), t["dy"], o["dq"], o["dk"], o["dv"], o["dlog"], o["dbeta"],
                          state_in=t["state_in"], dstate=t["dstate"], dstate_in=o["dS0"], **kw)
        return o


def near(got, want, rel, what):
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= rel * norm, f"{what}: {err / max(norm, 1e-300):.3e} > {rel:.3e}"


def check_forward(b, y, state, skip=()):
    tol = (b.dk + 48) * U
    y, state = y.double().cpu().numpy(), state.double().cpu().numpy()
    for i, s in b.parts():
        if i in skip:
            continue
        wy, ws = ref.forward(*b.seq(i, s))
        near(y[s], wy, tol, f"y of sequence {i}")
        near(state[i], ws, tol, f"state of sequence {i}")
    assert (y[sum(b.lens):] == 7).all()  # the tokens behind the last sequence


def check_backward(b, o):
    tol = (2 * b.dk + b.dv + 160) * U
    low = 2.0 ** -8 if b.tin == torch.bfloat16 else 0.0
    o = {x: None if t is None else t.double().cpu().numpy() for x, t in o.items()}
    dy, dS = b.host("dy"), b.host("dstate")
    for i, s in b.parts():
        end = np.zeros((b.H, b.dk, b.dv)) if dS is None else dS[i]
        want, size = ref.backward(*b.seq(i, s), dy[s], end)
        for x in ("dq", "dk", "dv"):
            near(o[x][s], want[x], tol + low, f"{x} of sequence {i}")
        if b.rule != "mamba2":
            near(o["dbeta"][s], want["dbeta"], tol, f"dbeta of sequence {i}")
        near(o["dS0"][i], want["dS0"], tol, f"dS0 of sequence {i}")
        off = np.abs(o["dlog"][s] - want["dlog"])
        assert (off <= (3 * b.dk + b.dv + 224) * U * size).all(), f"dlog of sequence {i}: {(off / size).max():.3e}"
    end = sum(b.lens)
    for x in ("dq", "dk", "dv", "dlog", "dbeta"):
        assert o[x] is None or (o[x][end:] == 7).all(), x


RULES = ("mamba2", "gdn", "kda")
SHAPES = [(16, 16), (16, 128), (32, 64), (64, 32), (128, 16), (128, 128)]
LENGTHS = [[1], [16, 15, 17, 0, 1], [63, 64, 65], [150, 3]]


@pytest.mark.parametrize("n", [1, 3, 41, 4096, 4097, 9000])
@pytest.mark.parametrize("total", [0, 1, 64, 5000, 300000])
def test_scan_plan(n, total):
    rng = np.random.default_rng([n, total])
    lens = rng.integers(-3, max(2, 3 * total // (2 * n)), n)
    if n > 2:
        lens[rng.integers(n)] = total // 3
    if total == 5000:
        lens[0] = 2 ** 31 - 1  # past the end of the arrays
    cap = total // 64 + n
    start = np.minimum(np.concatenate([[0], np.cumsum(np.maximum(lens, 0))]), total)
    chunks = np.concatenate([[0], np.cumsum((np.diff(start) + 63) // 64)])
    seq = np.full(cap, -1)
    for s in range(n):
        seq[chunks[s]:chunks[s + 1]] = s
    buf = torch.full((1 + 2 * (n + 1) + cap + 5,), -9, dtype=torch.int32, device="cuda")
    plan = buf[1:1 + 2 * (n + 1) + cap]  # 4-byte aligned only
    ssm.scan_plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), total, plan)
    np.testing.assert_array_equal(plan.cpu().numpy(), np.concatenate([start, chunks, seq]))
    assert buf[0] == -9 and (buf[-5:] == -9).all()


def test_scan_plan_of_the_longest_arrays():
    total = 2 ** 31 - 1
    lens = torch.tensor([total - 100, total], dtype=torch.int32, device="cuda")
    plan = torch.empty(6 + total // 64 + 2, dtype=torch.int32, device="cuda")
    ssm.scan_plan(lens, total, plan)
    first = (total - 100 + 63) // 64
    assert plan[:6].tolist() == [0, total - 100, total, 0, first, first + 2]
    assert (plan[6:6 + first] == 0).all() and plan[6 + first:].tolist() == [1, 1] + [-1] * (total // 64 - first)
    one = plan[:4 + total // 64 + 1]
    ssm.scan_plan(lens[1:], total, one)
    assert one[:4].tolist() == [0, total, 0, total // 64 + 1] and (one[4:] == 0).all()


@pytest.mark.parametrize("n", [1, 7, 1024, 4096, 4099, 50001])
@pytest.mark.parametrize("W", [1, 2, 7, 8, 15, 16])
def test_window_plan(n, W):
    rng = np.random.default_rng([n, W])
    lens = rng.integers(-2, 4 * W, n)
    lens[rng.integers(n)] = 2 ** 31 - 1
    tau = np.where(lens >= 0, lens % W + 1, 0)
    parity = np.where(lens >= 0, lens // W % 2, 0)
    rows = np.flatnonzero(tau == W)
    d = ssm.Dims.make("gdn", "bf16", n, 1, 128, 128, W, 8)
    src = torch.tensor(np.concatenate([[0], lens]), dtype=torch.int32, device="cuda")[1:]
    out = [torch.full((n + 4,), -9, dtype=torch.int32, device="cuda") for _ in range(3)]
    count = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    ssm.window_plan(d, src, *[x[:n] for x in out], count[:1])
    for x, want in zip(out, (tau, parity, np.concatenate([rows, np.full(n - len(rows), -1)]))):
        np.testing.assert_array_equal(x[:n].cpu().numpy(), want)
        assert (x[n:] == -9).all()
    assert count.tolist() == [len(rows), -9]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule", RULES)
def test_forward(rule, shape, lens):
    for dtype in ("bf16", "f32"):
        b = Batch(rule, dtype, lens, 3, *shape, spare=5)
        check_forward(b, *b.forward())


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule", RULES)
def test_backward(rule, shape, lens):
    for dtype in ("bf16", "f32"):
        b = Batch(rule, dtype, lens, 3, *shape, spare=5)
        check_backward(b, b.backward())


@pytest.mark.parametrize("rule", RULES)
def test_long_and_empty(rule):
    b = Batch(rule, "bf16", [0, 1500, 0], 2, 128, 64, carried=False)
    y, state = b.forward()
    check_forward(b, y, state)
    assert (state[0] == 0).all() and (state[2] == 0).all()
    check_backward(b, b.backward())
    b = Batch(rule, "f32", [0, 0], 2, 32, 32)  # no token at all
    y, state = b.forward()
    assert torch.equal(state, b.t["state_in"])
    assert torch.equal(b.backward()["dS0"], b.t["dstate"])


GATES = {
    "zeros and ones": lambda rng, s: rng.choice([0.0, 1.0, 0.9], s),
    "all zero": lambda rng, s: np.zeros(s),
    "all one": lambda rng, s: np.ones(s),
    "tiny": lambda rng, s: 10.0 ** -rng.uniform(0, 38, s),
}


@pytest.mark.parametrize("gates", GATES)
@pytest.mark.parametrize("rule", RULES)
def test_extreme_gates(rule, gates):
    """Gates of zero forget everything exactly; gates of one keep it; products that underflow are zero."""
    b = Batch(rule, "f32", [70, 33], 2, 32, 32, gates=GATES[gates])
    y, state = b.forward()
    check_forward(b, y, state)
    o = b.backward()
    check_backward(b, o)
    assert all(torch.isfinite(x).all() for x in o.values() if x is not None)


@pytest.mark.parametrize("rule", ["gdn", "kda"])
def test_beta_zero_and_one(rule):
    b = Batch(rule, "f32", [50], 2, 64, 32)
    b.t["beta"][::2] = 0.0
    b.t["beta"][1::4] = 1.0
    check_forward(b, *b.forward())
    check_backward(b, b.backward())


@pytest.mark.parametrize("rule", RULES)
def test_non_finite_stays_in_its_sequence(rule):
    b = Batch(rule, "bf16", [40, 37, 50], 2, 64, 64, spare=30)
    want_y, want_s = b.forward()
    want = b.backward()
    for x in ("q", "k", "v", "decay", "beta", "dy"):
        if b.t[x] is not None:
            b.t[x][50:60] = float("nan")   # of sequence 1
            b.t[x][127:] = float("inf")    # behind the last sequence
    b.t["state_in"][1] = float("nan")
    y, s = b.forward()
    got = b.backward()
    for i in (0, 2):
        assert torch.equal(s[i], want_s[i]) and torch.equal(got["dS0"][i], want["dS0"][i])
    for sl in (slice(0, 40), slice(77, 127)):
        assert torch.equal(y[sl], want_y[sl])
        for x in ("dq", "dk", "dv", "dlog", "dbeta"):
            assert want[x] is None or torch.equal(got[x][sl], want[x][sl]), x
    assert (y[127:] == 7).all()


@pytest.mark.parametrize("rule", RULES)
def test_slots_and_continuing_in_place(rule):
    """A prompt taken in two parts through a slot pool, in place, equals the whole, bit for bit
    where the cut falls between blocks; rows outside the pool are skipped."""
    lens = [96, 40, 64]
    b = Batch(rule, "bf16", lens, 2, 64, 32)
    y, state = b.forward()
    cut = 48
    pool = torch.full((7, 2, 64, 32), 3.0, device="cuda")
    slot = torch.tensor([5, -1, 2], dtype=torch.int32, device="cuda")
    pool[[5, 2]] = b.t["state_in"][[0, 2]]
    starts = [0, 96, 136]
    for lo, hi in ((0, cut), (cut, 96)):
        pick = torch.cat([torch.arange(s + min(lo, l), s + min(hi, l)) for s, l in zip(starts, lens)]).cuda()
        part = torch.tensor([min(hi, l) - min(lo, l) for l in lens], dtype=torch.int32, device="cuda")
        plan = torch.empty(ssm.scan_sizes(b.d, len(pick))[0], dtype=torch.int32, device="cuda")
        ssm.scan_plan(part, len(pick), plan)
        out = torch.full((len(pick), 2, 32), 7.0, device="cuda")
        ssm.scan_forward(b.d, len(pick), plan, *[None if b.t[x] is None else b.t[x][pick] for x in
                         ("q", "k", "v", "decay", "beta")], pool, out, state_in=pool, slot=slot, num_slots=7)
        skipped = (pick >= 96) & (pick < 136)
        assert torch.equal(out[~skipped], y[pick[~skipped]])
        assert (out[skipped] == 7).all()
    assert torch.equal(pool[5], state[0]) and torch.equal(pool[2], state[2])
    assert (pool[[0, 1, 3, 4, 6]] == 3).all()


@pytest.mark.parametrize("rule", RULES)
def test_bits_do_not_depend_on_the_batch_or_the_run(rule):
    b = Batch(rule, "bf16", [77, 130, 20], 3, 128, 128)
    y, s = b.forward()
    o = b.backward()
    y2, s2 = b.forward()
    o2 = b.backward()
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert all(o[x] is None or torch.equal(o[x], o2[x]) for x in o)
    one = Batch(rule, "bf16", [130], 3, 128, 128)
    for x in ("q", "k", "v", "decay", "beta", "dy"):
        one.t[x] = None if b.t[x] is None else b.t[x][77:207].contiguous()
    for x in ("state_in", "dstate"):
        one.t[x] = b.t[x][1:2].contiguous()
    y1, s1 = one.forward()
    o1 = one.backward()
    assert torch.equal(y1, y[77:207]) and torch.equal(s1[0], s[1])
    assert all(o[x] is None or torch.equal(o1[x], o[x][77:207]) for x in o if x != "dS0")
    assert torch.equal(o1["dS0"][0], o["dS0"][1])


@pytest.mark.parametrize("rule", RULES)
def test_gradient_against_differences(rule):
    """A directional derivative of the 64-bit forward against the gradient's product with the
    direction. Differences of step e: error e^2 of the third derivative, here under 1e-7."""
    b = Batch(rule, "f32", [37], 2, 32, 16)
    o = {x: None if t is None else t.double().cpu().numpy() for x, t in b.backward().items()}
    q, k, v, gate, beta, S0 = b.seq(0, slice(0, 37))
    dy, dS = b.host("dy"), b.host("dstate")[0]
    args = [q, k, v, np.log(gate), beta, S0]

    def loss(a):
        y, last = ref.forward(a[0], a[1], a[2], np.exp(a[3]), a[4], a[5])
        return (y * dy).sum() + (last * dS).sum()

    rng = np.random.default_rng(9)
    for i, name in enumerate(("dq", "dk", "dv", "dlog", "dbeta", "dS0")):
        if args[i] is None:
            continue
        g = o[name] if name != "dS0" else o[name][0]
        d = rng.standard_normal(args[i].shape)
        e = 1e-5
        hi, lo = (loss([a if j != i else a + sgn * e * d for j, a in enumerate(args)]) for sgn in (1, -1))
        room = (3 * b.dk + b.dv + 224) * U
        assert abs((hi - lo) / (2 * e) - (g * d).sum()) <= 1e-7 + room * 8 * np.linalg.norm(g) * np.linalg.norm(d), name


def test_other_stream_and_workspace():
    b = Batch("gdn", "bf16", [100, 60], 2, 64, 64)
    y, s = b.forward()
    o = b.backward()
    st = torch.cuda.Stream()
    _, fb, bb = ssm.scan_sizes(b.d, b.T)
    for ws in (None, torch.empty(bb, dtype=torch.uint8, device="cuda")):
        torch.cuda.synchronize()
        y2, s2 = torch.empty_like(y), torch.empty_like(s)
        st.wait_stream(torch.cuda.current_stream())
        ssm.scan_forward(*b.args(), s2, y2, state_in=b.t["state_in"], workspace=ws, stream=st)
        st.synchronize()
        assert torch.equal(y2, y) and torch.equal(s2, s)
        if ws is not None:
            o2 = b.backward(workspace=ws)
            assert torch.equal(o2["dk"], o["dk"]) and torch.equal(o2["dlog"], o["dlog"])
    with pytest.raises(ssm.SSMError, match="workspace"):
        b.forward(workspace=torch.empty(fb - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="elements"):
        ssm.scan_forward(b.d, b.T + 1, *b.args()[2:], s, y)


@pytest.mark.parametrize("rule", RULES)
def test_captured_and_replayed(rule):
    """Plan, forward and backward in one graph: replays with new inputs equal eager calls."""
    b = Batch(rule, "bf16", [100, 61, 5], 2, 64, 64)
    ws = torch.empty(ssm.scan_sizes(b.d, b.T)[2], dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        ssm.scan_plan(b.lengths, b.T, b.plan)
        y, s = b.forward(workspace=ws)
        o = b.backward(workspace=ws)
    for seed in range(3):
        other = Batch(rule, "bf16", [[100, 61, 5], [1, 160, 5], [0, 64, 102]][seed], 2, 64, 64, seed=seed)
        for x in b.t:
            if b.t[x] is not None:
                b.t[x].copy_(other.t[x])
        b.lengths.copy_(other.lengths)
        graph.replay()
        torch.cuda.synchronize()
        wy, ws_ = other.forward()
        wo = other.backward()
        assert torch.equal(y, wy) and torch.equal(s, ws_)
        assert all(o[x] is None or torch.equal(o[x], wo[x]) for x in o)
        torch.randn(1000, device="cuda").sum().item()


def test_a_table_that_is_no_plan_touches_nothing_outside():
    b = Batch("gdn", "f32", [64, 30], 2, 32, 32)
    y, s = b.forward()
    for bad in (-1, 2 ** 31 - 1, 1):
        b.plan.fill_(bad)
        y2 = torch.full_like(y, 7.0)
        s2 = torch.full_like(s, 7.0)
        ssm.scan_forward(*b.args(), s2, y2, state_in=b.t["state_in"])
        torch.cuda.synchronize()
        assert (y2 == 7).all()


@pytest.mark.parametrize("rule", RULES)
def test_prefill_then_serving_steps(rule):
    """The operators together: prompts into a slot pool, a refresh, and serving steps whose index
    arrays the device builds, against the recurrence over the whole token streams. The basis
    spans all of d_k = 16, so the sketch read is exact; its products add d_k roundings per
    factor: 4 (d_k + 48) u for the decode."""
    n, H, dk, dv, W, steps = 5, 2, 16, 32, 4, 11
    prompts, pool = [33, 1, 64, 0, 20], 8
    b = Batch(rule, "f32", prompts, H, dk, dv, carried=False)
    toks = [Batch(rule, "f32", [1] * n, H, dk, dv, seed=100 + t) for t in range(steps)]
    slot = torch.tensor([6, 0, 3, 7, 2], dtype=torch.int32, device="cuda")
    d = ssm.Dims.make(rule, "f32", n, H, dk, dv, W, dk)
    state = torch.zeros(pool, H, dk, dv, device="cuda")
    y0 = torch.empty(b.T, H, dv, device="cuda")
    ssm.scan_forward(d, *b.args()[1:], state, y0, slot=slot, num_slots=pool)
    rng = np.random.default_rng(1)
    basis = dev_f32(np.stack([np.linalg.qr(rng.standard_normal((dk, dk)))[0].T for _ in range(H)]))
    sk = [torch.zeros(pool, H, dk, dv, device="cuda") for _ in range(2)]
    kb, vb = torch.zeros(pool, H, W, dk, device="cuda"), torch.zeros(pool, H, W, dv, device="cuda")
    db = torch.zeros((pool, H, W, dk) if rule == "kda" else (pool, H, W), device="cuda")
    bb = None if rule == "mamba2" else torch.zeros(pool, H, W, device="cuda")
    ssm.window_update_refresh_varlen(d, pool, slot, torch.zeros(n, dtype=torch.int32, device="cuda"),
                                     state, sk[0], basis, kb, vb, db, bb)
    done = torch.zeros(n, dtype=torch.int32, device="cuda")
    tau, parity, rows = torch.empty(3, n, dtype=torch.int32, device="cuda")
    count = torch.empty(1, dtype=torch.int32, device="cuda")
    ys = []
    for t in toks:
        ssm.window_plan(d, done, tau, parity, rows, count)
        y = torch.empty(n, H, dv, device="cuda")
        ssm.decode_step_varlen(d, pool, slot, tau, parity, n, rows, state, sk[0], sk[1], basis,
                               t.t["q"], t.t["k"], t.t["v"], t.t["decay"], t.t["beta"], kb, vb, db,
                               bb, y)
        ys.append(y.double().cpu().numpy())
        done += 1
    for i, s in b.parts():
        *x, S = b.seq(i, s)
        x = [None if a is None else np.concatenate([a] + [t.host(m)[i:i + 1] for t in toks])
             for a, m in zip(x, ("q", "k", "v", "decay", "beta"))]
        want, _ = ref.forward(*x, S)
        if prompts[i]:
            near(y0.double().cpu().numpy()[s], want[:prompts[i]], (dk + 48) * U, f"prompt {i}")
        near(np.stack([y[i] for y in ys]), want[prompts[i]:], 4 * (dk + 48) * U, f"decode of row {i}")


@pytest.mark.parametrize("rule", RULES)
def test_decoders_prefill(rule):
    """WindowedDecoder and RecurrentDecoder from a prompt on: prefill (twice, the second time with
    tokens in the window), then steps, against the recurrence over the whole streams. The window
    sums its tokens apart from the state: 4 (d_k + 48) u as for the serving steps."""
    from sketched_recurrent_state_amd.decoder import RecurrentDecoder, WindowedDecoder
    n, H, dk, dv, W = 2, 3, 16, 32, 4
    first = Batch(rule, "f32", [21, 40], H, dk, dv)
    second = Batch(rule, "f32", [0, 17], H, dk, dv, seed=5)
    toks = [Batch(rule, "f32", [1] * n, H, dk, dv, seed=10 + t) for t in range(9)]
    d = ssm.Dims.make(rule, "f32", n, H, dk, dv, W, dk)
    rng = np.random.default_rng(2)
    basis = dev_f32(np.stack([np.linalg.qr(rng.standard_normal((dk, dk)))[0].T for _ in range(H)]))
    names = ("q", "k", "v", "decay", "beta")
    for dec in (WindowedDecoder(d, first.t["state_in"].clone(), basis),
                WindowedDecoder(d, first.t["state_in"].clone(), read="full"),
                RecurrentDecoder(d, first.t["state_in"].clone())):
        one = lambda t: dec.step(*[t.t[x] for x in names]).double().cpu().numpy()
        ya = dec.prefill(first.lens, *[first.t[x] for x in names]).double().cpu().numpy()
        got = [one(t) for t in toks[:3]]
        yb = dec.prefill(torch.tensor(second.lens), *[second.t[x] for x in names]).double().cpu().numpy()
        got += [one(t) for t in toks[3:]]
        at = [s for _, s in first.parts()], [s for _, s in second.parts()]
        for i in range(n):
            *a, S = first.seq(i, at[0][i])
            b = second.seq(i, at[1][i])
            x = [None if u is None else np.concatenate(
                [u] + [t.host(m)[i:i + 1] for t in toks[:3]] + [w] + [t.host(m)[i:i + 1] for t in toks[3:]])
                for u, w, m in zip(a, b, names)]
            want, _ = ref.forward(*x, S)
            p = first.lens[i]
            e = p + 3 + second.lens[i]
            near(ya[at[0][i]], want[:p], (dk + 48) * U, "first prompt")
            if second.lens[i]:
                near(yb[at[1][i]], want[p + 3:e], 4 * (dk + 48) * U, "second prompt")
            near(np.stack([g[i] for g in got]), np.concatenate([want[p:p + 3], want[e:]]),
                 4 * (dk + 48) * U, "steps")


SIZES = [(1, 2, 128, 128), (1, 40, 128, 128), (1, 80, 128, 64), (3, 150, 64, 128), (2, 400, 32, 16)]


@pytest.mark.parametrize("n,H,dk,dv", SIZES, ids=str)
@pytest.mark.parametrize("rule", RULES)
def test_every_shape_of_the_passes(rule, n, H, dk, dv):
    """Few units (rows divided over 4 or 2 waves) and many (a wave a column block), on a sample of
    heads, with the same bits from run to run."""
    for dtype in ("bf16", "f32"):
        b = Batch(rule, dtype, [70 + 13 * i for i in range(n)], H, dk, dv, spare=2)
        y, state = b.forward()
        o = b.backward()
        for _ in range(3):
            torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(255)  # NaN in new workspaces
            y2, state2 = b.forward()
            o2 = b.backward()
            assert torch.equal(y, y2) and torch.equal(state, state2)
            assert all(o[x] is None or torch.equal(o[x], o2[x]) for x in o)
        heads = [0, H // 2, H - 1]
        few = Batch.__new__(Batch)
        few.__dict__.update(b.__dict__, H=len(heads))
        pick = lambda x, dim: None if x is None else x.index_select(dim, torch.tensor(heads, device="cuda"))
        few.t = {x: pick(t, 1) for x, t in b.t.items()}
        check_forward(few, pick(y, 1), pick(state, 1))
        check_backward(few, {x: pick(t, 1) for x, t in o.items()})


def test_other_stream_beside_unfinished_work():
    """A call on a stream of its own, without a workspace, while the current stream still writes
    to memory that has been freed there."""
    b = Batch("gdn", "bf16", [100, 60], 2, 64, 64)
    y, s = b.forward()
    o = b.backward()
    st = torch.cuda.Stream()
    _, fb, bb = ssm.scan_sizes(b.d, b.T)
    y2, s2 = torch.empty_like(y), torch.empty_like(s)
    o2 = {x: None if t is None else torch.empty_like(t) for x, t in o.items()}
    t = b.t
    torch.cuda.synchronize()
    for stream in (st, st.cuda_stream):
        for size in (fb, bb):
            busy = torch.empty(size, dtype=torch.uint8, device="cuda")
            for _ in range(300):
                busy.fill_(255)
            del busy
            if size == fb:
                ssm.scan_forward(*b.args(), s2, y2, state_in=t["state_in"], stream=stream)
            else:
                ssm.scan_backward(*b.args(), t["dy"], o2["dq"], o2["dk"], o2["dv"], o2["dlog"], o2["dbeta"],
                                  state_in=t["state_in"], dstate=t["dstate"], dstate_in=o2["dS0"], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(s2, s)
        assert all(torch.equal(o2[x], o[x]) for x in o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule", RULES)
def test_gate_gradient_is_zero_where_the_gate_is(rule, dtype):
    """decay * dL/d(decay) at decay = 0 is 0, not what rounding leaves of the sums it comes from."""
    for lens, dk, dv in (([70, 0, 33], 64, 32), ([1, 130], 16, 64), ([65], 128, 128)):
        b = Batch(rule, dtype, lens, 3, dk, dv, gates=lambda rng, s: rng.choice([0.0, -0.0, 0.7, 1.0], s))
        o = b.backward()
        check_backward(b, o)
        assert (o["dlog"][b.t["decay"] == 0] == 0).all()
        assert (o["dlog"][b.t["decay"] != 0] != 0).any()


def test_prefill_with_lengths_on_the_device():
    """Lengths that are not read back: rows behind their sum are zero, and a prompt that does not
    fit is cut where the arrays end."""
    from sketched_recurrent_state_amd.decoder import RecurrentDecoder
    b = Batch("gdn", "f32", [21, 40], 2, 16, 32, spare=7)
    names = ("q", "k", "v", "decay", "beta")
    want, state = b.forward()
    for dtype in (torch.int32, torch.int64):
        torch.full((b.T, b.H, b.dv), float("nan"), device="cuda")  # what new memory may hold
        dec = RecurrentDecoder(b.d, b.t["state_in"].clone())
        y = dec.prefill(b.lengths.to(dtype), *[b.t[x] for x in names])
        assert torch.equal(y[:61], want[:61]) and (y[61:] == 0).all()
        assert torch.equal(dec.state, state)
    cut = RecurrentDecoder(b.d, b.t["state_in"].clone())
    y = cut.prefill(torch.tensor([21, 100], dtype=torch.int32, device="cuda"), *[b.t[x] for x in names])
    whole = RecurrentDecoder(b.d, b.t["state_in"].clone())
    assert torch.equal(y, whole.prefill([21, 47], *[b.t[x] for x in names]))
    assert torch.equal(cut.state, whole.state)


def test_prefill_with_wide_lengths_on_the_device():
    """64-bit lengths beyond 32 bits are cut where the arrays end, as any other; fractions are refused."""
    from sketched_recurrent_state_amd.decoder import RecurrentDecoder
    b = Batch("mamba2", "f32", [5, 30], 2, 16, 16)
    tokens = [b.t[x] for x in ("q", "k", "v", "decay", "beta")]
    want, state = b.forward()
    for lens in ([5, 2 ** 32 + 1], [5, 2 ** 31], [5, 30]):
        dec = RecurrentDecoder(b.d, b.t["state_in"].clone())
        assert torch.equal(dec.prefill(torch.tensor(lens, device="cuda"), *tokens), want)
        assert torch.equal(dec.state, state)
    for lens in (torch.tensor([5.0, 30.0]), torch.tensor([5, 30, 0])):
        with pytest.raises(ValueError, match="lengths"):
            dec.prefill(lens.cuda(), *tokens)


class Banded:
    """Tensors with guard bands before and behind them."""

    def __init__(self):
        self.whole = []

    def __call__(self, like_or_shape, dtype=torch.float32, fill=7):
        shape = getattr(like_or_shape, "shape", like_or_shape)
        dtype = getattr(like_or_shape, "dtype", dtype)
        n = int(np.prod(shape))
        buf = torch.full((n + 8192,), fill, dtype=dtype, device="cuda")
        self.whole.append((buf, n, fill))
        return buf[4096:4096 + n].view(shape)

    def intact(self):
        return all((b[:4096] == f).all() and (b[4096 + n:] == f).all() for b, n, f in self.whole)


# changes to the plan of lengths 100, 70, 30 (starts 0 100 170 200, chunks 0 2 4 5, table 0 0 1 1 2 -1): index, value,
# and the sequences that the change leaves as they were; tests/test_scan_table_cpu.py shows each of them accepted or
# skipped within the arrays
WRONG_PLANS = {
    "a sequence that ends past the arrays": (3, 201, [0, 1]),
    "far past the arrays": (3, 2 ** 31 - 1, [0, 1]),
    "starts in descending order": (1, 180, []),
    "a start below zero": (0, -1, [1, 2]),
    "an end below zero": (1, -5, [2]),
    "chunks past the table": (4 + 1, 5, [0, 2]),
    "chunks below zero": (4 + 2, -1, [0, 1]),
    "a chunk of a sequence that starts later": (8 + 3, 2, [0, 2]),
    "a chunk of a sequence that has ended": (8 + 4, 0, [0, 1]),
    "a chunk of no sequence": (8 + 1, 3, [1, 2]),
    "a chunk of a sequence far off": (8 + 1, 2 ** 31 - 1, [1, 2]),
}


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("name", WRONG_PLANS)
def test_wrong_plans_stay_in_their_arrays(rule, name):
    index, value, kept = WRONG_PLANS[name]
    b = Batch(rule, "bf16", [100, 70, 30], 2, 64, 32)
    want_y, want_s = b.forward()
    want = b.backward()
    b.plan[index] = value
    _, fb, bb = ssm.scan_sizes(b.d, b.T)
    t, new = b.t, Banded()
    y, s = new(want_y), new(want_s)
    ssm.scan_forward(*b.args(), s, y, state_in=t["state_in"], workspace=new((fb,), torch.uint8))
    o = {x: None if w is None else new(w) for x, w in want.items()}
    ssm.scan_backward(*b.args(), t["dy"], o["dq"], o["dk"], o["dv"], o["dlog"], o["dbeta"], state_in=t["state_in"],
                      dstate=t["dstate"], dstate_in=o["dS0"], workspace=new((bb,), torch.uint8))
    torch.cuda.synchronize()
    assert new.intact()
    for i, sl in b.parts():
        if i in kept:
            assert torch.equal(y[sl], want_y[sl]) and torch.equal(s[i], want_s[i])
            assert torch.equal(o["dS0"][i], want["dS0"][i])
            assert all(o[x] is None or torch.equal(o[x][sl], want[x][sl]) for x in o if x != "dS0")


@pytest.mark.parametrize("rule", RULES)
def test_captured_serving_loop(rule):
    """A serving loop in one graph: positions planned on the device, the step, and the lengths'
    increment. Replays equal a loop that the host plans with exact counts, bit for bit."""
    n, H, dk, dv, W, pool, steps = 6, 3, 64, 64, 4, 9, 13
    d = ssm.Dims.make(rule, "bf16", n, H, dk, dv, W, 8)
    slot = torch.tensor([8, 0, 3, 7, 2, 5], dtype=torch.int32, device="cuda")
    start = [0, 3, -1, 2, 7, 3]  # tokens decoded so far; row 2 is padding
    toks = [Batch(rule, "bf16", [1] * n, H, dk, dv, seed=t) for t in range(steps)]
    names = ("q", "k", "v", "decay", "beta")
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    basis = torch.linalg.qr(rand(H, dk, 8)).Q.transpose(1, 2).contiguous()
    t0 = toks[0].t
    first = {"state": rand(pool, H, dk, dv), "sk0": rand(pool, H, 8, dv), "sk1": rand(pool, H, 8, dv),
             "k": rand(pool, H, W, dk).bfloat16(), "v": rand(pool, H, W, dv).bfloat16(),
             "decay": torch.rand(pool, H, W, *t0["decay"].shape[2:], device="cuda", generator=gen),
             "beta": None if rule == "mamba2" else torch.rand(pool, H, W, device="cuda", generator=gen)}
    copy = lambda x: {k: None if v is None else v.clone() for k, v in x.items()}

    def step(m, cur, tau, parity, n_update, rows, y):
        ssm.decode_step_varlen(d, pool, slot, tau, parity, n_update, rows, m["state"], m["sk0"], m["sk1"],
                               basis, *[cur[x] for x in names], m["k"], m["v"], m["decay"], m["beta"], y)

    host, want = copy(first), []
    for i, t in enumerate(toks):
        done = [s + i if s >= 0 else -1 for s in start]
        tau = [x % W + 1 if x >= 0 else 0 for x in done]
        rows = [r for r in range(n) if tau[r] == W]
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        y = torch.full((n, H, dv), 7.0, device="cuda")
        step(host, t.t, ints(tau), ints([x // W % 2 if x >= 0 else 0 for x in done]), len(rows),
             ints(rows) if rows else None, y)
        want.append(y)

    m, cur = copy(first), copy({x: t0[x] for x in names})
    lengths = torch.tensor(start, dtype=torch.int32, device="cuda")
    tau, parity, rows = torch.zeros(3, n, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((n, H, dv), 7.0, device="cuda")
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        ssm.window_plan(d, lengths, tau, parity, rows, count)
        step(m, cur, tau, parity, n, rows, y)
        lengths += (lengths >= 0).int()
    for t, w in zip(toks, want):
        for x in names:
            if cur[x] is not None:
                cur[x].copy_(t.t[x])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)
        assert (y[2] == 7).all()
        torch.randn(1000, device="cuda").sum().item()
    for x in m:
        assert m[x] is None or torch.equal(m[x], host[x]), x


def test_two_graphs_and_eager_calls_without_workspaces():
    """Two graphs, each with workspaces that PyTorch gave its calls, replayed in turn beside eager calls."""
    batches = [Batch("gdn", "bf16", [100, 61], 2, 64, 64), Batch("kda", "f32", [33, 90, 7], 3, 32, 64)]
    graphs = []
    for b in batches:
        b.want = b.forward(), b.backward()
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            got = b.forward(), b.backward()
        graphs.append((graph, got))
    for _ in range(3):
        for b, (graph, got) in zip(batches, graphs):
            for t in (*got[0], *got[1].values()):
                t.zero_()
            graph.replay()
            eager = b.forward(), b.backward()
            torch.randn(1 << 20, device="cuda").sum().item()
            for y, o in (got, eager):
                assert all(torch.equal(x, w) for x, w in zip(y, b.want[0]))
                assert all(torch.equal(o[x], b.want[1][x]) for x in o)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own stream's."""
    a, b = Batch("gdn", "bf16", [700], 4, 128, 128), Batch("gdn", "bf16", [650, 3], 4, 128, 128, seed=1)
    want = [(x.forward(), x.backward()) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                got.append((x.forward(), x.backward()))
        torch.cuda.synchronize()
        for (y, o), (wy, wo) in zip(got, want):
            assert torch.equal(y[0], wy[0]) and torch.equal(y[1], wy[1])
            assert all(torch.equal(o[x], wo[x]) for x in o)


@pytest.mark.parametrize("read", ["sketch", "full"])
def test_captured_prefill(read):
    """A decoder's prefill with lengths on the device, captured: replays with other lengths and states."""
    from sketched_recurrent_state_amd.decoder import WindowedDecoder
    names = ("q", "k", "v", "decay", "beta")
    b = Batch("gdn", "bf16", [40, 20, 4], 2, 64, 32)
    d = ssm.Dims.make("gdn", "bf16", 3, 2, 64, 32, 4, 8)
    basis = torch.linalg.qr(torch.randn(2, 64, 8, device="cuda")).Q.transpose(1, 2).contiguous()
    make = lambda: WindowedDecoder(d, b.t["state_in"].clone(), basis, read=read)
    dec = make()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        y = dec.prefill(b.lengths, *[b.t[x] for x in names])
    for lens in ([40, 20, 4], [1, 63, 0], [0, 0, 5], [64, 64, 64]):
        b.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        dec.state.copy_(b.t["state_in"])
        graph.replay()
        torch.cuda.synchronize()
        other = make()
        want = other.prefill(b.lengths.clone(), *[b.t[x] for x in names])
        assert torch.equal(y, want) and torch.equal(dec.state, other.state)
        assert read == "full" or torch.equal(dec.sketch, other.sketch)
        assert (y[min(sum(lens), 64):] == 0).all()
        torch.randn(1000, device="cuda").sum().item()
