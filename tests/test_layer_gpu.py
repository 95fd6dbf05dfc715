"""The short convolution, the selective recurrence and the output norm on the GPU against their definitions in
64 bits (tests/layer_reference.py), element by element.

Tolerances: the reference's first-order bound of each element in units of 2^-24, times 2 for what
the first order leaves out, and for results in bf16 half a step, 2^-8 of the value.
"""
import numpy as np
import pytest

from tests import layer_reference as ref

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TIN = {"bf16": torch.bfloat16, "f32": torch.float32}
FILL = 7.0  # what outputs hold before a call


def dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype)


def host(x):
    return None if x is None else x.double().cpu().numpy()


def near(got, want, bound, what, low=True):
    """low: whether the result was rounded to the type that got has."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 and low else 0.0
    g = host(got).reshape(want.shape)
    off = np.abs(g - want)
    tol = 2 * U * bound * (1 + half) + half * np.abs(want) + 1e-37
    assert np.isfinite(g).all(), what
    if not (off <= tol).all():
        i = (off - tol).argmax()
        pytest.fail(f"{what}: {off.flat[i]:.3e} > {tol.flat[i]:.3e} at {want.flat[i]:.3e}")


def columns(x, pad, dtype):
    """x [rows][...] as a column range of a wider tensor."""
    flat = x.flatten(1)
    wide = torch.full((flat.shape[0], flat.shape[1] + 16 * pad), FILL, device="cuda", dtype=dtype)
    wide[:, 8 * pad:8 * pad + flat.shape[1]] = flat.to(dtype)
    return wide[:, 8 * pad:8 * pad + flat.shape[1]]


def plan_of(lens, total):
    n = len(lens)
    plan = torch.empty(2 * (n + 1) + total // 64 + n, dtype=torch.int32, device="cuda")
    ssm.scan_plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), total, plan)
    return plan


def spans(lens):
    at = 0
    for i, n in enumerate(lens):
        yield i, slice(at, at + n)
        at += n


# ---------------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------------
class Conv:
    def __init__(self, dtype, lens, channels, norm=None, scale=None, taps=4, silu=True, bias=True, carried=True,
                 pad=1, spare=0, seed=0, eps=1e-6):
        rng = np.random.default_rng([seed, taps, len(lens), *channels])
        self.lens, self.T, self.n, self.K = list(lens), sum(lens) + spare, len(lens), taps
        self.widths, self.tin, self.eps, self.silu = list(channels), TIN[dtype], eps, silu
        norm = [0] * len(channels) if norm is None else norm
        scale = [1.0] * len(channels) if scale is None else scale
        self.d = ssm.ConvDims.make(dtype, self.n, taps, channels, norm=norm, scale=scale,
                                   activation="silu" if silu else "none", eps=eps)
        self.parts = list(zip(channels, norm, [float(np.float32(s)) for s in scale]))
        C = self.C = sum(channels)
        T = self.T
        make = lambda *s: rng.standard_normal(s)
        x = dev(make(T, C), self.tin)
        if pad:
            wide = columns(x, pad, self.tin)
            self.x = list(wide.split(channels, 1))
        else:
            self.x = [p.contiguous() for p in x.split(channels, 1)]
        self.w, self.b = dev(make(C, taps) / 2), dev(make(C)) if bias else None
        self.kept = dev(make(self.n, taps - 1, C), self.tin) if carried else None
        self.dy = [dev(make(T, c), self.tin) for c in channels]
        self.dend = dev(make(self.n, taps - 1, C), self.tin) if carried else None
        self.plan = plan_of(self.lens, T)

    def out(self):
        return [torch.full((self.T, c), FILL, device="cuda", dtype=self.tin) for c in self.widths]

    def forward(self, in_place=False, **kw):
        y = self.out()
        state = (self.kept.clone() if in_place
                 else torch.full((self.n, self.K - 1, self.C), FILL, device="cuda", dtype=self.tin))
        ssm.conv_forward(self.d, self.T, self.plan, self.x, self.w, self.b, y, state,
                         state_in=state if in_place else self.kept, **kw)
        return y, state

    def backward(self, **kw):
        o = {"dx": self.out(), "dw": torch.full_like(self.w, FILL),
             "db": torch.full((self.C,), FILL, device="cuda"),
             "dkept": torch.full((self.n, self.K - 1, self.C), FILL, device="cuda", dtype=self.tin)}
        ssm.conv_backward(self.d, self.T, self.plan, self.x, self.w, self.b, self.dy, o["dx"], o["dw"],
                          o["db"], state_in=self.kept, dstate=self.dend, dstate_in=o["dkept"], **kw)
        return o

    def seq(self, i, s):
        kept = np.zeros((self.K - 1, self.C)) if self.kept is None else host(self.kept)[i]
        x = np.concatenate([host(x)[s] for x in self.x], 1)
        return (x, host(self.w), host(self.b), kept, self.parts, self.silu, float(np.float32(self.eps)))

    def check_forward(self, y, state, skip=()):
        end = sum(self.lens)
        for i, s in spans(self.lens):
            if i in skip:
                continue
            want, bound = ref.conv(*self.seq(i, s))
            c = 0
            for p, width in enumerate(self.widths):
                near(y[p][s], want["y"][:, c:c + width], bound["y"][:, c:c + width], f"y[{p}] of sequence {i}")
                c += width
            np.testing.assert_array_equal(host(state[i]), want["end"])
        for v in y:
            assert (v[end:] == FILL).all()

    def check_backward(self, o):
        dw = db = edw = edb = 0
        for i, s in spans(self.lens):
            dy = np.concatenate([host(v)[s] for v in self.dy], 1)
            want, bound = ref.conv(*self.seq(i, s), dy=dy, dend=None if self.dend is None else host(self.dend)[i])
            c = 0
            for p, width in enumerate(self.widths):
                near(o["dx"][p][s], want["dx"][:, c:c + width], bound["dx"][:, c:c + width], f"dx[{p}] of sequence {i}")
                c += width
            near(o["dkept"][i], want["dkept"], bound["dkept"], f"dkept of sequence {i}")
            dw, db = dw + want["dw"], db + want["db"]
            # the sums go on over all sequences: as many roundings again
            edw, edb = edw + bound["dw"] + self.T * np.abs(want["dw"]), edb + bound["db"] + self.T * np.abs(want["db"])
        near(o["dw"], dw, edw, "dw")
        near(o["db"], db, edb, "db")
        for v in o["dx"]:
            assert (v[sum(self.lens):] == FILL).all()


CHANNELS = [([8], None), ([24, 520], None), ([64, 64, 128], [16, 32, 0]), ([1024, 128, 384], [128, 64, 128]),
            ([16, 8, 128, 16], [16, 0, 128, 0])]
LENGTHS = [[1], [2, 0, 3, 1], [16, 15, 17, 0, 1], [63, 64, 65], [150, 3, 0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("channels", range(len(CHANNELS)))
def test_conv(channels, lens, dtype):
    widths, norm = CHANNELS[channels]
    for taps in (2, 3, 4):
        c = Conv(dtype, lens, widths, norm, [0.25, 1.0, 3.0, 1.0][:len(widths)], taps=taps, spare=5)
        c.check_forward(*c.forward())
        c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_without_bias_activation_or_state(dtype):
    c = Conv(dtype, [70, 0, 2, 40], [64, 40], silu=False, bias=False, carried=False, pad=0)
    y, state = c.forward()
    c.check_forward(y, state)
    o = c.backward()
    c.check_backward(o)
    z = c.out()  # outputs alone
    ssm.conv_forward(c.d, c.T, c.plan, c.x, c.w, None, z)
    assert all(torch.equal(a, b) for a, b in zip(y, z))
    dx, dw = c.out(), torch.empty_like(c.w)
    ssm.conv_backward(c.d, c.T, c.plan, c.x, c.w, None, c.dy, dx, dw)
    assert torch.equal(dw, o["dw"]) and all(torch.equal(a, b) for a, b in zip(dx, o["dx"]))


def test_conv_empty_batches():
    c = Conv("bf16", [0, 0, 0], [64, 16])
    y, state = c.forward()
    assert torch.equal(state, c.kept)
    o = c.backward()
    assert torch.equal(o["dkept"], c.dend) and (o["dw"] == 0).all() and (o["db"] == 0).all()
    d = ssm.ConvDims.make("bf16", 0, 4, [64])
    dw, db = torch.full((64, 4), FILL, device="cuda"), torch.full((64,), FILL, device="cuda")
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    plan = torch.zeros(2, dtype=torch.int32, device="cuda")
    ssm.conv_forward(d, 0, plan, none, dw, None, none)
    ssm.conv_backward(d, 0, plan, none, torch.ones_like(dw), None, none, none, dw, db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("channels", range(len(CHANNELS)))
def test_conv_steps_are_the_prompt(channels, dtype):
    """A prompt token by token gives the prompt's outputs and states, bit for bit, with rows anywhere in a pool."""
    widths, norm = CHANNELS[channels]
    c = Conv(dtype, [9, 9, 9], widths, norm, spare=2, pad=2)
    y, state = c.forward()
    pool = torch.full((7, c.K - 1, c.C), FILL, device="cuda", dtype=c.tin)
    slot = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slot.long()] = c.kept
    for t in range(9):
        at = torch.tensor([t, 9 + t, 18 + t], device="cuda")
        out = [torch.empty(3, w, device="cuda", dtype=c.tin) for w in widths]
        ssm.conv_step(c.d, [v[at] for v in c.x], c.w, c.b, pool, out, slot=slot, num_slots=7)
        for a, b in zip(out, y):
            assert torch.equal(a, b[at])
    assert torch.equal(pool[slot.long()], state)
    assert (pool[[1, 2, 4, 6]] == FILL).all()


def test_conv_slots_and_in_place():
    c = Conv("bf16", [30, 0, 2, 70, 5], [128, 64], [64, 0])
    y, state = c.forward()
    y2, state2 = c.forward(in_place=True)
    assert torch.equal(state, state2) and all(torch.equal(a, b) for a, b in zip(y, y2))
    # a pool; a sequence without a slot is skipped
    slot = torch.tensor([6, 2, -1, 0, 8], dtype=torch.int32, device="cuda")
    pool = torch.full((8, c.K - 1, c.C), FILL, device="cuda", dtype=c.tin)
    for i in (0, 1, 3):
        pool[slot[i]] = c.kept[i]
    out = c.out()
    ssm.conv_forward(c.d, c.T, c.plan, c.x, c.w, c.b, out, pool, state_in=pool, slot=slot, num_slots=8)
    for i, s in spans(c.lens):
        for a, b in zip(out, y):
            assert torch.equal(a[s], b[s]) if i in (0, 1, 3) else (a[s] == FILL).all()
        if i in (0, 1, 3):
            assert torch.equal(pool[slot[i]], state[i])
    assert (pool[[1, 3, 4, 5, 7]] == FILL).all()
    # prompts in two parts are the prompt
    cut = [20, 0, 1, 64, 3]
    one, two = c.out(), c.out()
    first = torch.cat([torch.arange(s.start, s.start + k) for (_, s), k in zip(spans(c.lens), cut)]).cuda()
    rest = torch.cat([torch.arange(s.start + k, s.stop) for (_, s), k in zip(spans(c.lens), cut)]).cuda()
    kept = c.kept.clone()
    for at, lens in ((first, cut), (rest, [a - b for a, b in zip(c.lens, cut)])):
        part = [torch.empty(len(at), w, device="cuda", dtype=c.tin) for w in c.widths]
        ssm.conv_forward(c.d, len(at), plan_of(lens, len(at)), [v[at] for v in c.x], c.w, c.b, part, kept,
                         state_in=kept)
        for a, b in zip(part, y):
            assert torch.equal(a, b[at])
    assert torch.equal(kept, state)


def test_conv_non_finite_stays():
    """A NaN reaches its own channel (or norm's run), from its token on for the taps, and no other sequence."""
    c = Conv("f32", [40, 40], [64, 64], [32, 0], pad=0)
    y, _ = c.forward()
    c.x[0][10, 3] = float("nan")
    c.x[1][20, 5] = float("inf")
    z, state = c.forward()
    a, b = torch.zeros_like(y[0], dtype=torch.bool), torch.zeros_like(y[1], dtype=torch.bool)
    a[10:14, 0:32], b[20:24, 5] = True, True
    assert torch.isnan(z[0][a]).all() and not torch.isfinite(z[1][b]).all()
    assert torch.equal(z[0][~a], y[0][~a]) and torch.equal(z[1][~b], y[1][~b])
    o = c.backward()
    bad = torch.isnan(o["dx"][0]) | torch.isinf(o["dx"][0])
    assert not bad[:7].any() and not bad[14:].any() and not bad[:, 32:].any() and bad[7:14, 3].any()
    assert torch.isfinite(o["dw"][32:64]).all() and torch.isfinite(o["dw"][70:]).all()


def test_conv_large_values():
    """Where e^-u overflows and where it vanishes: silu is 0 and u."""
    c = Conv("f32", [3], [16], bias=True, carried=False, pad=0)
    c.w.zero_()
    c.w[:, -1] = 1
    c.b.zero_()
    c.x[0].copy_(torch.tensor([-200.0, 200.0, 0.0], device="cuda")[:, None].expand(3, 16))
    y, _ = c.forward()
    assert (y[0][0].abs() <= 1e-30).all() and (y[0][1] == 200).all() and (y[0][2] == 0).all()
    o = c.backward()
    assert all(torch.isfinite(v).all() for v in (o["dx"][0], o["dw"], o["db"]))


# ---------------------------------------------------------------------------------
# selective recurrence
# ---------------------------------------------------------------------------------
class Selective:
    def __init__(self, dtype, lens, ch, N, G=1, gated=True, skip=True, bias=True, soft=True, carried=True, pad=1,
                 spare=0, seed=0):
        rng = np.random.default_rng([seed, ch, N, G, len(lens)])
        self.lens, self.T, self.n = list(lens), sum(lens) + spare, len(lens)
        self.ch, self.N, self.G, self.soft = ch, N, G, soft
        self.tin = TIN[dtype]
        T = self.T
        make = lambda *s: rng.standard_normal(s)
        wide = lambda v: columns(dev(v), pad, self.tin) if pad else dev(v, self.tin)
        self.x, dt = wide(make(T, ch)), make(T, ch)
        self.dt = wide(dt if soft else np.abs(dt) / 10)
        self.B, self.C = wide(make(T, G * N)), wide(make(T, G * N))
        self.z = wide(make(T, ch)) if gated else None
        self.A = dev(-np.exp(rng.uniform(-2, np.log(N), (ch, N))))
        self.D = dev(make(ch)) if skip else None
        self.bias = dev(rng.uniform(-5, 0, ch) if soft else rng.uniform(0, 0.1, ch)) if bias else None
        self.h0 = dev(make(self.n, ch, N)) if carried else None
        self.dout = wide(make(T, ch))
        self.dend = dev(make(self.n, ch, N)) if carried else None
        self.d = ssm.SelectiveDims.make(dtype, self.n, ch, N, groups=G, softplus=soft)
        self.plan = plan_of(self.lens, T)

    def inputs(self):
        return self.x, self.dt, self.A, self.B, self.C

    def more(self):
        return {"D": self.D, "z": self.z, "dt_bias": self.bias}

    def rows(self, width=None):
        return torch.full((self.T, width or self.ch), FILL, device="cuda", dtype=self.tin)

    def forward(self, in_place=False, **kw):
        out = self.rows()
        state = self.h0.clone() if in_place else torch.full((self.n, self.ch, self.N), FILL, device="cuda")
        ssm.selective_forward(self.d, self.T, self.plan, *self.inputs(), state, out, **self.more(),
                              state_in=state if in_place else self.h0, **kw)
        return out, state

    def backward(self, **kw):
        gn = self.G * self.N
        o = {"dx": self.rows(), "ddt": self.rows(), "dB": self.rows(gn), "dC": self.rows(gn),
             "dA": torch.full_like(self.A, FILL), "dend": torch.full((self.n, self.ch, self.N), FILL, device="cuda"),
             "dD": None if self.D is None else torch.full_like(self.D, FILL),
             "dbias": None if self.bias is None else torch.full_like(self.bias, FILL),
             "dz": None if self.z is None else self.rows()}
        ssm.selective_backward(self.d, self.T, self.plan, *self.inputs(), self.dout, o["dx"], o["ddt"], o["dA"],
                               o["dB"], o["dC"], **self.more(), dD=o["dD"], dz=o["dz"], ddt_bias=o["dbias"],
                               state_in=self.h0, dstate=self.dend, dstate_in=o["dend"], **kw)
        return o

    def seq(self, i, s):
        bc = lambda v: host(v)[s].reshape(-1, self.G, self.N)
        h0 = np.zeros((self.ch, self.N)) if self.h0 is None else host(self.h0)[i]
        return dict(x=host(self.x)[s], dt=host(self.dt)[s], A=host(self.A), B=bc(self.B), C=bc(self.C), h0=h0,
                    D=host(self.D), z=None if self.z is None else host(self.z)[s], bias=host(self.bias),
                    soft=self.soft)

    def check_forward(self, out, state):
        for i, s in spans(self.lens):
            want, bound = ref.selective(**self.seq(i, s))
            near(out[s], want["out"], bound["out"], f"out of sequence {i}")
            near(state[i], want["end"], bound["end"], f"state of sequence {i}")
        assert (out[sum(self.lens):] == FILL).all()

    def check_backward(self, o):
        total, bounds = {}, {}
        for i, s in spans(self.lens):
            want, bound = ref.selective(**self.seq(i, s), dout=host(self.dout)[s],
                                        dend=None if self.dend is None else host(self.dend)[i])
            for k in ("dx", "ddt", "dB", "dC", "dz"):
                if k in want:
                    near(o[k][s], want[k].reshape(o[k][s].shape), bound[k].reshape(o[k][s].shape),
                         f"{k} of sequence {i}")
            near(o["dend"][i], want["dend"], bound["dend"], f"dend of sequence {i}")
            for k in ("dA", "dD", "dbias"):
                total[k] = total.get(k, 0) + want[k]
                bounds[k] = bounds.get(k, 0) + bound[k] + self.T * np.abs(want[k])
        for k in ("dA", "dD", "dbias"):
            if o[k] is not None:
                near(o[k], total[k], bounds[k], k)
        for k in ("dx", "ddt", "dB", "dC", "dz"):
            assert o[k] is None or (o[k][sum(self.lens):] == FILL).all(), k


SHAPES = [(16, 8, 1), (48, 16, 1), (64, 16, 2), (16, 32, 1), (32, 64, 1), (96, 8, 3), (80, 32, 5), (272, 16, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_selective(shape, lens, dtype):
    s = Selective(dtype, lens, *shape, spare=5)
    s.check_forward(*s.forward())
    s.check_backward(s.backward())


@pytest.mark.parametrize("without", ["gated", "skip", "bias", "soft", "carried"])
def test_selective_without(without):
    s = Selective("f32", [37, 0, 20], 64, 16, 2, **{without: False}, pad=0)
    s.check_forward(*s.forward())
    s.check_backward(s.backward())


def test_selective_long():
    s = Selective("f32", [0, 700, 1, 300, 0], 32, 16)
    s.check_forward(*s.forward())
    s.check_backward(s.backward())


def test_selective_empty_batches():
    s = Selective("f32", [0, 0], 32, 16)
    _, state = s.forward()
    assert torch.equal(state, s.h0)
    o = s.backward()
    assert torch.equal(o["dend"], s.dend)
    assert all((o[k] == 0).all() for k in ("dA", "dD", "dbias"))
    e = Selective("f32", [], 32, 16)
    e.forward()
    o = e.backward()
    assert all((o[k] == 0).all() for k in ("dA", "dD", "dbias"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_selective_steps(shape, dtype):
    """A prompt token by token, rows anywhere in a pool, against the definition."""
    s = Selective(dtype, [6, 6, 6], *shape)
    pool = torch.full((7, s.ch, s.N), FILL, device="cuda")
    slot = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slot.long()] = s.h0
    out = s.rows()
    for t in range(6):
        at = torch.tensor([t, 6 + t, 12 + t], device="cuda")
        o = torch.empty(3, s.ch, device="cuda", dtype=s.tin)
        pick = lambda v: None if v is None else v[at]
        ssm.selective_step(s.d, s.x[at], s.dt[at], s.A, s.B[at], s.C[at], pool, o, D=s.D, z=pick(s.z),
                           dt_bias=s.bias, slot=slot, num_slots=7)
        out[at] = o
    s.check_forward(out, pool[slot.long()])
    assert (pool[[1, 2, 4, 6]] == FILL).all()
    # a row without a slot
    before = pool.clone()
    o = torch.full((3, s.ch), FILL, device="cuda", dtype=s.tin)
    ssm.selective_step(s.d, s.x[:3], s.dt[:3], s.A, s.B[:3], s.C[:3], pool, o, D=s.D,
                       z=None if s.z is None else s.z[:3], dt_bias=s.bias,
                       slot=torch.tensor([-1, 7, 3], dtype=torch.int32, device="cuda"), num_slots=7)
    assert (o[:2] == FILL).all() and torch.isfinite(o[2]).all()
    assert torch.equal(before[[0, 1, 2, 4, 5, 6]], pool[[0, 1, 2, 4, 5, 6]])


def test_selective_slots_and_in_place():
    s = Selective("bf16", [30, 0, 2, 70, 5], 64, 16)
    out, state = s.forward()
    out2, state2 = s.forward(in_place=True)
    assert torch.equal(out, out2) and torch.equal(state, state2)
    slot = torch.tensor([6, 2, -1, 0, 8], dtype=torch.int32, device="cuda")
    pool = torch.full((8, s.ch, s.N), FILL, device="cuda")
    for i in (0, 1, 3):
        pool[slot[i]] = s.h0[i]
    o = s.rows()
    ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), pool, o, **s.more(), state_in=pool, slot=slot, num_slots=8)
    for i, at in spans(s.lens):
        if i in (0, 1, 3):
            assert torch.equal(o[at], out[at]) and torch.equal(pool[slot[i]], state[i])
        else:
            assert (o[at] == FILL).all()
    assert (pool[[1, 3, 4, 5, 7]] == FILL).all()


def test_selective_non_finite_stays():
    s = Selective("f32", [40, 40], 64, 16, 2, pad=0)
    out, state = s.forward()
    s.x[10, 3] = float("nan")
    s.B[60, 2] = float("inf")
    bad, end = s.forward()
    a = torch.zeros_like(out, dtype=torch.bool)
    a[10:40, 3], a[60:, :32] = True, True
    assert torch.isnan(bad[10:40, 3]).all() and not torch.isfinite(bad[60:, :32]).any()
    assert torch.equal(bad[~a], out[~a])
    assert torch.isnan(end[0, 3]).all() and torch.equal(end[0, 4:], state[0, 4:])
    assert torch.equal(end[1, 32:], state[1, 32:])
    o = s.backward()
    assert torch.isfinite(o["dA"][33:]).all() and torch.isfinite(o["dx"][40:60, 32:]).all()


def test_selective_extremes():
    """Steps of zero keep the state; huge steps forget it; a zero decay rate sums."""
    s = Selective("f32", [20], 16, 16, soft=False, bias=False, gated=False, skip=False, pad=0)
    s.dt.zero_()
    out, state = s.forward()
    assert torch.equal(state, s.h0)
    s.dt.fill_(1e4)
    s.check_forward(*s.forward())
    s.check_backward(s.backward())
    s.A.zero_()
    s.dt.fill_(0.5)
    s.check_forward(*s.forward())
    s.check_backward(s.backward())
    t = Selective("f32", [20], 16, 16, bias=False, pad=0)
    t.dt[::2] = 90.0   # softplus(x) = x
    t.dt[1::2] = -90.0
    t.check_forward(*t.forward())
    t.check_backward(t.backward())


# ---------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------
class Norm:
    def __init__(self, x_dtype, dtype, rows, G, W, gate="after", act="silu", shared=False, centred=False, bias=True,
                 pad=1, seed=0, eps=1e-5, offset=0.0):
        rng = np.random.default_rng([seed, rows, G, W])
        self.rows, self.G, self.W, self.gate, self.act, self.centred = rows, G, W, gate, act, centred
        self.tin, self.tx, self.eps = TIN[dtype], TIN[x_dtype], eps
        self.d = ssm.NormDims.make(x_dtype, dtype, G, W, gate=gate, activation=act, shared=shared, centred=centred,
                                   eps=eps)
        make = lambda: rng.standard_normal((rows, G * W))
        wide = lambda v, t: columns(dev(v), pad, t) if pad and rows else dev(v, t)
        self.x, self.z = wide(make() + offset, self.tx), wide(make(), self.tin) if gate != "none" else None
        self.dout = wide(make(), self.tin)
        wg = 1 if shared else G
        self.w = dev(1 + 0.3 * rng.standard_normal((wg, W)))
        self.b = dev(rng.standard_normal((wg, W))) if bias else None

    def out(self, dtype):
        return torch.full((self.rows, self.G * self.W), FILL, device="cuda", dtype=dtype)

    def forward(self, **kw):
        o = self.out(self.tin)
        ssm.gated_norm(self.d, self.rows, self.x, self.z, self.w, self.b, o, **kw)
        return o

    def backward(self, **kw):
        o = {"dx": self.out(self.tx), "dz": self.out(self.tin) if self.gate != "none" else None,
             "dw": torch.full_like(self.w, FILL), "db": torch.full_like(self.w, FILL)}
        ssm.gated_norm_backward(self.d, self.rows, self.x, self.z, self.w, self.b, self.dout, o["dx"], o["dz"],
                                o["dw"], o["db"], **kw)
        return o

    def want(self, **kw):
        s = lambda v: None if v is None else host(v).reshape(self.rows, self.G, self.W)
        if "dout" in kw:
            kw["dout"] = s(self.dout)
        return ref.norm(s(self.x), s(self.z), host(self.w), host(self.b), gate=self.gate,
                        sig_gate=self.act == "sigmoid", centred=self.centred, eps=float(np.float32(self.eps)), **kw)

    def check(self):
        want, bound = self.want()
        near(self.forward(), want["out"].reshape(self.rows, -1), bound["out"].reshape(self.rows, -1), "out")
        want, bound = self.want(dout=True)
        o = self.backward()
        for k in ("dx", "dz"):
            if o[k] is not None:
                near(o[k], want[k].reshape(self.rows, -1), bound[k].reshape(self.rows, -1), k)
        for k in ("dw", "db"):
            near(o[k], want[k], bound[k], k)


GROUPS = [(1, 8, 1), (1, 8, 2), (3, 16, 5), (7, 40, 3), (5, 64, 4), (33, 128, 6), (4, 136, 2), (3, 256, 2), (9, 512, 1),
          (2, 520, 3), (3, 2048, 1), (2, 2056, 2), (3, 5120, 1), (2, 8192, 1), (300, 32, 8)]


@pytest.mark.parametrize("gate", ["after", "before", "none"])
@pytest.mark.parametrize("shape", GROUPS, ids=str)
def test_norm(shape, gate):
    rows, W, G = shape
    for x_dtype, dtype in (("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")):
        for shared, centred in ((False, True), (True, False)):
            Norm(x_dtype, dtype, rows, G, W, gate, "sigmoid" if centred else "silu", shared, centred).check()


def test_norm_without_bias_and_flat_groups():
    n = Norm("f32", "f32", 6, 4, 64, bias=False, centred=True, offset=3.0)
    n.check()
    n.x[2] = 0.0  # nothing in a group
    n.x[3] = 5.0  # nothing but its mean
    n.check()


def test_norm_no_rows():
    n = Norm("f32", "bf16", 0, 4, 64)
    n.forward()
    o = n.backward()
    assert (o["dw"] == 0).all() and (o["db"] == 0).all()


def test_norm_non_finite_stays():
    n = Norm("f32", "f32", 8, 4, 64, pad=0)
    out = n.forward()
    n.x[3, 70] = float("nan")
    n.z[5, 130] = float("inf")
    bad = n.forward()
    a = torch.zeros_like(out, dtype=torch.bool)
    a[3, 64:128], a[5, 130] = True, True
    assert torch.isnan(bad[3, 64:128]).all() and not torch.isfinite(bad[5, 130])
    assert torch.equal(bad[~a], out[~a])


@pytest.mark.parametrize("shape", [(9, 512, 1), (33, 128, 6), (3, 5120, 1)], ids=str)
def test_norm_more_rows_than_workgroups(shape):
    _, W, G = shape
    n = Norm("f32", "bf16", 3001 if W < 5120 else 1500, G, W, "before", shared=G > 1)
    n.check()
