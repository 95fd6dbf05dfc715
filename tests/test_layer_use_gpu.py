"""The short convolution, the selective recurrence and the output norm as they are used: together and with
the framework's recurrences (decoders, a training step), captured, on other streams, two at once, with
workspaces of the caller's, wrong plans, and sizes beyond 32 bits."""
import numpy as np
import pytest

from tests import layer_reference as ref
from tests import scan_reference as scan

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from sketched_recurrent_state_amd.decoder import (GatedNorm, RecurrentDecoder, SelectiveDecoder,  # noqa: E402
                                                  ShortConv, WindowedDecoder)
from tests.test_layer_gpu import (FILL, TIN, Conv, Norm, Selective, dev, host, near, plan_of, spans)  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def flat(v):
    """The tensors of a result."""
    if isinstance(v, torch.Tensor):
        return [v]
    return [] if v is None else [t for x in (v.values() if isinstance(v, dict) else v) for t in flat(x)]


def same(a, b):
    a, b = flat(a), flat(b)
    assert len(a) == len(b) > 0
    return all(torch.equal(x, y) for x, y in zip(a, b))


# every operator once, with a batch that crosses chunks and groups of chunks
def everything():
    c = Conv("bf16", [100, 0, 61, 3], [128, 128, 64], [64, 64, 0], [0.125, 1.0, 1.0])
    s = Selective("bf16", [100, 0, 61, 3], 80, 16)
    n = Norm("f32", "bf16", 130, 4, 64, "after")
    w = Norm("bf16", "f32", 77, 1, 1032, "before")
    return [c.forward, c.backward, s.forward, s.backward, n.forward, n.backward, w.forward, w.backward]


@pytest.mark.parametrize("which", range(8))
def test_same_bits_from_run_to_run(which):
    """Whatever memory that PyTorch hands out as the workspace holds."""
    f = everything()[which]
    want = f()
    for fill in (float("nan"), 3e38):
        junk = torch.full((1 << 26,), fill, device="cuda")
        del junk
        assert same(f(), want)


@pytest.mark.parametrize("which", [1, 2, 3, 5, 7])
def test_workspaces(which):
    """A workspace of the caller's, exactly large enough, full of NaN and between guard bands."""
    f = everything()[which]
    x = f.__self__
    need = {1: lambda: ssm.conv_sizes(x.d, x.T), 2: lambda: ssm.selective_sizes(x.d, x.T)[0],
            3: lambda: ssm.selective_sizes(x.d, x.T)[1], 5: lambda: ssm.gated_norm_sizes(x.d, x.rows),
            7: lambda: ssm.gated_norm_sizes(x.d, x.rows)}[which]()
    assert need > 0
    want = f()
    buf = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN as fp32
    assert same(f(workspace=buf[4096:4096 + need]), want)
    assert (buf[:4096] == 0xFF).all() and (buf[4096 + need:] == 0xFF).all()
    with pytest.raises(ssm.SSMError, match="workspace"):
        f(workspace=buf[:need - 1])


def test_other_stream_beside_unfinished_work():
    """Calls on a stream of their own, by argument and as the current one, whose inputs that stream makes
    late, and whose workspaces must not be another stream's."""
    fs = everything()
    want = [f() for f in fs]
    st = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for by_argument in (True, False):
        for f, w in zip(fs, want):
            o = f.__self__
            data = o.dout if hasattr(o, "dout") else o.dy[0]
            first = o.x[0] if isinstance(o.x, list) else o.x
            keep, kept = first.clone(), data.clone()
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                first.zero_()
                data.zero_()
                for _ in range(20):
                    x @ x
                first.copy_(keep)
                data.copy_(kept)
                if not by_argument:
                    got = f()
            if by_argument:
                fill = torch.cuda.current_stream()
                got = f(stream=st)  # its outputs were filled on the current stream, before the products end
                fill.wait_stream(st)
            torch.cuda.synchronize()
            assert same(got, w)


def test_two_calls_at_once():
    for make in (lambda k: Conv("bf16", [700, 3], [512, 256], [128, 0], seed=k).backward,
                 lambda k: Selective("bf16", [700, 60], 128, 16, seed=k).forward,
                 lambda k: Selective("bf16", [700, 60], 128, 16, seed=k).backward,
                 lambda k: Norm("f32", "bf16", 3000, 4, 128, seed=k).backward):
        fs = [make(0), make(1)]
        want = [f() for f in fs]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            got = []
            for f, st in zip(fs, streams):
                with torch.cuda.stream(st):
                    got.append(f())
            torch.cuda.synchronize()
            assert all(same(g, w) for g, w in zip(got, want))


def test_two_graphs_beside_eager_calls():
    """Two graphs of every operator, with the workspaces that PyTorch gave the calls, replayed in turn beside
    eager calls."""
    graphs = []
    for _ in range(2):
        fs = everything()
        want = [f() for f in fs]
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            got = [f() for f in fs]
        graphs.append((graph, fs, got, want))
    for _ in range(3):
        for graph, fs, got, want in graphs:
            for t in flat(got):
                t.zero_()
            graph.replay()
            eager = [f() for f in fs]
            torch.randn(1 << 20, device="cuda").sum().item()
            assert all(same(g, w) for g, w in zip(got, want))
            assert all(same(e, w) for e, w in zip(eager, want))


# ---------------------------------------------------------------------------------
# what a call may leave out, and where its outputs may go
# ---------------------------------------------------------------------------------
def test_optional_states():
    """A kept state without a wanted one, a wanted one without a kept, and gradients of either alone."""
    c = Conv("bf16", [20, 0, 2], [64, 32], [32, 0])
    y, state = c.forward()
    out = c.out()
    ssm.conv_forward(c.d, c.T, c.plan, c.x, c.w, c.b, out, state_in=c.kept)
    assert same(out, y)
    whole = c.backward()
    for end in (c.dend, None):
        dx, dw, db, dk = c.out(), torch.empty_like(c.w), torch.empty_like(c.b), torch.empty_like(c.kept)
        keep, c.dend = c.dend, end
        ssm.conv_backward(c.d, c.T, c.plan, c.x, c.w, c.b, c.dy, dx, dw, db, state_in=c.kept, dstate=end)
        assert end is None or (same(dx, whole["dx"]) and same(dw, whole["dw"]))
        c.check_backward(c.backward())
        c.dend = keep
    s = Selective("f32", [20, 0, 2], 32, 16)
    s.dend = None
    s.check_backward(s.backward())
    s.h0, s.dend = None, dev(np.random.default_rng(1).standard_normal((3, 32, 16)))
    s.check_forward(*s.forward())
    s.check_backward(s.backward())


@pytest.mark.parametrize("without", ["gated", "skip", "bias", "soft"])
def test_selective_step_without(without):
    s = Selective("f32", [5], 48, 16, **{without: False}, pad=0)
    pool, out = s.h0.clone(), s.rows()
    d = ssm.SelectiveDims.make("f32", 1, 48, 16, softplus=s.soft)
    for t in range(5):
        at = slice(t, t + 1)
        ssm.selective_step(d, s.x[at], s.dt[at], s.A, s.B[at], s.C[at], pool, out[at], D=s.D,
                           z=None if s.z is None else s.z[at], dt_bias=s.bias)
    s.check_forward(out, pool)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_in_wider_tensors(dtype):
    """Every output of rows as a column range of a wider tensor whose other columns stay as they are."""
    wide = []

    def into(x):
        w = torch.full((x.shape[0], x.shape[1] + 24), FILL, device="cuda", dtype=x.dtype)
        wide.append((w, x.shape[1]))
        return w[:, 8:8 + x.shape[1]]

    c = Conv(dtype, [70, 3], [64, 40], [16, 0])
    (y, state), back = c.forward(), c.backward()
    out, dx = [into(v) for v in y], [into(v) for v in back["dx"]]
    ssm.conv_forward(c.d, c.T, c.plan, c.x, c.w, c.b, out, torch.empty_like(state), state_in=c.kept)
    ssm.conv_backward(c.d, c.T, c.plan, c.x, c.w, c.b, c.dy, dx, torch.empty_like(c.w), state_in=c.kept, dstate=c.dend)
    assert same(out, y) and same(dx, back["dx"])
    s = Selective(dtype, [70, 3], 48, 16)
    (y, state), back = s.forward(), s.backward()
    out = into(y)
    ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), torch.empty_like(state), out, **s.more(), state_in=s.h0)
    g = {k: into(back[k]) for k in ("dx", "ddt", "dB", "dC", "dz")}
    ssm.selective_backward(s.d, s.T, s.plan, *s.inputs(), s.dout, g["dx"], g["ddt"], torch.empty_like(s.A), g["dB"],
                           g["dC"], **s.more(), dD=torch.empty_like(s.D), dz=g["dz"],
                           ddt_bias=torch.empty_like(s.bias), state_in=s.h0, dstate=s.dend)
    assert same(out, y) and all(same(v, back[k]) for k, v in g.items())
    for W, G in ((64, 3), (1032, 1)):
        n = Norm("f32", dtype, 9, G, W)
        y, back = n.forward(), n.backward()
        out, dx, dz = into(y), into(back["dx"]), into(back["dz"])
        ssm.gated_norm(n.d, 9, n.x, n.z, n.w, n.b, out)
        ssm.gated_norm_backward(n.d, 9, n.x, n.z, n.w, n.b, n.dout, dx, dz, torch.empty_like(n.w))
        assert same([out, dx, dz], [y, back["dx"], back["dz"]])
    for w, width in wide:
        assert (w[:, :8] == FILL).all() and (w[:, 8 + width:] == FILL).all()


def test_norm_without_activation_in_the_convolution():
    for norm in (16, 32, 64, 128):
        c = Conv("f32", [40, 7], [norm, 3 * norm, 256], [norm, norm, 128], [2.0, 0.5, 1.0], silu=False, eps=0.5)
        c.check_forward(*c.forward())
        c.check_backward(c.backward())


def test_large_and_tiny_values():
    """Sums of squares that leave fp32's range above are 0 behind the norm; rows of zeros stay zeros."""
    c = Conv("f32", [4], [32], [32], silu=False, bias=False, carried=False, pad=0)
    c.w.zero_()
    c.w[:, -1] = 1
    c.x[0].copy_(torch.tensor([1e30, 0.0, 1e-30, 1.0], device="cuda")[:, None].expand(4, 32))
    y, _ = c.forward()
    assert (y[0][0] == 0).all() and (y[0][1] == 0).all() and (y[0][3] > 0.17).all()
    assert (y[0][2] == y[0][2]).all() and (y[0][2] <= 1e-26).all()
    o = c.backward()
    assert all(torch.isfinite(v[1:]).all() for v in o["dx"])


# ---------------------------------------------------------------------------------
# the decoders with their convolution and norm
# ---------------------------------------------------------------------------------
class Layer:
    """A linear-attention layer from its projections on: convolution, recurrence, gated norm."""

    def __init__(self, rule, dtype, N, H, dk, dv, T, seed=0):
        rng = np.random.default_rng([seed, N, H, dk, dv])
        self.rule, self.N, self.H, self.dk, self.dv = rule, N, H, dk, dv
        self.tin, widths = TIN[dtype], [H * dk, H * dk, H * dv]
        over = 0 if rule == "mamba2" else (dk if dk >= 16 else 0)
        self.cd = ssm.ConvDims.make(dtype, N, 4, widths, norm=[over, over, 0], scale=[dk ** -0.5, 1.0, 1.0])
        self.parts = [(widths[0], over, float(np.float32(dk ** -0.5)) if over else 1.0), (widths[1], over, 1.0),
                      (widths[2], 0, 1.0)]
        self.nd = ssm.NormDims.make("f32", dtype, H, dv, gate="after", shared=True)
        self.d = ssm.Dims.make(rule, dtype, N, H, dk, dv, 4, 4)
        make = lambda *s: rng.standard_normal(s)
        self.w, self.b = dev(make(sum(widths), 4) / 2), dev(make(sum(widths)) / 4)
        self.nw = dev(1 + 0.2 * make(dv))
        C = sum(widths)
        # one projection holds queries, keys, values and the gate
        self.proj = dev(make(T, C + H * dv), self.tin)
        self.q, self.k, self.v, self.z = self.proj.split(widths + [H * dv], 1)
        gate = rng.uniform(0.85, 0.999, (T, H, dk) if rule == "kda" else (T, H))
        self.decay, self.beta = dev(gate), None if rule == "mamba2" else dev(rng.uniform(0, 1, (T, H)))
        self.state = dev(0.3 * make(N, H, dk, dv))

    def tokens(self, at):
        pick = lambda x: None if x is None else x[at]
        return [pick(x) for x in (self.q, self.k, self.v, self.decay, self.beta)], pick(self.z)

    def decoder(self, which):
        conv, norm = ShortConv(self.cd, self.w, self.b), GatedNorm(self.nd, self.nw)
        if which == "recurrent":
            return RecurrentDecoder(self.d, self.state.clone(), conv=conv, norm=norm)
        basis = dev(np.linalg.qr(np.random.default_rng(1).standard_normal((self.H, self.dk, 4)))[0].transpose(0, 2, 1))
        return WindowedDecoder(self.d, self.state.clone(), basis, read=which, conv=conv, norm=norm)

    def exact(self, i, at):
        """Sequence i's outputs from the definitions, its tokens at rows `at`."""
        x = np.concatenate([host(v)[at] for v in (self.q, self.k, self.v)], 1)
        C = x.shape[1]
        o, _ = ref.conv(x, host(self.w), host(self.b), np.zeros((3, C)), self.parts, True, float(np.float32(1e-6)))
        L, H, nk = len(at), self.H, self.H * self.dk
        q, k, v = (o["y"][:, a:b].reshape(L, H, -1) for a, b in ((0, nk), (nk, 2 * nk), (2 * nk, C)))
        beta = None if self.beta is None else host(self.beta)[at]
        y, S = scan.forward(q, k, v, host(self.decay)[at], beta, host(self.state)[i])
        n, _ = ref.norm(y, host(self.z)[at].reshape(L, H, -1), host(self.nw)[None], None, eps=float(np.float32(1e-5)))
        return n["out"], S


@pytest.mark.parametrize("rule", ["mamba2", "gdn", "kda"])
def test_layer_prompts_then_steps(rule):
    """Prompts of unlike lengths, then tokens one at a time, through both decoders, against the
    definitions of all three parts in 64 bits. Of the outputs of a row: the convolution's values are within
    30 u of theirs, the recurrence's path has d_k + 48 roundings and mixes values that lie up to ten times apart,
    the norm divides by the row's own size and adds 60: (10 (d_k + 78) + 60) u of the row's norm."""
    lens, steps = [37, 0, 70], 6
    N, T = 3, sum(lens) + 3 * steps
    for which in ("recurrent", "full"):
        l = Layer(rule, "f32", N, 2, 32, 64, T)
        dec = l.decoder(which)
        first = torch.arange(sum(lens), device="cuda")
        tokens, z = l.tokens(first)
        y = dec.prefill(lens, *tokens, gate=z)
        assert y.shape == (sum(lens), 2, 64) and y.dtype == torch.float32
        outs = []
        for t in range(steps):
            at = sum(lens) + torch.arange(N, device="cuda") * steps + t
            tokens, z = l.tokens(at)
            outs.append(dec.step(*tokens, gate=z))
        if which == "full":
            dec.flush()
        tol = (10 * (32 + 78) + 60) * U
        for i, s in spans(lens):
            at = np.concatenate([np.arange(s.start, s.stop), sum(lens) + i * steps + np.arange(steps)])
            want, S = l.exact(i, at)
            got = np.concatenate([host(y)[s], np.stack([host(o)[i] for o in outs])])
            off = np.linalg.norm(got - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), 1e-30)
            assert off.max() <= tol, (which, i, off.max(), tol)
            assert np.linalg.norm(host(dec.state[i]) - S) <= tol * np.linalg.norm(S)


@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
def test_decoder_is_its_parts(which):
    """In bf16, bit for bit what the calls give one after another."""
    lens = [9, 20, 3]
    l = Layer("gdn", "bf16", 3, 4, 64, 32, sum(lens) + 6)
    dec = l.decoder(which)
    bare = l.decoder(which)
    conv, norm = ShortConv(l.cd, l.w, l.b), bare.norm
    bare.conv = bare.norm = None
    tokens, z = l.tokens(slice(0, sum(lens)))
    y = dec.prefill(lens, *tokens, gate=z)
    q, k, v = (x.view(sum(lens), 4, -1) for x in conv.prefill(lens, *tokens[:3]))
    assert torch.equal(y, norm(bare.prefill(lens, q, k, v, *tokens[3:]), z)) and y.dtype == torch.bfloat16
    for t in range(2):
        tokens, z = l.tokens(slice(sum(lens) + 3 * t, sum(lens) + 3 * t + 3))
        y = dec.step(*tokens, gate=z)
        q, k, v = (x.view(3, 4, -1) for x in conv.step(*tokens[:3]))
        assert torch.equal(y, norm(bare.step(q, k, v, *tokens[3:]), z))
    assert torch.equal(dec.state, bare.state) and torch.equal(dec.conv.state, conv.state)


def test_decoder_refusals():
    l = Layer("gdn", "bf16", 2, 2, 32, 32, 4)
    with pytest.raises(ValueError, match="queries"):
        RecurrentDecoder(l.d, l.state, conv=ShortConv(ssm.ConvDims.make("bf16", 2, 4, [64, 64]), l.w[:128]))
    with pytest.raises(ValueError, match="queries"):
        RecurrentDecoder(l.d, l.state, conv=ShortConv(ssm.ConvDims.make("bf16", 3, 4, [64, 64, 64]), l.w))
    with pytest.raises(ValueError, match="outputs"):
        RecurrentDecoder(l.d, l.state, norm=GatedNorm(ssm.NormDims.make("bf16", "bf16", 2, 32), l.nw))
    with pytest.raises(ValueError, match="norm"):
        WindowedDecoder(l.d, l.state, torch.zeros(2, 4, 32, device="cuda"), read="both", norm=GatedNorm(l.nd, l.nw))
    with pytest.raises(ValueError, match="lengths"):
        ShortConv(l.cd, l.w).prefill([3, 2], l.q, l.k, l.v)


@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
@pytest.mark.parametrize("prefill", [False, True])
def test_refused_calls_leave_the_state(which, prefill):
    """What the recurrence or the norm refuses is refused before the convolution has taken the token."""
    l = Layer("gdn", "bf16", 2, 2, 32, 32, 2)
    dec = l.decoder(which)
    (q, k, v, decay, beta), z = l.tokens(slice(0, 2))
    call = (lambda *a, **kw: dec.prefill([1, 1], *a, **kw)) if prefill else dec.step
    call(q, k, v, decay, beta, gate=z)
    held = [dec.conv.state, dec.state] + ([] if which == "recurrent" else [dec.k_buf, dec.v_buf])
    before = [x.clone() for x in held]
    bad = torch.zeros(3, device="cuda")
    for args, kw in [((decay, beta), {}), ((decay, beta), dict(gate=z[:1])), ((decay, beta), dict(gate=z.float())),
                     ((decay,), dict(gate=z)), ((bad, beta), dict(gate=z)), ((decay, bad), dict(gate=z)),
                     ((None, beta), dict(gate=z)), ((decay.double(), beta), dict(gate=z))]:
        with pytest.raises((ValueError, TypeError)):
            call(q, k, v, *args, **kw)
    weight, dec.norm.weight = dec.norm.weight, bad
    with pytest.raises(ValueError, match="weight"):
        call(q, k, v, decay, beta, gate=z)
    norm, dec.norm = dec.norm, None
    with pytest.raises(ValueError, match="no norm"):
        call(q, k, v, decay, beta, gate=z)
    dec.norm, norm.weight = norm, weight
    assert all(torch.equal(x, y) for x, y in zip(held, before))
    assert call(q, k, v, decay, beta, gate=z).shape == (2, 2, 32)


def test_lengths_on_the_device():
    """Prompts that fill the arrays in part: rows behind them are zero, also behind a norm with a bias."""
    T = 64
    l = Layer("gdn", "bf16", 3, 2, 32, 32, T)
    bias = torch.full((32,), 0.5, device="cuda")
    tokens, z = l.tokens(slice(0, T))
    for lens in ([20, 30, 4], [0, 0, 0], [64, 0, 0]):
        on = torch.tensor(lens, device="cuda")
        n = sum(lens)
        make = lambda: RecurrentDecoder(l.d, l.state.clone(), conv=ShortConv(l.cd, l.w, l.b),
                                        norm=GatedNorm(l.nd, l.nw, bias))
        a, b = make(), make()
        y = a.prefill(on, *tokens, gate=z)
        cut, zc = l.tokens(slice(0, n))
        if n:
            assert torch.equal(y[:n], b.prefill(lens, *cut, gate=zc)) and torch.equal(a.state, b.state)
        assert (y[n:] == 0).all()
        out = ShortConv(l.cd, l.w, l.b).prefill(on, *tokens[:3])
        assert all((v[n:] == 0).all() for v in out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_selective_layer(dtype):
    """A selective layer: convolution, recurrence and norm, prompts and then tokens, as in one long prompt."""
    lens, more, ch, N = [33, 0, 66], 5, 64, 16
    whole = [n + more for n in lens]
    s = Selective(dtype, whole, ch, N, carried=False, pad=0)
    cd = ssm.ConvDims.make(dtype, 3, 4, [ch])
    rng = np.random.default_rng(3)
    w, b = dev(rng.standard_normal((ch, 4)) / 2), dev(rng.standard_normal(ch))
    nd = ssm.NormDims.make(dtype, dtype, 4, 16, gate="none")
    norm = GatedNorm(nd, torch.ones(4, 16, device="cuda"))
    zero = lambda: torch.zeros(3, ch, N, device="cuda")
    make = lambda: SelectiveDecoder(s.d, zero(), s.A, D=s.D, dt_bias=s.bias)

    def rows(at):
        return [v[at] for v in (s.dt, s.B, s.C, s.z)]

    conv, dec = ShortConv(cd, w, b), make()
    long = norm(dec.prefill(whole, *conv.prefill(whole, s.x), *rows(slice(None))))
    c2, d2 = ShortConv(cd, w, b), make()
    first = torch.cat([torch.arange(a.start, a.stop - more) for _, a in spans(whole)]).cuda()
    got = torch.empty_like(long)
    x = s.x.view(-1, ch)
    got[first] = norm(d2.prefill(lens, *c2.prefill(lens, x[first]), *rows(first)))
    for t in range(more):
        at = torch.tensor([a.stop - more + t for _, a in spans(whole)], device="cuda")
        got[at] = norm(d2.step(*c2.step(x[at]), *rows(at)))
    # the same roundings but for the order of the joins: both within the bound of the definition
    assert torch.equal(c2.state, conv.state)
    tol = 400 * U + (2 ** -7 if dtype == "bf16" else 0)
    assert (got.float() - long.float()).norm() <= tol * long.float().norm()
    assert (d2.state - dec.state).norm() <= 400 * U * dec.state.norm()
    want, _ = ref.conv(host(x[:whole[0]]), host(w), host(b), np.zeros((3, ch)), [(ch, 0, 1.0)])
    y, _ = ref.selective(**{**s.seq(0, slice(0, whole[0])), "x": want["y"], "h0": np.zeros((ch, N))})
    n, _ = ref.norm(y["out"].reshape(-1, 4, 16), None, np.ones((4, 16)), None, gate="none", eps=float(np.float32(1e-5)))
    off = np.linalg.norm(host(long[:whole[0]]) - n["out"].reshape(-1, ch)) / np.linalg.norm(n["out"])
    assert off <= 400 * U + (3 * 2 ** -7 if dtype == "bf16" else 0), off


def test_captured_decode_step():
    """A layer's decode step in one graph: projections are written into its inputs between replays."""
    for which in ("recurrent", "full"):
        l = Layer("gdn", "bf16", 4, 2, 64, 64, 4)
        host_side, dec = l.decoder("recurrent"), l.decoder("recurrent")
        tokens, z = l.tokens(slice(0, 4))
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            y = dec.step(*tokens, gate=z)
        for t in range(4):
            l.proj.copy_(torch.randn(l.proj.shape, device="cuda"))
            graph.replay()
            want = host_side.step(*tokens, gate=z)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            torch.randn(1000, device="cuda").sum().item()
        assert torch.equal(dec.state, host_side.state) and torch.equal(dec.conv.state, host_side.conv.state)
        s = Selective("bf16", [4], 64, 16, pad=0)
        sd = ssm.SelectiveDims.make("bf16", 4, 64, 16)
        a, b = (SelectiveDecoder(sd, torch.zeros(4, 64, 16, device="cuda"), s.A, D=s.D, dt_bias=s.bias) for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            out = a.step(s.x, s.dt, s.B, s.C, s.z)
        for t in range(3):
            s.x.copy_(torch.randn(4, 64, device="cuda"))
            graph.replay()
            want = b.step(s.x, s.dt, s.B, s.C, s.z)
            assert torch.equal(out, want) and torch.equal(a.state, b.state)


@pytest.mark.parametrize("rule", ["mamba2", "gdn"])
def test_training_step(rule):
    """Gradients through norm, recurrence and convolution as a training step calls them, against differences
    of the loss in 64 bits along random directions. The loss's own value is L(x); the call's gradient is
    exact to (2 d_k + d_v + 160 + 200) u of the sum of its terms' sizes, taken as the norms' product; the
    differences' own error is h^2 of the third derivative, 1e-6 at h = 1e-4."""
    lens, H, dk, dv = [21, 34], 2, 16, 32
    T = sum(lens)
    l = Layer(rule, "f32", 2, H, dk, dv, T)
    plan = plan_of(lens, T)
    rng = np.random.default_rng(9)
    r = rng.standard_normal((T, H, dv))
    # forward
    conv_in = [l.q, l.k, l.v]
    qkv = [torch.empty(T, w, device="cuda") for w in (H * dk, H * dk, H * dv)]
    ssm.conv_forward(l.cd, T, plan, conv_in, l.w, l.b, qkv)
    y, S = torch.empty(T, H, dv, device="cuda"), torch.empty(2, H, dk, dv, device="cuda")
    ssm.scan_forward(l.d, T, plan, *qkv, l.decay, l.beta, S, y, state_in=l.state)
    # backward; the projection's gradient is one tensor whose column ranges the calls write
    dproj = torch.full_like(l.proj, FILL)
    dq, dk_, dv_, dz = dproj.split([H * dk, H * dk, H * dv, H * dv], 1)
    dy, dnw = torch.empty_like(y), torch.empty_like(l.nw)
    ssm.gated_norm_backward(l.nd, T, y, l.z, l.nw, None, dev(r), dy, dz, dnw)
    g = [torch.empty_like(x) for x in qkv]
    dlog, dbeta, dS = torch.empty_like(l.decay), None if l.beta is None else torch.empty_like(l.beta), torch.empty_like(S)
    ssm.scan_backward(l.d, T, plan, *qkv, l.decay, l.beta, dy, *g, dlog, dbeta, state_in=l.state, dstate_in=dS)
    dw, db = torch.empty_like(l.w), torch.empty_like(l.b)
    ssm.conv_backward(l.cd, T, plan, conv_in, l.w, l.b, g, [dq, dk_, dv_], dw, db)

    v = {"proj": host(l.proj), "w": host(l.w), "b": host(l.b), "nw": host(l.nw)}
    grads = {"proj": host(dproj), "w": host(dw), "b": host(db), "nw": host(dnw)}

    def loss(v):
        total, C, nk = 0.0, 2 * H * dk + H * dv, H * dk
        for i, s in spans(lens):
            o, _ = ref.conv(v["proj"][s, :C], v["w"], v["b"], np.zeros((3, C)), l.parts, True, float(np.float32(1e-6)))
            L = s.stop - s.start
            q, k, x = (o["y"][:, a:b].reshape(L, H, -1) for a, b in ((0, nk), (nk, 2 * nk), (2 * nk, C)))
            y, _ = scan.forward(q, k, x, host(l.decay)[s], None if l.beta is None else host(l.beta)[s], host(l.state)[i])
            n, _ = ref.norm(y, v["proj"][s, C:].reshape(L, H, -1), v["nw"][None], None, eps=float(np.float32(1e-5)))
            total += (n["out"] * r[s]).sum()
        return total

    for name in v:
        for _ in range(3):
            way = rng.standard_normal(v[name].shape)
            h = 1e-4
            up, down = ({**v, name: v[name] + h * k * way} for k in (1, -1))
            want, got = (loss(up) - loss(down)) / (2 * h), (grads[name] * way).sum()
            scale = np.linalg.norm(grads[name]) * np.linalg.norm(way)
            assert abs(got - want) <= ((2 * dk + dv + 360) * U + 1e-6) * scale, (name, got, want, scale)


# ---------------------------------------------------------------------------------
# plans that are none, and sizes
# ---------------------------------------------------------------------------------
class Banded:
    """Tensors with guard bands before and behind them."""

    def __init__(self):
        self.whole = []

    def __call__(self, like, fill=7):
        n = like.numel()
        buf = torch.full((n + 8192,), fill, dtype=like.dtype, device="cuda")
        self.whole.append((buf, n, fill))
        return buf[4096:4096 + n].view(like.shape)

    def intact(self):
        return all((b[:4096] == f).all() and (b[4096 + n:] == f).all() for b, n, f in self.whole)


# changes to the plan of lengths 100, 70, 30 (starts 0 100 170 200, chunks 0 2 4 5, table 0 0 1 1 2 -1)
WRONG = [(3, 201), (3, 2 ** 31 - 1), (1, 180), (0, -1), (1, -5), (4 + 1, 5), (4 + 1, 2 ** 31 - 1), (4 + 2, -1),
         (4 + 3, -2 ** 31), (4 + 3, 2 ** 31 - 1), (4 + 0, 4), (8 + 3, 2), (8 + 4, 0), (8 + 1, 3), (8 + 1, 2 ** 31 - 1),
         (8 + 5, 2), (8 + 0, 1), (2, 100), (1, 0)]


@pytest.mark.parametrize("index,value", WRONG)
def test_wrong_plans_stay_in_their_arrays(index, value):
    c = Conv("bf16", [100, 70, 30], [64, 48], [32, 0], pad=0)
    s = Selective("bf16", [100, 70, 30], 48, 16, pad=0)
    for x in (c, s):
        x.plan[index] = value
    new = Banded()
    y, st = [new(v) for v in c.out()], new(c.kept)
    ssm.conv_forward(c.d, c.T, c.plan, c.x, c.w, c.b, y, st, state_in=c.kept)
    ssm.conv_backward(c.d, c.T, c.plan, c.x, c.w, c.b, c.dy, [new(v) for v in c.out()], new(c.w), new(c.b),
                      state_in=c.kept, dstate=c.dend, dstate_in=new(c.kept),
                      workspace=new(torch.empty(ssm.conv_sizes(c.d, c.T), dtype=torch.uint8, device="cuda")))
    fwd, bwd = ssm.selective_sizes(s.d, s.T)
    ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), new(s.h0), new(s.x), **s.more(), state_in=s.h0,
                          workspace=new(torch.empty(fwd, dtype=torch.uint8, device="cuda")))
    ssm.selective_backward(s.d, s.T, s.plan, *s.inputs(), s.dout, new(s.x), new(s.x), new(s.A), new(s.B), new(s.C),
                           **s.more(), dD=new(s.D), dz=new(s.z), ddt_bias=new(s.bias), state_in=s.h0, dstate=s.dend,
                           dstate_in=new(s.h0), workspace=new(torch.empty(bwd, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    assert new.intact()


def test_many_sequences_of_a_token():
    """100,000 of them, each the first token of a sequence: the convolution's last tap on it and the kept
    ones before, the recurrence's one step."""
    n = 100000
    c = Conv("f32", [1] * n, [16, 8], [16, 0], pad=0)
    y, state = c.forward()
    o = c.backward()
    s = Selective("f32", [1] * n, 16, 8, pad=0)
    out, end = s.forward()
    g = s.backward()
    assert torch.equal(state[:, :2], c.kept[:, 1:]) and torch.equal(state[:, 2], torch.cat(c.x, 1))
    for i in (0, 1, 63, 64, 49999, n - 1):
        at = slice(i, i + 1)
        want, bound = ref.conv(*c.seq(i, at))
        near(y[0][at], want["y"][:, :16], bound["y"][:, :16], f"y of {i}")
        dy = np.concatenate([host(v[at]) for v in c.dy], 1)
        want, bound = ref.conv(*c.seq(i, at), dy=dy, dend=host(c.dend[i]))
        near(o["dkept"][i], want["dkept"], bound["dkept"], f"dkept of {i}")
        want, bound = ref.selective(**s.seq(i, at))
        near(out[at], want["out"], bound["out"], f"out of {i}")
        near(end[i], want["end"], bound["end"], f"end of {i}")
        want, bound = ref.selective(**s.seq(i, at), dout=host(s.dout)[at], dend=host(s.dend[i]))
        near(g["dx"][at], want["dx"], bound["dx"], f"dx of {i}")
        near(g["dend"][i], want["dend"], bound["dend"], f"dend of {i}")


def big(*shape):
    """bf16 values made on the device, a piece at a time."""
    gen = torch.Generator(device="cuda").manual_seed(len(shape))
    return torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)


def test_conv_beyond_32_bits():
    """180,000 tokens x 12,288 channels: 2.2e9 elements. The last sequence lies behind 2^31 of them."""
    lens, C = [179000, 1000], 12288
    T = sum(lens)
    d = ssm.ConvDims.make("bf16", 2, 4, [C], norm=[128])
    w, plan = torch.randn(C, 4, device="cuda") / 2, plan_of(lens, T)
    x, y = big(T, C), torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    ssm.conv_forward(d, T, plan, x, w, None, y)
    cols = slice(C - 128, C)
    parts = [(128, 128, 1.0)]

    def check(first, last, lo):
        want, bound = ref.conv(host(x[first:last, cols]), host(w[cols]), None, np.zeros((3, 128)), parts)
        near(y[first + lo:last, cols], want["y"][lo:], bound["y"][lo:], "y")

    check(0, 5, 0)
    check(178900, 179000, 3)   # inside the first sequence: the first three rows lack their inputs here
    check(179000, 179020, 0)   # its own start
    check(T - 20, T, 3)
    dx, dw = y, torch.empty_like(w)  # y is not needed any more
    ssm.conv_backward(d, T, plan, x, w, None, x, dx, dw)
    xs = host(x[179000:, cols])
    want, bound = ref.conv(xs, host(w[cols]), None, np.zeros((3, 128)), parts, dy=xs)
    near(dx[179000:, cols], want["dx"], bound["dx"], "dx")
    pool = torch.zeros(60000, 3, C, dtype=torch.bfloat16, device="cuda")  # a state pool of 2.2e9
    slot = torch.tensor([59999, 7], dtype=torch.int32, device="cuda")
    out = torch.empty(2, C, dtype=torch.bfloat16, device="cuda")
    for t in range(4):
        ssm.conv_step(d, x[179000 + t:T:500][:2].contiguous(), w, None, pool, out, slot=slot, num_slots=60000)
    near(out[0:1, cols], ref.conv(xs[:4], host(w[cols]), None, np.zeros((3, 128)), parts)[0]["y"][3:],
         ref.conv(xs[:4], host(w[cols]), None, np.zeros((3, 128)), parts)[1]["y"][3:], "step")
    assert (pool[59998] == 0).all() and torch.equal(pool[59999], x[179001:179004])


def test_selective_beyond_32_bits():
    """270,000 tokens x 8,192 channels: 2.2e9 elements of x and of the backward pass's states, and a state pool
    as large; the last sequence lies behind 2^31 of them."""
    lens, ch, N = [269950, 50], 8192, 16
    T = sum(lens)
    d = ssm.SelectiveDims.make("bf16", 2, ch, N)
    A = -torch.rand(ch, N, device="cuda") - 0.5
    plan, x, B = plan_of(lens, T), big(T, ch), big(T, N)
    pool = torch.zeros(20000, ch, N, device="cuda")
    slot = torch.tensor([3, 19999], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    ssm.selective_forward(d, T, plan, x, x, A, B, B, pool, out, slot=slot, num_slots=20000, state_in=pool)
    cols = slice(ch - 16, ch)
    seq = lambda s: dict(x=host(x[s, cols]), dt=host(x[s, cols]), A=host(A[cols]), B=host(B[s])[:, None],
                         C=host(B[s])[:, None], h0=np.zeros((16, N)))
    last = slice(269950, T)
    want, bound = ref.selective(**seq(last))
    near(out[last, cols], want["out"], bound["out"], "out")
    near(pool[19999, cols], want["end"], bound["end"], "end")
    assert (pool[19998] == 0).all()
    # deep in the first sequence, where 300 tokens have forgotten what was before (decays below e^-0.3 a token
    # on average): the outputs of the definition from any state
    want, bound = ref.selective(**seq(slice(269000, 269400)))
    near(out[269300:269400, cols], want["out"][300:], bound["out"][300:], "out inside")
    del pool
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dA, dB, dC = torch.empty_like(A), torch.empty_like(B), torch.empty_like(B)
    ssm.selective_backward(d, T, plan, x, x, A, B, B, x, dx, ddt, dA, dB, dC)
    want, bound = ref.selective(**seq(last), dout=host(x[last, cols]))
    near(dx[last, cols], want["dx"], bound["dx"], "dx")
    near(ddt[last, cols], want["ddt"], bound["ddt"], "ddt")


def test_norm_beyond_32_bits():
    """420,000 rows x 5,120: 2.2e9 elements."""
    n, G, W = 420000, 40, 128
    d = ssm.NormDims.make("bf16", "bf16", G, W, shared=True)
    x, w = big(n, G * W), torch.rand(W, device="cuda") + 0.5
    out = torch.empty_like(x)
    ssm.gated_norm(d, n, x, x, w, None, out)
    at = slice(n - 3, n)
    s = lambda v: host(v[at]).reshape(3, G, W)
    want, bound = ref.norm(s(x), s(x), host(w)[None], None, eps=float(np.float32(1e-5)))
    near(out[at], want["out"].reshape(3, -1), bound["out"].reshape(3, -1), "out")
    dz, dw = torch.empty_like(x), torch.empty_like(w)
    ssm.gated_norm_backward(d, n, x, x, w, None, x, out, dz, dw)
    want, bound = ref.norm(s(x), s(x), host(w)[None], None, eps=float(np.float32(1e-5)), dout=s(x))
    near(out[at], want["dx"].reshape(3, -1), bound["dx"].reshape(3, -1), "dx")
    near(dz[at], want["dz"].reshape(3, -1), bound["dz"].reshape(3, -1), "dz")


@pytest.mark.parametrize("N", [8, 64])
def test_most_channels(N):
    """2^20 of them."""
    ch = 1 << 20
    s = Selective("f32", [3, 2], ch, N, pad=0, gated=False, skip=False)
    out, state = s.forward()
    at = slice(ch - 16, ch)
    for i, t in spans(s.lens):
        q = s.seq(i, t)
        q = {k: (v[:, at] if k in ("x", "dt") else v[at] if k in ("A", "h0", "bias") else v) for k, v in q.items()}
        want, bound = ref.selective(**q)
        near(out[t, at], want["out"], bound["out"], "out")
        near(state[i, at], want["end"], bound["end"], "end")
    c = Conv("f32", [3, 2], [ch], pad=0)
    c.check_forward(*c.forward())
    n = Norm("f32", "f32", 3, 128, 8192, pad=0)
    n.check()
