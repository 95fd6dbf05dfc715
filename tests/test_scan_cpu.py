"""Whole-sequence scan and serving plans without a GPU: argument checks, sizes, and the
64-bit reference against differences."""
import numpy as np
import pytest

import sketched_recurrent_state_amd as ssm
from tests import scan_reference as ref

A = 1 << 32  # a 16-byte aligned fake device address (never dereferenced)


def dims(rule="gdn", in_dtype="bf16", batch=2, heads=3, d_k=32, d_v=64):
    return ssm.Dims.make(rule, in_dtype, batch, heads, d_k, d_v, 4, 4)


def addrs(n, gap=1 << 28):
    return [A + i * gap for i in range(n)]


def raw(name, *args):
    import ctypes
    lib = ssm.library()
    args = [ctypes.byref(a) if isinstance(a, ssm.Dims) else a for a in args]
    st = getattr(lib, name)(*args)
    return st, lib.ssm_last_error().decode()


def forward(d, total=100, **kw):
    p = addrs(12)
    a = dict(plan=p[0], num_slots=d.batch, slot=None, state_in=p[1], q=p[2], k=p[3], v=p[4],
             decay=p[5], beta=p[6], state=p[7], y=p[8], workspace=p[9], nbytes=1 << 40)
    a.update(kw)
    return raw("ssm_scan_forward", d, total, a["plan"], a["num_slots"], a["slot"], a["state_in"],
               a["q"], a["k"], a["v"], a["decay"], a["beta"], a["state"], a["y"], a["workspace"],
               a["nbytes"], None)


def backward(d, total=100, **kw):
    p = addrs(18)
    names = ["plan", "state_in", "q", "k", "v", "decay", "beta", "dy", "dstate", "dq", "dk", "dv",
             "dlog_decay", "dbeta", "dstate_in", "workspace"]
    a = dict(zip(names, p), nbytes=1 << 40)
    a.update(kw)
    return raw("ssm_scan_backward", d, total, *[a[n] for n in names], a["nbytes"], None)


def test_forward_refusals():
    d = dims()
    for name in ("plan", "q", "k", "v", "decay", "beta", "state", "y", "workspace"):
        st, msg = forward(d, **{name: None})
        assert st == 1 and name in msg, (name, st, msg)
    assert forward(dims(rule="mamba2"))[0] == 4  # Mamba-2 takes no beta
    for name in ("q", "state", "y", "workspace", "state_in"):
        st, msg = forward(d, **{name: A + (13 << 28) + 8})
        assert st == 3 and name in msg
    st, msg = forward(d, plan=A + 2)
    assert st == 3 and "plan" in msg
    st, msg = forward(d, y=A + (2 << 28))
    assert st == 5
    st, msg = forward(d, state=A + (1 << 28) + 64)  # partly over state_in
    assert st == 5 and "state" in msg
    need = ssm.scan_sizes(d, 100)[1]
    st, msg = forward(d, nbytes=need - 1)
    assert st == 4 and "workspace" in msg
    st, msg = forward(d, nbytes=-1)
    assert st == 4
    st, msg = forward(d, total=-1)
    assert st == 2 and "total_tokens" in msg
    st, msg = forward(d, num_slots=0)
    assert st == 2 and "num_slots" in msg
    st, msg = forward(d, num_slots=1)
    assert st == 2 and "slot map" in msg
    st, msg = forward(dims(heads=1 << 12), total=1 << 17)
    assert st == 2 and "heads" in msg
    st, msg = forward(dims(heads=65537, batch=1), total=1)
    assert st == 2 and "heads" in msg
    assert forward(dims(batch=0))[0] == 0
    bad = dims()
    bad.d_k = 48
    assert forward(bad)[0] == 2


def test_backward_refusals():
    d = dims()
    for name in ("plan", "q", "k", "v", "decay", "beta", "dy", "dq", "dk", "dv", "dlog_decay",
                 "dbeta", "workspace"):
        st, msg = backward(d, **{name: None})
        assert st == 1 and name in msg, (name, st, msg)
    m = dims(rule="mamba2")
    assert backward(m)[0] == 4
    st, msg = backward(m, beta=None)
    assert st == 4 and "dbeta" in msg
    st, msg = backward(d, dq=A + (3 << 28))  # over k
    assert st == 5
    st, msg = backward(d, dstate_in=A + (1 << 28))  # over state_in
    assert st == 5 and "dstate_in" in msg
    st, msg = backward(d, dlog_decay=A + (20 << 28) + 2)
    assert st == 3 and "dlog_decay" in msg
    st, msg = backward(dims(rule="kda"), dlog_decay=A + (20 << 28) + 4)
    assert st == 3 and "dlog_decay" in msg
    st, msg = backward(d, nbytes=ssm.scan_sizes(d, 100)[2] - 1)
    assert st == 4 and "workspace" in msg
    assert backward(dims(batch=0))[0] == 0


def test_plan_refusals():
    assert raw("ssm_scan_plan", A, -1, 10, A + 4096, None)[0] == 2
    assert raw("ssm_scan_plan", A, 1 << 24, 10, A + 4096, None)[0] == 2
    assert raw("ssm_scan_plan", A, 4, -1, A + 4096, None)[0] == 2
    assert raw("ssm_scan_plan", None, 4, 10, A, None)[0] == 1
    assert raw("ssm_scan_plan", A, 4, 10, None, None)[0] == 1
    assert raw("ssm_scan_plan", A, 4, 10, A + 8, None)[0] == 5
    assert raw("ssm_scan_plan", A + 2, 4, 10, A + 4096, None)[0] == 3
    assert raw("ssm_scan_plan", None, 0, 10, None, None)[0] == 0
    d = dims(batch=8)
    p = addrs(5)
    for i, name in enumerate(("lengths", "tau", "parity", "update_rows", "n_update")):
        q = list(p)
        q[i] = None
        st, msg = raw("ssm_window_plan", d, *q, None)
        assert st == 1 and name in msg
    st, msg = raw("ssm_window_plan", d, p[0], p[1], p[1] + 16, p[3], p[4], None)
    assert st == 5
    st, msg = raw("ssm_window_plan", d, p[0] + 1, *p[1:], None)
    assert st == 3
    assert raw("ssm_window_plan", dims(batch=0), None, None, None, None, None, None)[0] == 0


def test_sizes():
    for rule in ("mamba2", "gdn", "kda"):
        d = dims(rule=rule, batch=5)
        ints, fwd, bwd = ssm.scan_sizes(d, 1000)
        assert ints == 2 * 6 + 1000 // 64 + 5
        assert 0 < fwd < bwd
        assert ssm.scan_sizes(d, 0)[0] == 2 * 6 + 5
    with pytest.raises(ssm.SSMError):
        ssm.scan_sizes(dims(), -1)


def test_binding_checks():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="device tensor"):
        ssm.scan_plan(torch.zeros(3, dtype=torch.int32), 10, torch.zeros(20, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        ssm.window_plan(dims(), *[torch.zeros(2, dtype=torch.int32)] * 5)
    with pytest.raises(ValueError):
        p = addrs(10)
        ssm.scan_forward(dims(), 100, *p[:6], p[6], p[7])  # raw addresses, no workspace


@pytest.mark.parametrize("rule", ["mamba2", "gdn", "kda"])
def test_reference_gradients_match_differences(rule):
    rng = np.random.default_rng(3)
    T, H, dk, dv = 7, 2, 4, 3
    q, k, v = rng.standard_normal((T, H, dk)), rng.standard_normal((T, H, dk)) / 2, rng.standard_normal((T, H, dv))
    gate = rng.uniform(0.3, 0.99, (T, H, dk) if rule == "kda" else (T, H))
    beta = None if rule == "mamba2" else rng.uniform(0, 1, (T, H))
    S0, dy, dS = rng.standard_normal((H, dk, dv)), rng.standard_normal((T, H, dv)), rng.standard_normal((H, dk, dv))
    got, _ = ref.backward(q, k, v, gate, beta, S0, dy, dS)

    def loss(q, k, v, lg, b, S):
        y, last = ref.forward(q, k, v, np.exp(lg), b, S)
        return (y * dy).sum() + (last * dS).sum()

    args = [q, k, v, np.log(gate), beta, S0]
    for i, name in enumerate(("dq", "dk", "dv", "dlog", "dbeta", "dS0")):
        if args[i] is None:
            continue
        # central differences: error of order eps^2 of the third derivative, and 2^-53 / eps
        d = rng.standard_normal(args[i].shape)
        eps = 1e-5
        hi = loss(*[a if j != i else a + eps * d for j, a in enumerate(args)])
        lo = loss(*[a if j != i else a - eps * d for j, a in enumerate(args)])
        want = (got[name] * d).sum()
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-7 * (np.abs(got[name] * d).sum() + 1)


def test_prefill_refuses_lengths_that_do_not_fit():
    import torch
    from sketched_recurrent_state_amd.decoder import RecurrentDecoder
    d = ssm.Dims.make("mamba2", "f32", 2, 1, 16, 16, 4, 4)
    dec = RecurrentDecoder(d, torch.zeros(2, 1, 16, 16))
    q, decay = torch.zeros(5, 1, 16), torch.ones(5, 1)
    for lengths in ([5], [2, 2], [3, 3], [6, -1], torch.tensor([2, 2]), []):
        with pytest.raises(ValueError):
            dec.prefill(lengths, q, q, q, decay)


class _Streams:
    """What the binding uses of torch.cuda, without a device: notes the stream that is current when
    memory is taken."""

    class Stream:
        def __init__(self, handle, device):
            self.cuda_stream, self.device = handle, device

    def __init__(self, device):
        self.device, self.now, self.took = device, self.Stream(0x100, device), []
        self.uint8 = "uint8"
        self.cuda = self

    def ExternalStream(self, handle, device=None):
        assert handle != 0, "the default stream has no external handle"
        return self.Stream(handle, device)

    def default_stream(self, device=None):
        return self.Stream(0, device)

    def current_stream(self, device=None):
        return self.now

    def stream(self, s):
        import contextlib

        @contextlib.contextmanager
        def switched():
            before, self.now = self.now, s
            yield
            self.now = before
        return switched()

    def empty(self, n, dtype=None, device=None):
        self.took.append(self.now.cuda_stream)

        class Block:
            def record_stream(self, stream):
                pass
        return Block()


@pytest.mark.parametrize("kind", ["current", "stream", "address", "default", "foreign object"])
def test_workspace_is_taken_on_the_calls_stream(monkeypatch, kind):
    """A block from another stream's pool may still be in use by work queued on that stream."""
    import types
    fake = _Streams("cuda:0")
    monkeypatch.setattr(ssm, "_torch", fake)
    tensor = types.SimpleNamespace(device="cuda:0")
    stream, want = {"current": (None, 0x100), "stream": (fake.Stream(0x200, "cuda:0"), 0x200),
                    "address": (0x300, 0x300), "default": (0, 0),
                    "foreign object": (types.SimpleNamespace(cuda_stream=0x400), 0x400)}[kind]
    for which in (1, 2):
        ssm._scan_workspace(None, dims(), 100, which, (None, tensor), stream)
    assert fake.took == [want, want] and fake.now.cuda_stream == 0x100


def test_workspace_of_a_stream_on_another_device_is_refused(monkeypatch):
    import types
    fake = _Streams("cuda:0")
    monkeypatch.setattr(ssm, "_torch", fake)
    with pytest.raises(ValueError, match="device"):
        ssm._scan_workspace(None, dims(), 100, 1, (types.SimpleNamespace(device="cuda:0"),),
                            fake.Stream(0x200, "cuda:1"))
    assert fake.took == []


def _prefill_cpu(monkeypatch, lengths, tokens):
    """prefill with the library calls noted instead of made: the lengths that reach the plan."""
    import torch
    from sketched_recurrent_state_amd import decoder
    seen = []
    monkeypatch.setattr(decoder, "scan_plan", lambda lens, total, plan: seen.append((lens.tolist(), total)))
    monkeypatch.setattr(decoder, "scan_forward", lambda *a, **kw: None)
    d = ssm.Dims.make("mamba2", "f32", 2, 1, 16, 16, 4, 4)
    q, decay = torch.zeros(tokens, 1, 16), torch.ones(tokens, 1)
    decoder.RecurrentDecoder(d, torch.zeros(2, 1, 16, 16)).prefill(lengths, q, q, q, decay)
    return seen


def test_prefill_counts_lengths_of_any_integer_type(monkeypatch):
    """The sum of lengths is that of the numbers, whatever the width of their type."""
    import torch
    assert _prefill_cpu(monkeypatch, torch.tensor([[1], [2]]), 3) == [([1, 2], 3)]
    narrow = [torch.tensor([100, 100], dtype=torch.int8), np.array([100, 100], np.int8),
              torch.tensor([100, 100], dtype=torch.uint8), np.array([100, 100], np.uint16), (100, np.int8(100))]
    for lengths in narrow:
        with pytest.MonkeyPatch.context() as m:
            assert _prefill_cpu(m, lengths, 200) == [([100, 100], 200)]
    for lengths in (torch.tensor([200, 100], dtype=torch.uint8), np.array([200, 100], np.uint8)):
        with pytest.raises(ValueError):  # 300 modulo 2^8 is 44
            _prefill_cpu(monkeypatch, lengths, 44)
    with pytest.raises(ValueError):  # 2^32 tokens; the numbers modulo 2^32 sum to 0
        _prefill_cpu(monkeypatch, np.array([2 ** 31, 2 ** 31], np.uint32), 0)
    with pytest.raises(ValueError):
        _prefill_cpu(monkeypatch, np.array([2 ** 32 + 1, 0]), 1)


def test_prefill_refuses_lengths_that_are_no_counts(monkeypatch):
    import torch
    for lengths in ([1.5, 1.5], torch.tensor([1.5, 1.5]), np.array([2.5, 0.5]), ["1", "2"], [None, 3],
                    torch.tensor([[1, 2], [0, 0]]), np.array([3]), [[1], [2]], 3, torch.tensor(3)):
        with pytest.raises((TypeError, ValueError)):
            _prefill_cpu(monkeypatch, lengths, 3)


def test_counts_beyond_32_bits_are_refused():
    """The library takes 32-bit counts: one of 2^32 + 100 must not arrive as 100."""
    torch = pytest.importorskip("torch")
    big, d, p = 2 ** 32 + 100, dims(), addrs(20)
    ws = torch.empty(16)
    for total in (big, -big, 2 ** 31):
        with pytest.raises(ValueError, match="total_tokens"):
            ssm.scan_sizes(d, total)
        with pytest.raises(ValueError, match="total_tokens"):
            ssm.scan_plan(A, total, 2 * A, n_seqs=2)
        with pytest.raises(ValueError, match="total_tokens"):
            ssm.scan_forward(d, total, *p[:8], workspace=ws, stream=0)
        with pytest.raises(ValueError, match="total_tokens"):
            ssm.scan_backward(d, total, *p[:12], workspace=ws, stream=0)
    with pytest.raises(ValueError, match="n_seqs"):
        ssm.scan_plan(A, 100, 2 * A, n_seqs=2 ** 32 + 2)
    with pytest.raises(ValueError, match="num_slots"):
        ssm.scan_forward(d, 100, *p[:8], num_slots=2 ** 32 + 2, workspace=ws, stream=0)
    assert ssm.scan_sizes(d, 100)[0] == 2 * 3 + 1 + 2


@pytest.mark.parametrize("open_window", [False, True])
def test_prefill_runs_on_the_states_device(monkeypatch, open_window):
    """All of a prefill's calls, the window's flush and the sketch's refresh with it, are made on the
    state's device, whichever is the current one: the scan's own stream is that device's."""
    import contextlib
    import torch
    from sketched_recurrent_state_amd import decoder
    now, made = ["cuda:0"], []

    @contextlib.contextmanager
    def switched(device):
        before, now[0] = now[0], str(device)
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "device_of", lambda x: switched("the state's"))
    for name in ("scan_plan", "scan_forward", "window_update_refresh"):
        monkeypatch.setattr(decoder, name, lambda *a, name=name, **kw: made.append((name, now[0])))
    d = ssm.Dims.make("mamba2", "f32", 2, 1, 16, 16, 4, 4)
    q, decay = torch.zeros(5, 1, 16), torch.ones(5, 1)
    dec = decoder.WindowedDecoder(d, torch.zeros(2, 1, 16, 16), torch.zeros(1, 4, 16))
    dec.tau = 1 if open_window else 0
    dec.prefill([2, 3], q, q, q, decay)
    decoder.RecurrentDecoder(d, dec.state).prefill([2, 3], q, q, q, decay)
    names = ["scan_plan", "scan_forward"]
    want = ["window_update_refresh"] * open_window + names + ["window_update_refresh"] + names
    assert made == [(x, "the state's") for x in want] and now == ["cuda:0"]


def _parts(x):
    """An fp32 value cut into three bf16 ones, as the scan cuts it."""
    cut = lambda x: (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    h = cut(x)
    m = cut(x - h)
    return h, m, x - h - m


def test_three_parts_hold_an_fp32_value():
    """Parts of 8 bits that add up to the value, and what the six products of parts that are taken
    leave of a product of two values: below 2 * 2^-22 + 2^-30, toward zero, 0.6 * 2^-24 in the mean."""
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(200000), rng.uniform(1, 2, 200000),
                        np.ldexp(1.0, rng.integers(-90, 90, 1000)), [1 + 2 ** -7 - 2 ** -23] * 2])
    a, b = (v.astype(np.float32) for v in (x, np.roll(x, 1)))
    pa, pb = _parts(a), _parts(b)
    for v, parts in ((a, pa), (b, pb)):
        assert all(np.array_equal(p, (p.view(np.uint32) >> 16 << 16).view(np.float32)) for p in parts)
        assert np.array_equal(sum(p.astype(np.float64) for p in parts), v.astype(np.float64))
    ha, ma, la, hb, mb, lb = (p.astype(np.float64) for p in pa + pb)
    taken = la * hb + ha * lb + ma * mb + ma * hb + ha * mb + ha * hb
    product = a.astype(np.float64) * b.astype(np.float64)
    lost = (product - taken) / product
    assert lost.min() > -2.0 ** -50 and lost.max() < 2.0 ** -21 + 2.0 ** -30
    assert lost.max() > 7.5 * 2.0 ** -24  # of 1 + 2^-7 - 2^-23, squared
    assert 0.55 < lost[:200000].mean() * 2.0 ** 24 < 0.7
