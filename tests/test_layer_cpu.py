"""The short convolution, the selective recurrence and the output norm without a GPU: refusals, sizes, and
the 64-bit references' gradients against differences."""
import ctypes

import numpy as np
import pytest

import sketched_recurrent_state_amd as ssm
from tests import layer_reference as ref

class Rows(ctypes.Structure):
    """ssm_rows"""

    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class SelectiveInputs(ctypes.Structure):
    """ssm_selective_inputs"""

    _fields_ = ([(n, Rows) for n in ("x", "dt", "z", "B", "C")]
                + [(n, ctypes.c_void_p) for n in ("A", "D", "dt_bias")])


class SelectiveGrads(ctypes.Structure):
    """ssm_selective_grads"""

    _fields_ = ([(n, Rows) for n in ("dx", "ddt", "dz", "dB", "dC")]
                + [(n, ctypes.c_void_p) for n in ("dA", "dD", "ddt_bias")])


A = 1 << 32  # a 16-byte aligned fake device address (never dereferenced)
GAP = 1 << 28


def at(i):
    return A + i * GAP


def rows(i, stride):
    return Rows(at(i), stride)


def parts(first, strides):
    return (Rows * 4)(*[rows(first + p, s) for p, s in enumerate(strides)])


def call(name, *args):
    lib = ssm.library()
    args = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    st = getattr(lib, name)(*args)
    return st, lib.ssm_last_error().decode()


# ---------------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------------
def conv_dims(**kw):
    a = dict(in_dtype="bf16", batch=2, taps=4, channels=[64, 64, 128], norm=[32, 32, 0])
    a.update(kw)
    return ssm.ConvDims.make(a.pop("in_dtype"), a.pop("batch"), a.pop("taps"), a.pop("channels"), **a)


def conv_forward(d, total=100, **kw):
    a = dict(plan=at(0), num_slots=2, slot=at(1), state_in=at(2), x=parts(3, [64, 64, 128]), weight=at(7),
             bias=at(8), state=at(9), y=parts(10, [64, 64, 128]))
    a.update(kw)
    return call("ssm_conv_forward", d, total, a["plan"], a["num_slots"], a["slot"], a["state_in"], a["x"],
                a["weight"], a["bias"], a["state"], a["y"], None)


def conv_backward(d, total=100, **kw):
    a = dict(plan=at(0), state_in=at(2), x=parts(3, [64, 64, 128]), weight=at(7), bias=at(8),
             dy=parts(10, [64, 64, 128]), dstate=at(14), dx=parts(15, [64, 64, 128]), dweight=at(19),
             dbias=at(20), dstate_in=at(21), workspace=at(22), nbytes=1 << 28)
    a.update(kw)
    return call("ssm_conv_backward", d, total, a["plan"], a["state_in"], a["x"], a["weight"], a["bias"],
                a["dy"], a["dstate"], a["dx"], a["dweight"], a["dbias"], a["dstate_in"], a["workspace"],
                a["nbytes"], None)


def conv_step(d, **kw):
    a = dict(num_slots=2, slot=at(1), x=parts(3, [64, 64, 128]), weight=at(7), bias=at(8), state=at(9),
             y=parts(10, [64, 64, 128]))
    a.update(kw)
    return call("ssm_conv_step", d, a["num_slots"], a["slot"], a["x"], a["weight"], a["bias"], a["state"],
                a["y"], None)


def test_conv_dims():
    for kw, status, word in [
            (dict(taps=1), 2, "taps"), (dict(taps=5), 2, "taps"), (dict(batch=-1), 2, "batch"),
            (dict(batch=1 << 24), 2, "batch"), (dict(channels=[60, 64, 128], norm=[0, 0, 0]), 2, "channels[0]"),
            (dict(channels=[0, 64, 128]), 2, "channels[0]"), (dict(channels=[64, 64, 1 << 20]), 2, "channels"),
            (dict(norm=[48, 0, 0]), 2, "norm[0]"), (dict(channels=[64, 72, 128]), 2, "norm[1]"),
            (dict(eps=0.0), 4, "eps"), (dict(eps=float("nan")), 4, "eps"), (dict(activation="sigmoid"), 4, "activation"),
            (dict(in_dtype=2), 4, "in_dtype")]:
        d = conv_dims(**kw)
        for f in (conv_forward, conv_backward):
            st, msg = f(d)
            assert st == status and word in msg, (kw, st, msg)
        st, msg = conv_step(d)
        assert st == status and word in msg, (kw, st, msg)
        with pytest.raises(ssm.SSMError):
            ssm.conv_sizes(d, 10)
    for n in (0, 5):
        d = conv_dims()
        d.parts = n
        assert conv_forward(d)[0] == 2
    with pytest.raises(ValueError):
        ssm.ConvDims.make("bf16", 1, 4, [8] * 5)
    with pytest.raises(ValueError):
        ssm.ConvDims.make("bf16", 1, 4, [8, 8], norm=[0])
    assert call("ssm_conv_sizes", None, 10, None)[0] == 1
    assert conv_forward(conv_dims(), total=-1)[0] == 2
    assert conv_forward(conv_dims(channels=[1 << 19], norm=None, batch=1 << 14), x=parts(3, [1 << 19]))[0] == 2


def test_conv_forward_refusals():
    d = conv_dims()
    for name in ("plan", "weight", "x", "y"):
        st, msg = conv_forward(d, **{name: None})
        assert st == 1 and name in msg, (name, st, msg)
    for name in ("weight", "bias", "state", "state_in"):
        st, msg = conv_forward(d, **{name: at(30) + 8})
        assert st == 3 and name in msg
    st, msg = conv_forward(d, slot=at(30) + 2)
    assert st == 3
    for name, first in (("x", 3), ("y", 10)):
        p = parts(first, [64, 64, 128])
        p[1].data = None
        st, msg = conv_forward(d, **{name: p})
        assert st == 1 and f"{name}[1]" in msg
        p = parts(first, [64, 64, 128])
        p[2].data = at(first + 2) + 8
        st, msg = conv_forward(d, **{name: p})
        assert st == 3 and f"{name}[2]" in msg
        for stride in (56, 68, 0, -64, 1 << 26):
            p = parts(first, [64, 64, 128])
            p[0].stride = stride
            st, msg = conv_forward(d, **{name: p})
            assert st == 2 and f"{name}[0]" in msg, (stride, st, msg)
    st, msg = conv_forward(d, num_slots=0)
    assert st == 2 and "num_slots" in msg
    st, msg = conv_forward(d, num_slots=1, slot=None)
    assert st == 2 and "slot map" in msg
    assert conv_forward(conv_dims(batch=0))[0] == 0
    # outputs over inputs or each other
    st, msg = conv_forward(d, y=parts(3, [64, 64, 128]))
    assert st == 5
    st, msg = conv_forward(d, state=at(2) + 64)
    assert st == 5 and "state" in msg
    one = (Rows * 4)(*[Rows(at(10), 256)] * 3)
    assert conv_forward(d, y=one)[0] == 5


def test_interleaved_rows():
    """Column ranges of one matrix are apart, unless the ranges meet."""
    d = conv_dims()

    def ranges(base, starts, stride=320):
        return (Rows * 4)(*[Rows(base + 2 * s, stride) for s in starts])

    for starts, pair in [((0, 56, 128), (0, 1)), ((0, 64, 120), (1, 2)), ((64, 0, 56), (0, 2)),
                         ((128, 192, 72), (0, 2)), ((0, 128, 184), (1, 2)), ((0, 256, 160), (1, 2)),
                         ((264, 0, 136), (0, 1))]:
        st, msg = conv_forward(d, y=ranges(at(10), starts))
        # pairs are looked at in order: the ones before the named pair were found apart
        assert st == 5 and msg.endswith("y[%d] overlaps y[%d]" % pair), (starts, st, msg)
    # x and y as ranges of one matrix: the last pair alone meets
    x = ranges(at(10), (0, 64, 128), 640)
    st, msg = conv_forward(d, x=x, y=ranges(at(10), (256, 320, 376), 640))
    assert st == 5 and msg.endswith("y[1] overlaps y[2]"), msg
    st, msg = conv_forward(d, x=x, y=ranges(at(10), (576, 320, 376), 640))  # up to a row's end
    assert st == 5 and msg.endswith("y[1] overlaps y[2]"), msg
    st, msg = conv_forward(d, x=x, y=ranges(at(10), (584, 320, 384), 640))  # over the next row's x
    assert st == 5 and msg.endswith("x[0] overlaps y[0]"), msg
    # a row's start before the other array's
    st, msg = conv_forward(d, x=ranges(at(10) + 2 * 640, (0, 64, 128), 640), y=ranges(at(10), (256, 320, 376), 640))
    assert st == 5 and msg.endswith("y[1] overlaps y[2]"), msg
    # another stride: only where the whole spans are apart
    st, msg = conv_forward(d, x=x, y=ranges(at(10) + 2 * 640, (256, 320, 384), 520))
    assert st == 5 and "x[0] overlaps" in msg


def test_conv_backward_refusals():
    d = conv_dims()
    for name in ("plan", "weight", "x", "dy", "dx", "dweight", "workspace"):
        st, msg = conv_backward(d, **{name: None})
        assert st == 1 and name in msg, (name, st, msg)
    need = ssm.conv_sizes(d, 100)
    assert need > 0
    st, msg = conv_backward(d, nbytes=need - 1)
    assert st == 4 and "workspace" in msg
    assert conv_backward(d, nbytes=-1)[0] == 4
    st, msg = conv_backward(d, dweight=at(7))
    assert st == 5
    st, msg = conv_backward(d, dstate_in=at(2))
    assert st == 5 and "dstate_in" in msg
    st, msg = conv_backward(d, dx=parts(10, [64, 64, 128]))
    assert st == 5
    st, msg = conv_backward(d, dbias=at(30) + 4)
    assert st == 3 and "dbias" in msg


def test_conv_step_refusals():
    d = conv_dims()
    for name in ("weight", "x", "y", "state"):
        st, msg = conv_step(d, **{name: None})
        assert st == 1 and name in msg, (name, st, msg)
    assert conv_step(d, num_slots=0)[0] == 2
    assert conv_step(d, num_slots=1, slot=None)[0] == 2
    assert conv_step(d, y=parts(3, [64, 64, 128]))[0] == 5
    assert conv_step(conv_dims(batch=0))[0] == 0


# ---------------------------------------------------------------------------------
# selective recurrence
# ---------------------------------------------------------------------------------
def sel_dims(**kw):
    a = dict(in_dtype="bf16", batch=2, channels=128, d_state=16, groups=2)
    a.update(kw)
    return ssm.SelectiveDims.make(a.pop("in_dtype"), a.pop("batch"), a.pop("channels"), a.pop("d_state"), **a)


def sel_in(**kw):
    a = dict(x=rows(1, 128), dt=rows(2, 128), z=rows(3, 128), B=rows(4, 32), C=rows(5, 32), A=at(6), D=at(7),
             dt_bias=at(8))
    a.update(kw)
    return SelectiveInputs(*a.values())


def sel_grads(**kw):
    a = dict(dx=rows(21, 128), ddt=rows(22, 128), dz=rows(23, 128), dB=rows(24, 32), dC=rows(25, 32), dA=at(26),
             dD=at(27), ddt_bias=at(28))
    a.update(kw)
    return SelectiveGrads(*a.values())


def sel_forward(d, total=100, **kw):
    a = dict(plan=at(0), num_slots=2, slot=at(10), state_in=at(11), ins=sel_in(), state=at(12), out=rows(13, 128),
             workspace=at(14), nbytes=1 << 28)
    a.update(kw)
    return call("ssm_selective_forward", d, total, *a.values(), None)


def sel_backward(d, total=100, **kw):
    a = dict(plan=at(0), state_in=at(11), ins=sel_in(), dout=rows(13, 128), dstate=at(12), grads=sel_grads(),
             dstate_in=at(15), workspace=at(40), nbytes=1 << 40)
    a.update(kw)
    return call("ssm_selective_backward", d, total, *a.values(), None)


def sel_step(d, **kw):
    a = dict(num_slots=2, slot=at(10), ins=sel_in(), state=at(12), out=rows(13, 128))
    a.update(kw)
    return call("ssm_selective_step", d, *a.values(), None)


def test_selective_dims():
    for kw, status, word in [
            (dict(in_dtype=3), 4, "in_dtype"), (dict(batch=-1), 2, "batch"), (dict(d_state=12), 2, "d_state"),
            (dict(d_state=128), 2, "d_state"), (dict(groups=0), 2, "groups"), (dict(groups=3), 2, "channels"),
            (dict(channels=144), 2, "channels"), (dict(channels=0), 2, "channels"),
            (dict(channels=1 << 21), 2, "channels"), (dict(softplus=2), 4, "softplus")]:
        d = sel_dims(**kw)
        for f in (sel_forward, sel_backward, sel_step):
            st, msg = f(d)
            assert st == status and word in msg, (kw, st, msg)
        with pytest.raises(ssm.SSMError):
            ssm.selective_sizes(d, 10)
    assert call("ssm_selective_sizes", None, 10, None, None)[0] == 1
    assert sel_forward(sel_dims(), total=-1)[0] == 2
    st, msg = sel_step(sel_dims(batch=(1 << 24) - 1, channels=1 << 10, d_state=64, groups=1), num_slots=1 << 24)
    assert st == 2 and "batch * channels" in msg
    st, msg = sel_backward(sel_dims(), total=1 << 27)
    assert st == 2 and "total_tokens" in msg


def test_selective_refusals():
    d = sel_dims()
    none = Rows(None, 128)
    for name in ("x", "dt", "B", "C"):
        for f in (sel_forward, sel_backward, sel_step):
            st, msg = f(d, ins=sel_in(**{name: none}))
            assert st == 1 and name in msg, (name, st, msg)
            st, msg = f(d, ins=sel_in(**{name: rows(1, 24)}))
            assert st == 2 and name in msg, (name, st, msg)
    for f in (sel_forward, sel_backward, sel_step):
        assert f(d, ins=None)[0] == 1
        st, msg = f(d, ins=sel_in(A=None))
        assert st == 1 and "A" in msg
        st, msg = f(d, ins=sel_in(D=at(30) + 4))
        assert st == 3 and "D" in msg
    for name in ("plan", "state", "out"):
        st, msg = sel_forward(d, **{name: None})
        assert st == 1 and name in msg
    assert sel_forward(d, out=rows(1, 128))[0] == 5
    assert sel_forward(d, state=at(11) + 64)[0] == 5
    assert sel_forward(d, num_slots=1, slot=None)[0] == 2
    assert sel_forward(sel_dims(batch=0))[0] == 0
    need = ssm.selective_sizes(d, 100)
    if need[0]:
        assert sel_forward(d, nbytes=need[0] - 1)[0] == 4
    assert sel_backward(d, nbytes=need[1] - 1)[0] == 4
    for name in ("plan", "dout", "grads", "workspace"):
        st, msg = sel_backward(d, **{name: None})
        assert st == 1 and name in msg
    for name in ("dx", "ddt", "dz", "dB", "dC", "dA"):
        st, msg = sel_backward(d, grads=sel_grads(**{name: None if name == "dA" else none}))
        assert st == 1 and name in msg, (name, msg)
    st, msg = sel_backward(d, ins=sel_in(z=none))
    assert st == 4 and "dz" in msg
    for name, g in (("D", "dD"), ("dt_bias", "ddt_bias")):
        st, msg = sel_backward(d, ins=sel_in(**{name: None}))
        assert st == 4 and g in msg
        st, msg = sel_backward(d, grads=sel_grads(**{g: None}))
        assert st == 1 and g in msg
    assert sel_backward(d, grads=sel_grads(dB=rows(25, 32)))[0] == 5
    assert sel_step(sel_dims(batch=0))[0] == 0
    assert sel_step(d, state=None)[0] == 1
    assert sel_step(d, out=rows(3, 128))[0] == 5


# ---------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------
def norm_dims(**kw):
    a = dict(x_dtype="f32", in_dtype="bf16", groups=4, width=64)
    a.update(kw)
    return ssm.NormDims.make(a.pop("x_dtype"), a.pop("in_dtype"), a.pop("groups"), a.pop("width"), **a)


def norm_forward(d, n=10, **kw):
    a = dict(x=rows(1, 256), z=rows(2, 256), weight=at(3), bias=at(4), out=rows(5, 256))
    a.update(kw)
    return call("ssm_gated_norm", d, n, *a.values(), None)


def norm_backward(d, n=10, **kw):
    a = dict(x=rows(1, 256), z=rows(2, 256), weight=at(3), bias=at(4), dout=rows(5, 256), dx=rows(6, 256),
             dz=rows(7, 256), dweight=at(8), dbias=at(9), workspace=at(10), nbytes=1 << 28)
    a.update(kw)
    return call("ssm_gated_norm_backward", d, n, *a.values(), None)


def test_norm_refusals():
    for kw, status, word in [
            (dict(x_dtype=2), 4, "x_dtype"), (dict(in_dtype=-1), 4, "in_dtype"), (dict(groups=0), 2, "groups"),
            (dict(width=0), 2, "width"), (dict(width=60), 2, "width"), (dict(width=8200), 2, "width"),
            (dict(width=8192, groups=129), 2, "groups * width"), (dict(gate=3), 4, "gate"),
            (dict(activation="none"), 4, "activation"), (dict(shared=2), 4, "shared"), (dict(eps=0.0), 4, "eps"),
            (dict(eps=float("nan")), 4, "eps")]:
        d = norm_dims(**kw)
        for f in (norm_forward, norm_backward):
            st, msg = f(d)
            assert st == status and word in msg, (kw, st, msg)
        with pytest.raises(ssm.SSMError):
            ssm.gated_norm_sizes(d, 3)
    d = norm_dims()
    assert norm_forward(d, n=-1)[0] == 2
    assert norm_forward(d, n=1 << 30)[0] == 2
    assert norm_forward(d, n=0)[0] == 0
    for name in ("x", "z", "weight", "out"):
        st, msg = norm_forward(d, **{name: None})
        assert st == 1 and name in msg
    for name in ("x", "z", "weight", "dout", "dx", "dz", "dweight", "workspace"):
        st, msg = norm_backward(d, **{name: None})
        assert st == 1 and name in msg, name
    plain = norm_dims(gate="none")
    st, msg = norm_forward(plain)
    assert st == 4 and "z" in msg
    st, msg = norm_backward(plain, z=None)
    assert st == 4 and "dz" in msg
    assert norm_forward(d, out=rows(1, 256))[0] == 5
    assert norm_forward(d, x=rows(1, 248))[0] == 2
    assert norm_backward(d, dx=rows(5, 256))[0] == 5
    assert norm_backward(d, nbytes=ssm.gated_norm_sizes(d, 10) - 1)[0] == 4


@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -127, -1e-6])
def test_eps_below_the_normal_numbers(eps):
    """The kernels' reciprocal root takes them for 0, and 0 / 0 is not the formula's 0."""
    for f in (conv_forward, conv_backward, conv_step):
        st, msg = f(conv_dims(eps=eps))
        assert st == 4 and "eps" in msg
    for f in (norm_forward, norm_backward):
        st, msg = f(norm_dims(eps=eps))
        assert st == 4 and "eps" in msg
    assert ssm.conv_sizes(conv_dims(eps=eps, norm=[0, 0, 0]), 10) > 0  # not used without a norm
    assert ssm.conv_sizes(conv_dims(eps=2.0 ** -126), 10) > 0
    assert ssm.gated_norm_sizes(norm_dims(eps=2.0 ** -126), 10) > 0


def test_selective_grids_below_32_bits():
    """Calls whose launches would have 2^32 threads: a token of 2047 rows of 2^20 channels x 8 states (a lane has 2 of
    them, for two rows), and dB and dC (a thread each) of 2^27 - 1 tokens x 16 states."""
    st, msg = sel_step(sel_dims(batch=2047, channels=1 << 20, d_state=8, groups=1), num_slots=2047)
    assert st == 2 and "batch * channels" in msg
    st, msg = sel_backward(sel_dims(groups=1), total=(1 << 27) - 1)
    assert st == 2 and "total_tokens" in msg


def test_binding_checks():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ssm.gated_norm(norm_dims(), 3, x, x, torch.zeros(256), None, x)
    with pytest.raises(ValueError, match="parts"):
        ssm.conv_step(conv_dims(), [at(1)], at(2), None, at(3), [at(4)] * 3)
    with pytest.raises(ValueError, match="32 bits"):
        ssm.gated_norm(norm_dims(), 1 << 31, at(1), at(2), at(3), None, at(4))
    with pytest.raises(ValueError):
        ssm.conv_backward(conv_dims(), 10, at(0), [at(1)] * 3, at(2), None, [at(3)] * 3, [at(4)] * 3, at(5))


# ---------------------------------------------------------------------------------
# the references' gradients against differences
# ---------------------------------------------------------------------------------
def differences(f, leaves, got, eps=1e-6, rel=2e-7):
    """f(leaves) -> a number; got[name]: its gradient. Central differences of every element."""
    for name, grad in got.items():
        x = leaves[name]
        for i in np.ndindex(x.shape):
            old = x[i]
            x[i] = old + eps
            up = f(leaves)
            x[i] = old - eps
            down = f(leaves)
            x[i] = old
            want = (up - down) / (2 * eps)
            assert abs(want - grad[i]) <= rel * (1 + abs(want)) * 50, (name, i, want, grad[i])


@pytest.mark.parametrize("L", [1, 2, 7])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_reference_gradients(L, silu):
    rng = np.random.default_rng([L, silu])
    K, ps = 4, [(4, 2, 0.7), (3, 0, 1.0)]
    v = dict(x=rng.standard_normal((L, 7)), w=rng.standard_normal((7, K)), b=rng.standard_normal(7),
             kept=rng.standard_normal((K - 1, 7)))
    dy, dend = rng.standard_normal((L, 7)), rng.standard_normal((K - 1, 7))

    def f(v):
        o, _ = ref.conv(v["x"], v["w"], v["b"], v["kept"], ps, silu)
        return (o["y"] * dy).sum() + (o["end"] * dend).sum()

    o, _ = ref.conv(v["x"], v["w"], v["b"], v["kept"], ps, silu, dy=dy, dend=dend)
    differences(f, v, {"x": o["dx"], "w": o["dw"], "b": o["db"], "kept": o["dkept"]})


@pytest.mark.parametrize("soft", [True, False])
def test_selective_reference_gradients(soft):
    rng = np.random.default_rng(5)
    L, D, N, G = 5, 4, 3, 2
    v = dict(x=rng.standard_normal((L, D)), dt=rng.standard_normal((L, D)), A=-rng.uniform(0.2, 2, (D, N)),
             B=rng.standard_normal((L, G, N)), C=rng.standard_normal((L, G, N)), h0=rng.standard_normal((D, N)),
             D=rng.standard_normal(D), z=rng.standard_normal((L, D)), bias=rng.standard_normal(D))
    if not soft:
        v["dt"], v["bias"] = np.abs(v["dt"]), np.abs(v["bias"])
    dout, dend = rng.standard_normal((L, D)), rng.standard_normal((D, N))

    def f(v):
        o, _ = ref.selective(**v, soft=soft)
        return (o["out"] * dout).sum() + (o["end"] * dend).sum()

    o, _ = ref.selective(**v, soft=soft, dout=dout, dend=dend)
    differences(f, v, {"x": o["dx"], "dt": o["ddt"], "A": o["dA"], "B": o["dB"], "C": o["dC"], "h0": o["dend"],
                       "D": o["dD"], "z": o["dz"], "bias": o["dbias"]})


@pytest.mark.parametrize("gate", ["after", "before", "none"])
@pytest.mark.parametrize("centred", [True, False])
@pytest.mark.parametrize("sig", [True, False])
def test_norm_reference_gradients(gate, centred, sig):
    rng = np.random.default_rng(7)
    for wg in (1, 2):
        v = dict(x=rng.standard_normal((3, 2, 5)), z=rng.standard_normal((3, 2, 5)),
                 w=rng.standard_normal((wg, 5)), b=rng.standard_normal((wg, 5)))
        dout = rng.standard_normal((3, 2, 5))
        kw = dict(gate=gate, sig_gate=sig, centred=centred)

        def f(v):
            o, _ = ref.norm(v["x"], v["z"] if gate != "none" else None, v["w"], v["b"], **kw)
            return (o["out"] * dout).sum()

        o, _ = ref.norm(v["x"], v["z"] if gate != "none" else None, v["w"], v["b"], **kw, dout=dout)
        got = {"x": o["dx"], "w": o["dw"], "b": o["db"]}
        if gate != "none":
            got["z"] = o["dz"]
        differences(f, v, got)
