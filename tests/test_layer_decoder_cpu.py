"""The decoders' checks of a call's arguments, with stand-ins for device tensors: an array on another device than the
state, arrays that overlap, addresses that the library cannot read."""
import pytest

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from sketched_recurrent_state_amd import decoder  # noqa: E402


class Stub:
    """A contiguous device tensor's description; nothing is behind its address."""

    is_cuda = True

    def __init__(self, at, shape, dtype=torch.float32, device=0):
        self.at, self.shape, self.dtype, self.device = at, torch.Size(shape), dtype, device

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)


D = ssm.Dims.make("gdn", "bf16", 2, 2, 32, 32, 4, 4)
NORM = ssm.NormDims.make("f32", "bf16", 2, 32, shared=True)
MB = 1 << 20


def call(**kw):
    a = dict(decay=Stub(1 * MB, (2, 2)), beta=Stub(2 * MB, (2, 2)), gate=Stub(3 * MB, (2, 64), torch.bfloat16),
             weight=Stub(4 * MB, (32,)), state=Stub(5 * MB, (2, 2, 32, 32)), y=Stub(6 * MB, (2, 2, 32)),
             conv_state=Stub(7 * MB, (2, 3, 192), torch.bfloat16), sketch=Stub(8 * MB, (2, 2, 4, 32)))
    a.update(kw)
    conv = type("Conv", (), {"state": a["conv_state"]})
    norm = decoder.GatedNorm(NORM, a["weight"])
    decoder._check_around(D, 2, conv, norm, a["decay"], a["beta"], a["gate"], a["state"], kept=(a["sketch"],),
                          ys=(a["y"],))


def test_arguments_that_fit():
    call()
    call(y=None)


@pytest.mark.parametrize("name,shape,dtype", [("decay", (2, 2), torch.float32), ("beta", (2, 2), torch.float32),
                                              ("gate", (2, 64), torch.bfloat16), ("weight", (32,), torch.float32),
                                              ("y", (2, 2, 32), torch.float32)])
def test_one_argument(name, shape, dtype):
    with pytest.raises(ValueError, match=f"{name}: on device 1"):
        call(**{name: Stub(20 * MB, shape, dtype, device=1)})
    with pytest.raises(ValueError, match=f"{name}: not 16-byte aligned"):
        call(**{name: Stub(20 * MB + 8, shape, dtype)})
    for at, own in ((5, "state"), (7, "conv_state")):
        with pytest.raises(ValueError, match="overlaps"):
            call(**{name: Stub(at * MB + 16, shape, dtype)})


@pytest.mark.parametrize("at", [1, 2, 3, 4, 8])
def test_the_output_over_what_the_call_reads(at):
    with pytest.raises(ValueError, match="y overlaps"):
        call(y=Stub(at * MB, (2, 2, 32)))


def test_neighbours_do_not_overlap():
    call(y=Stub(1 * MB + 16, (2, 2, 32)))
    call(y=Stub(5 * MB - 512, (2, 2, 32)))


@pytest.mark.parametrize("norm", [dict(eps=0.0), dict(eps=float("nan")), dict(gate=3), dict(activation="none")])
def test_a_norm_that_every_call_would_refuse(norm):
    d = ssm.NormDims.make("f32", "bf16", 2, 32, **norm)
    with pytest.raises(ssm.SSMError):
        decoder.RecurrentDecoder(D, None, norm=decoder.GatedNorm(d, None))
    with pytest.raises(ssm.SSMError):
        decoder.WindowedDecoder(D, None, read="full", norm=decoder.GatedNorm(d, None))
    decoder.RecurrentDecoder(D, None, norm=decoder.GatedNorm(NORM, None))


@pytest.mark.parametrize("which", ["recurrent", "windowed"])
def test_steps_on_another_device_than_the_current_one(which, monkeypatch):
    """Every call of a step is made with the state's device current, and the old one is back afterwards."""
    now, calls = [0], []

    class On:
        def __init__(self, x):
            self.to = x.get_device()

        def __enter__(self):
            self.back, now[0] = now[0], self.to

        def __exit__(self, *_):
            now[0] = self.back

    def note(name, result=None):
        return lambda *a, **kw: (calls.append((name, now[0])), result)[1]

    monkeypatch.setattr(decoder.torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(decoder.torch.cuda, "device_of", On)
    for name in ("recurrent_decode_step", "full_read_decode_step", "window_update_refresh"):
        monkeypatch.setattr(decoder, name, note(name))
    cls = decoder.RecurrentDecoder if which == "recurrent" else decoder.WindowedDecoder
    dec = cls.__new__(cls)
    x = torch.zeros(2, 64)
    conv = type("Conv", (), {"state": Stub(7 * MB, (2, 3, 192), torch.bfloat16, 1), "step": note("conv", (x, x, x))})

    class Norm(decoder.GatedNorm):
        __call__ = note("norm", x)

    dec.__dict__.update(d=D, conv=conv, norm=Norm(NORM, Stub(4 * MB, (32,), device=1)), read="full", fused=True, tau=3,
                        state=Stub(5 * MB, (2, 2, 32, 32), device=1), sketch=None, basis=None, read_map=None,
                        offsets=None, k_buf=None, v_buf=None, decay_buf=None, beta_buf=None, _placed=((), []))
    gate = Stub(3 * MB, (2, 64), torch.bfloat16, 1)
    assert dec.step(x, x, x, Stub(1 * MB, (2, 2), device=1), Stub(2 * MB, (2, 2), device=1), gate=gate) is x
    want = ["conv"] + (["recurrent_decode_step"] if which == "recurrent" else
                       ["full_read_decode_step", "window_update_refresh"]) + ["norm"]
    assert calls == [(name, 1) for name in want] and now == [0]


def test_buffers_that_were_replaced(monkeypatch):
    """What a step must not lie over are the window buffers of now."""
    dec = decoder.WindowedDecoder.__new__(decoder.WindowedDecoder)
    x = torch.zeros(2, 64)
    conv = type("Conv", (), {"state": Stub(7 * MB, (2, 3, 192), torch.bfloat16), "step": lambda *a: (x, x, x)})
    bufs = [Stub((30 + i) * MB, (2, 2, 4, 32)) for i in range(4)]
    monkeypatch.setattr(decoder, "full_read_decode_step", lambda *a, **kw: None)
    monkeypatch.setattr(decoder.torch.cuda, "current_device", lambda: 0)
    dec.__dict__.update(d=D, conv=conv, norm=None, read="full", fused=True, tau=0, state=Stub(5 * MB, (2, 2, 32, 32)),
                        sketch=None, basis=None, read_map=None, offsets=None, k_buf=bufs[0], v_buf=bufs[1],
                        decay_buf=bufs[2], beta_buf=bufs[3], _placed=((), []))
    step = lambda at: dec.step(x, x, x, Stub(at, (2, 2)), Stub(2 * MB, (2, 2)))
    for _ in range(2):
        with pytest.raises(ValueError, match="overlaps"):
            step(31 * MB)
    dec.v_buf = Stub(40 * MB, (2, 2, 4, 32))
    step(31 * MB)
    with pytest.raises(ValueError, match="overlaps"):
        step(40 * MB)
