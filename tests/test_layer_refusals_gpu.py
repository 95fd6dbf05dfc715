"""What a decoder with a convolution or a norm refuses, it refuses before any of its states has changed: addresses that
the recurrence or the norm cannot read, rows of the gate that it cannot step over, arrays that overlap."""
import pytest

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from tests.test_layer_use_gpu import Layer  # noqa: E402

pytestmark = pytest.mark.gpu


def off(x, by=1):
    """x's values `by` elements behind an address that is a multiple of 16 bytes."""
    buf = torch.empty(x.numel() + 64, device="cuda", dtype=x.dtype)
    assert buf.data_ptr() % 16 == 0
    v = buf[by:by + x.numel()].view(x.shape)
    v.copy_(x)
    return v


def strided(x, lead, stride):
    """x [rows][width] as a column range that begins `lead` elements into rows of `stride`."""
    buf = torch.zeros(x.shape[0], stride, device="cuda", dtype=x.dtype)
    v = buf[:, lead:lead + x.shape[1]]
    v.copy_(x)
    return v


class Held:
    """A decoder and copies of all that it keeps."""

    def __init__(self, dec, which):
        self.now = [dec.state] + ([dec.conv.state] if dec.conv else [])
        if which != "recurrent":
            self.now += [dec.k_buf, dec.v_buf, dec.decay_buf] + ([dec.beta_buf] if dec.beta_buf is not None else [])
        self.before = [x.clone() for x in self.now]

    def same(self):
        return all(torch.equal(x, y) for x, y in zip(self.now, self.before))


@pytest.mark.parametrize("with_conv", [True, False])
@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
@pytest.mark.parametrize("rule", ["mamba2", "gdn", "kda"])
def test_steps(rule, which, with_conv):
    l = Layer(rule, "bf16", 2, 2, 32, 32, 2)
    dec = l.decoder(which)
    if not with_conv:
        dec.conv = None
    (q, k, v, decay, beta), z = l.tokens(slice(0, 2))
    if not with_conv:
        q, k, v = (x.reshape(2, 2, 32).contiguous() for x in (q, k, v))
    y = lambda: torch.zeros(2, 2, 32, device="cuda")
    out = "y_full" if which == "full" else "y"
    dec.step(q, k, v, decay, beta, gate=z)
    held = Held(dec, which)
    wide = y()
    bad = [((off(decay), beta), dict(gate=z)),                       # the recurrence's loads
           ((decay, beta), dict(gate=off(z))), ((decay, beta), dict(gate=strided(z, 1, 72))),
           ((decay, beta), dict(gate=strided(z, 0, 76))), ((decay, beta), {"gate": z, out: off(y())}),
           ((decay, beta), {"gate": z, out: dec.state.view(-1)[:128].view(2, 2, 32)})]
    if rule != "kda":
        bad.append(((wide.view(-1)[:4].view(2, 2), beta), {"gate": z, out: wide}))  # the output over decay
    if rule != "mamba2":
        bad.append(((decay, off(beta)), dict(gate=z)))
    for args, kw in bad:
        with pytest.raises((ValueError, ssm.SSMError)):
            dec.step(q, k, v, *args, **kw)
        assert held.same(), (args, kw)
    weight, dec.norm.weight = dec.norm.weight, off(dec.norm.weight)
    with pytest.raises((ValueError, ssm.SSMError)):
        dec.step(q, k, v, decay, beta, gate=z)
    dec.norm.weight = weight
    assert held.same()
    assert dec.step(q, k, v, decay, beta, gate=z, **{out: wide}).shape == (2, 2, 32)


@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
def test_the_gate_is_not_written_before_it_is_read(which):
    l = Layer("gdn", "f32", 2, 2, 32, 32, 2)
    dec = l.decoder(which)
    (q, k, v, decay, beta), z = l.tokens(slice(0, 2))
    z = z.contiguous()
    held = Held(dec, which)
    with pytest.raises(ValueError, match="overlaps"):
        dec.step(q, k, v, decay, beta, gate=z, **{"y_full" if which == "full" else "y": z.view(2, 2, 32)})
    assert held.same()


@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
@pytest.mark.parametrize("rule", ["gdn", "kda"])
def test_prompts(rule, which):
    l = Layer(rule, "bf16", 2, 2, 32, 32, 2)
    dec = l.decoder(which)
    (q, k, v, decay, beta), z = l.tokens(slice(0, 2))
    dec.prefill([1, 1], q, k, v, decay, beta, gate=z)
    held = Held(dec, which)
    bad = [((decay, beta), dict(gate=off(z))), ((decay, beta), dict(gate=strided(z, 1, 72))),
           ((decay, beta), dict(gate=strided(z, 0, 76))), ((decay, beta[:1]), dict(gate=z))]
    if rule == "kda":  # read four channels at a time
        bad.append(((off(decay), beta), dict(gate=z)))
    for args, kw in bad:
        with pytest.raises((ValueError, ssm.SSMError)):
            dec.prefill([1, 1], q, k, v, *args, **kw)
        assert held.same(), kw
    weight, dec.norm.weight = dec.norm.weight, off(dec.norm.weight)
    with pytest.raises((ValueError, ssm.SSMError)):
        dec.prefill([1, 1], q, k, v, decay, beta, gate=z)
    dec.norm.weight = weight
    assert held.same()
    # gates that the recurrence takes as they lie
    want = l.decoder(which)
    got = l.decoder(which)
    args = (off(decay) if rule == "gdn" else decay, off(beta))
    assert torch.equal(want.prefill([1, 1], q, k, v, decay, beta, gate=z),
                       got.prefill([1, 1], q, k, v, *args, gate=strided(z, 8, 96)))
