"""Decoders whose output norm goes over several heads, as a Mamba-2 layer's does: its groups divide a token's channels,
whatever the heads are."""
import numpy as np
import pytest

from tests import layer_reference as ref

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from sketched_recurrent_state_amd.decoder import GatedNorm, RecurrentDecoder, WindowedDecoder  # noqa: E402
from tests.test_layer_gpu import dev, host, near  # noqa: E402
from tests.test_layer_use_gpu import Layer  # noqa: E402

pytestmark = pytest.mark.gpu
H, DV = 4, 32


@pytest.mark.parametrize("which", ["recurrent", "full", "sketch"])
@pytest.mark.parametrize("groups,gate,centred", [(1, "before", False), (2, "before", False), (2, "after", True),
                                                 (8, "after", False), (4, "before", False)])
def test_groups(groups, gate, centred, which):
    """The norm of a decoder is the norm of its outputs, element by element against the definition: the recurrence's
    outputs are the inputs of both, so what is off is the norm's."""
    l = Layer("mamba2", "f32", 2, H, 32, DV, 12)
    width = H * DV // groups
    rng = np.random.default_rng(groups)
    nd = ssm.NormDims.make("f32", "f32", groups, width, gate=gate, centred=centred)
    norm = GatedNorm(nd, dev(1 + 0.2 * rng.standard_normal((groups, width))), dev(rng.standard_normal((groups, width))))
    dec, bare = l.decoder(which), l.decoder(which)
    make = lambda d, n: (RecurrentDecoder(l.d, d.state, conv=d.conv, norm=n) if which == "recurrent" else
                         WindowedDecoder(l.d, d.state, d.basis, read=which, conv=d.conv, norm=n))
    dec, bare = make(dec, norm), make(bare, None)
    got, want, at = [], [], slice(0, 8)
    tokens, z = l.tokens(at)
    got.append(dec.prefill([5, 3], *tokens, gate=z))
    want.append((bare.prefill([5, 3], *tokens), z))
    for t in range(2):
        tokens, z = l.tokens(slice(8 + 2 * t, 10 + 2 * t))
        got.append(dec.step(*tokens, gate=z))
        want.append((bare.step(*tokens), z))
    for o, (y, z) in zip(got, want):
        assert o.shape == y.shape == (y.shape[0], H, DV)
        rows = lambda x: host(x).reshape(-1, groups, width)
        n, bound = ref.norm(rows(y), rows(z.contiguous()), host(norm.weight), host(norm.bias), gate=gate, centred=centred,
                            eps=float(np.float32(1e-5)))
        near(o, n["out"].reshape(o.shape), bound["out"].reshape(o.shape), "out")


def test_other_widths_are_refused():
    l = Layer("mamba2", "bf16", 2, H, 32, DV, 2)
    for groups, width, x in ((1, 64, "f32"), (4, 64, "f32"), (2, 32, "f32"), (1, H * DV, "bf16")):
        with pytest.raises(ValueError, match="outputs"):
            RecurrentDecoder(l.d, l.state, norm=GatedNorm(ssm.NormDims.make(x, "bf16", groups, width), l.nw))
