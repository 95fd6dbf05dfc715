"""Every launch shape of the scan's passes: all d_k and d_v, both input types and both directions, on
either side of the numbers of column blocks (sequences x heads x d_v / 16) at which the shape may
change, 256 and 512, with the same bits from run to run. Tolerances as in test_scan_gpu.py."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_scan_gpu import RULES, Batch, check_backward, check_forward  # noqa: E402

pytestmark = pytest.mark.gpu
SIZES = (16, 32, 64, 128)


def sampled(b, heads):
    """The batch's heads `heads` (host checks of all would take minutes)."""
    few = Batch.__new__(Batch)
    few.__dict__.update(b.__dict__, H=len(heads))
    at = torch.tensor(heads, device="cuda")
    pick = lambda x: None if x is None else x.index_select(1, at)
    few.t = {x: pick(t) for x, t in b.t.items()}
    return few, pick


@pytest.mark.parametrize("blocks", [256, 512, 513])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d_v", SIZES)
@pytest.mark.parametrize("d_k", SIZES)
@pytest.mark.parametrize("rule", RULES)
def test_launch_shapes(rule, d_k, d_v, dtype, blocks):
    """`blocks` column blocks, or the next number of them that whole heads give."""
    lens = [70, 3]
    H = -(-blocks // (len(lens) * d_v // 16))
    b = Batch(rule, dtype, lens, H, d_k, d_v, spare=2)
    y, state = b.forward()
    o = b.backward()
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(255)  # NaN in new workspaces
    y2, state2 = b.forward()
    o2 = b.backward()
    assert torch.equal(y, y2) and torch.equal(state, state2)
    assert all(o[x] is None or torch.equal(o[x], o2[x]) for x in o)
    few, pick = sampled(b, sorted({0, H - 1}))
    check_forward(few, pick(y), pick(state))
    check_backward(few, {x: pick(t) for x, t in o.items()})
