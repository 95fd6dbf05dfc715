"""Selective prompts whose groups of chunks hold several chunks each: states continued in place, and sequences that
begin late in a group, end early in one or go over several.

Tolerances are those of tests/test_layer_gpu.py. A join takes n tokens' decays as one of the sum of their steps, whose n
roundings are n/2 |A sum| u of the decay at most: within the 3 n u that the reference counts for n decays up to |A sum| = 6,
and beyond that less than 0.0075 n u of the state (e^-6 and falling), 1.5 u for the longest group here (192 tokens), where
the reference counts four roundings of the state.
"""
import pytest

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from sketched_recurrent_state_amd.decoder import SelectiveDecoder  # noqa: E402
from tests.test_layer_gpu import FILL, Selective, spans  # noqa: E402
from tests.test_layer_use_gpu import Banded  # noqa: E402

pytestmark = pytest.mark.gpu

# 10,240 waves in all and a table of more than 50 entries: 2 chunks a group, 3 from 200 entries on
BATCHES = {"a chunk then pairs": [64] + [128] * 40,  # each pair is one group's last chunk and the next one's first
           "unlike": [10, 0, 700, 64, 1, 300, 129, 63, 0, 1500, 5, 65, 400, 0],
           "three chunks a group": [200] * 64}
SHAPES = [(16, 8, 1), (32, 16, 2), (16, 32, 1), (32, 64, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("batch", BATCHES)
def test_in_place(batch, shape, dtype):
    s = Selective(dtype, BATCHES[batch], *shape, spare=3)
    out, state = s.forward()
    s.check_forward(out, state)
    for _ in range(3):
        out2, state2 = s.forward(in_place=True)
        assert torch.equal(out, out2) and torch.equal(state, state2)


@pytest.mark.parametrize("lens,ch,N", [([200] * 64, 5120, 16), ([100] * 64, 5120, 64), ([8192], 5120, 16)],
                         ids=["prompts", "64 states", "one prompt"])
def test_in_place_wide(lens, ch, N):
    """Thousands of waves, groups of 9, 21 and 5 chunks: through the call and through the decoder."""
    T, n = sum(lens), len(lens)
    torch.manual_seed(5)
    r = lambda *shape: torch.randn(*shape, device="cuda", dtype=torch.bfloat16)
    x, dt, z, B, C = r(T, ch), r(T, ch), r(T, ch), r(T, N), r(T, N)
    A = -torch.rand(ch, N, device="cuda") - 0.01
    D, bias = torch.randn(ch, device="cuda"), torch.randn(ch, device="cuda") - 5
    h0 = torch.randn(n, ch, N, device="cuda")
    d = ssm.SelectiveDims.make("bf16", n, ch, N)
    plan = torch.empty(2 * (n + 1) + T // 64 + n, dtype=torch.int32, device="cuda")
    ssm.scan_plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), T, plan)
    out, state = torch.full_like(x, FILL), torch.full_like(h0, FILL)
    ssm.selective_forward(d, T, plan, x, dt, A, B, C, state, out, D=D, z=z, dt_bias=bias, state_in=h0)
    for _ in range(3):
        o, h = torch.full_like(x, FILL), h0.clone()
        ssm.selective_forward(d, T, plan, x, dt, A, B, C, h, o, D=D, z=z, dt_bias=bias, state_in=h)
        assert torch.equal(out, o) and torch.equal(state, h)
    dec = SelectiveDecoder(d, h0.clone(), A, D=D, dt_bias=bias)
    assert torch.equal(dec.prefill(lens, x, dt, B, C, z), out) and torch.equal(dec.state, state)
    on = SelectiveDecoder(d, h0.clone(), A, D=D, dt_bias=bias)
    assert torch.equal(on.prefill(torch.tensor(lens, device="cuda"), x, dt, B, C, z), out)
    assert torch.equal(on.state, state)


def test_in_place_pool():
    """Slots in any order, some sequences without one, a workspace of NaN exactly large enough."""
    s = Selective("f32", [64] + [128] * 40, 16, 16)
    out, state = s.forward()
    torch.manual_seed(3)
    slot = torch.randperm(60, device="cuda")[:41].int()
    skipped = [0, 5, 6, 19, 40]
    slot[skipped] = torch.tensor([-1, 60, 61, -7, 2 ** 30], dtype=torch.int32, device="cuda")
    kept = [i for i in range(41) if i not in skipped]
    at = slot[kept].long()
    pool = torch.full((60, s.ch, s.N), FILL, device="cuda")
    pool[at] = s.h0[kept]
    o, need = s.rows(), ssm.selective_sizes(s.d, s.T)[0]
    buf = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), pool, o, **s.more(), state_in=pool, slot=slot, num_slots=60,
                          workspace=buf[4096:4096 + need])
    assert (buf[:4096] == 0xFF).all() and (buf[4096 + need:] == 0xFF).all()
    for i, rows in spans(s.lens):
        assert torch.equal(o[rows], out[rows]) if i in kept else (o[rows] == FILL).all(), i
    assert torch.equal(pool[at], state[kept])
    rest = torch.ones(60, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (pool[rest] == FILL).all()


def test_in_place_without_a_state():
    """No kept state: zeros, whatever the states hold."""
    s = Selective("f32", [64] + [128] * 40, 16, 8, carried=False)
    out, state = s.forward()
    s.h0 = torch.zeros(41, 16, 8, device="cuda")
    out2, state2 = s.forward(in_place=True)
    assert torch.equal(out, out2) and torch.equal(state, state2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("batch", BATCHES)
def test_gradients(batch, shape, dtype):
    """The switch from the sequence that began before a group to later ones, kept states completed over several chunks,
    joins forwards and backwards over such groups."""
    s = Selective(dtype, BATCHES[batch], *shape, spare=3)
    o = s.backward()
    s.check_backward(o)
    again = s.backward()
    assert all(v is None or torch.equal(v, again[k]) for k, v in o.items())


@pytest.mark.parametrize("without", ["gated", "soft", "carried"])
def test_without(without):
    s = Selective("f32", BATCHES["unlike"], 32, 16, 2, **{without: False}, pad=0)
    out, state = s.forward()
    s.check_forward(out, state)
    s.check_backward(s.backward())
    if s.h0 is not None:
        assert all(torch.equal(a, b) for a, b in zip(s.forward(in_place=True), (out, state)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slow_decays(dtype):
    """Decays near 1, so that a state of the first tokens is still there groups later and joins count."""
    s = Selective(dtype, [64, 0, 900, 31] + [300] * 8, 16, 16)
    s.A.mul_(1e-3)
    out, state = s.forward()
    s.check_forward(out, state)
    assert all(torch.equal(a, b) for a, b in zip(s.forward(in_place=True), (out, state)))
    s.check_backward(s.backward())


@pytest.mark.parametrize("index,value", [(1, 0), (1, 5000), (2, 5185), (41, 2 ** 31 - 1), (1, -5), (42 + 1, 2 ** 31 - 1),
                                         (42 + 1, -1), (42 + 5, 0), (42 + 41, 2 ** 31 - 1), (42 + 2, 121), (84 + 2, 40),
                                         (84 + 3, -2 ** 31), (84 + 1, 0), (84 + 121, 40), (0, 64), (30, 60)])
def test_wrong_plans_in_place(index, value):
    s = Selective("bf16", BATCHES["a chunk then pairs"], 16, 16, pad=0)
    s.plan[index] = value
    new = Banded()
    state = new(s.h0)
    state.copy_(s.h0)
    need = torch.empty(ssm.selective_sizes(s.d, s.T)[0], dtype=torch.uint8, device="cuda")
    ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), state, new(s.x), **s.more(), state_in=state, workspace=new(need))
    torch.cuda.synchronize()
    assert new.intact()


def test_captured_in_place():
    """A prompt continued in place in a graph, replayed: each replay goes on from the last one's states."""
    s = Selective("bf16", BATCHES["a chunk then pairs"], 48, 16)
    state, eager = s.h0.clone(), s.h0.clone()
    out, want = s.rows(), s.rows()
    call = lambda h, o: ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), h, o, **s.more(), state_in=h)
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        call(state, out)
    for _ in range(3):
        before = eager.clone()
        graph.replay()
        call(eager, want)
        apart, end = s.rows(), torch.empty_like(before)
        ssm.selective_forward(s.d, s.T, s.plan, *s.inputs(), end, apart, **s.more(), state_in=before)
        torch.randn(1 << 16, device="cuda").sum().item()
        assert torch.equal(out, want) and torch.equal(state, eager)
        assert torch.equal(apart, want) and torch.equal(end, eager)


def test_two_calls_at_once_in_place():
    ss = [Selective("bf16", BATCHES["unlike"], 128, 16, seed=k) for k in range(2)]
    want = [s.forward() for s in ss]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, st in zip(ss, streams):
            with torch.cuda.stream(st):
                got.append(s.forward(in_place=True))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
