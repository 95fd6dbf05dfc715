"""The scan at sizes whose element offsets pass 2^31 (inputs, outputs, workspace and state pool), with
the most heads that it takes, and with many sequences of one token. Only a sample is checked against
the token-by-token recurrence, with the tolerances of test_scan_gpu.py; inputs are made on the device."""
import pytest

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402
from tests.test_scan_gpu import RULES, U, Batch, check_backward, near, ref  # noqa: E402

pytestmark = pytest.mark.gpu


def made(rule, dtype, lens, H, dk, dv, states=True):
    """A Batch whose inputs are made on the device."""
    gen = torch.Generator(device="cuda").manual_seed(len(lens))
    T, n = sum(lens), len(lens)
    tin = torch.bfloat16 if dtype == "bf16" else torch.float32
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=tin)
    uni = lambda *s: torch.rand(*s, device="cuda", generator=gen)
    b = Batch.__new__(Batch)
    b.rule, b.lens, b.H, b.dk, b.dv, b.n, b.T, b.tin = rule, list(lens), H, dk, dv, n, T, tin
    b.t = {"q": rand(T, H, dk) / dk ** 0.5, "k": rand(T, H, dk) / dk ** 0.5, "v": rand(T, H, dv),
           "decay": 0.85 + 0.149 * uni(*((T, H, dk) if rule == "kda" else (T, H))),
           "beta": None if rule == "mamba2" else uni(T, H) / 2,
           "state_in": torch.randn(n, H, dk, dv, device="cuda", generator=gen) if states else None,
           "dy": None, "dstate": None}
    b.d = ssm.Dims.make(rule, dtype, n, H, dk, dv, 4, 4)
    b.lengths = torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    b.plan = torch.empty(ssm.scan_sizes(b.d, T)[0], dtype=torch.int32, device="cuda")
    ssm.scan_plan(b.lengths, T, b.plan)
    return b


def part(b, seqs, tokens, heads):
    """The sequences `seqs` (whose tokens are `tokens`, all of one slice) and the heads `heads` of b."""
    p = Batch.__new__(Batch)
    p.__dict__.update(b.__dict__, lens=[b.lens[i] for i in seqs], n=len(seqs), H=len(heads))
    p.T = sum(p.lens)
    per_token = lambda x: None if x is None else x[tokens][:, heads]
    per_seq = lambda x: None if x is None else x[seqs][:, heads]
    p.t = {x: (per_seq if x in ("state_in", "dstate") else per_token)(t) for x, t in b.t.items()}
    return p, per_token, per_seq


def check(p, y, state):
    tol = (p.dk + 48) * U
    y, state = y.double().cpu().numpy(), state.double().cpu().numpy()
    for i, s in p.parts():
        wy, ws = ref.forward(*p.seq(i, s))
        near(y[s], wy, tol, "y")
        near(state[i], ws, tol, "state")


@pytest.mark.parametrize("rule", RULES)
def test_offsets_beyond_32_bits(rule):
    """66,000 tokens of 512 heads, 16 x 64: 2.2e9 elements of v, y and dy, and of the workspace; the
    second sequence lies behind all of them."""
    lens, heads = [65930, 70], [0, 511]
    b = made(rule, "bf16", lens, 512, 16, 64, states=False)
    assert b.t["v"].numel() > 2 ** 31
    y = torch.empty(b.T, 512, 64, device="cuda")
    state = torch.empty(2, 512, 16, 64, device="cuda")
    ssm.scan_forward(*b.args(), state, y)
    p, per_token, per_seq = part(b, [1], slice(lens[0], b.T), heads)
    check(p, per_token(y), per_seq(state))
    b.t["dy"] = y.clamp_(-2, 2)
    o = b.backward()
    p, per_token, per_seq = part(b, [1], slice(lens[0], b.T), heads)
    check_backward(p, {x: None if t is None else (per_seq if x == "dS0" else per_token)(t) for x, t in o.items()})


def test_state_pool_beyond_32_bits():
    """Slots of a pool of 2.2e9 elements, continued in place."""
    slots, H = 4200, 32
    b = made("gdn", "bf16", [20, 33], H, 128, 128)
    pool = torch.full((slots, H, 128, 128), 3.0, device="cuda")
    slot = torch.tensor([4199, 4097], dtype=torch.int32, device="cuda")
    assert pool.numel() > 2 ** 31
    pool[slot.long()] = b.t["state_in"]
    y = torch.empty(b.T, H, 128, device="cuda")
    ssm.scan_forward(*b.args(), pool, y, state_in=pool, slot=slot, num_slots=slots)
    p, per_token, per_seq = part(b, [0, 1], slice(None), [0, 31])
    check(p, per_token(y), per_seq(pool[slot.long()]))
    others = torch.ones(slots, dtype=torch.bool, device="cuda")
    others[slot.long()] = False
    assert all((pool[i:i + 100][others[i:i + 100]] == 3).all() for i in range(0, slots, 100))


@pytest.mark.parametrize("rule", RULES)
def test_most_heads(rule):
    """65,536 heads: a block's 16 tokens span 512 MB of fp32 keys."""
    H = 65536
    b = made(rule, "f32", [19], H, 128, 16, states=False)
    heads = [0, 40000, H - 1]
    y, state = torch.empty(b.T, H, 16, device="cuda"), torch.empty(1, H, 128, 16, device="cuda")
    ssm.scan_forward(*b.args(), state, y)
    p, per_token, per_seq = part(b, [0], slice(None), heads)
    check(p, per_token(y), per_seq(state))
    b.t["dy"] = y
    o = b.backward()
    p, per_token, per_seq = part(b, [0], slice(None), heads)
    check_backward(p, {x: None if t is None else (per_seq if x == "dS0" else per_token)(t) for x, t in o.items()})


@pytest.mark.parametrize("rule", RULES)
def test_many_sequences_of_one_token(rule):
    """100,000 sequences of one token, and empty ones between them."""
    n = 100000
    lens = [1, 0, 1, 1] * (n // 4)
    b = made(rule, "bf16", lens, 4, 32, 32)
    y, state = torch.empty(b.T, 4, 32, device="cuda"), torch.empty(n, 4, 32, 32, device="cuda")
    ssm.scan_forward(*b.args(), state, y, state_in=b.t["state_in"])
    assert torch.equal(state[1::4], b.t["state_in"][1::4])
    b.t["dy"], b.t["dstate"] = y, state
    o = b.backward()
    at = [n - 4, n - 3, n - 2, n - 1]
    p, per_token, per_seq = part(b, at, slice(b.T - 3, b.T), [0, 3])
    check(p, per_token(y), per_seq(state))
    check_backward(p, {x: None if t is None else (per_seq if x == "dS0" else per_token)(t) for x, t in o.items()})
