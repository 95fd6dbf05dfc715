"""The scan's fp32 values through the bf16 matrix cores: a value cut into three parts keeps all 24
bits, whichever operand it is.

Exact cases have one product different from zero in every sum, by 1, or two of opposite value, so
the result is the operand itself or zero, without a tolerance: a lost part of 8 bits would be off
by 2^-16 of the value or more.

Single products of two values of 24 bits: of the nine products of parts, six are taken. The dropped
ones, with |m| < 2^-7 and |l| < 2^-15 of the value's power of two, are below 2 * 2^-22 + 2^-30 of
the product (tests/test_scan_cpu.py has the same in whole numbers); the six are added in at most
five roundings of 2^-24: under 2^-21 + 2^-30 + 5 * 2^-24 < 14 * 2^-24. Without the least of the six
a product would be off by up to 2^-15.
"""
import pytest

torch = pytest.importorskip("torch")

import sketched_recurrent_state_amd as ssm  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
RULES = ("mamba2", "gdn", "kda")
# d_k, d_v, heads: few column blocks (rows divided over waves) and many (a wave a block)
SHAPES = [(16, 16, 2), (32, 64, 2), (64, 64, 3), (128, 128, 2), (128, 128, 70), (64, 32, 300), (16, 64, 130)]


class Layer:
    """One sequence of T tokens: keys, queries and values of zero, gates of one, beta of one."""

    def __init__(self, rule, dtype, dk, dv, H, T, seed=0):
        self.rule, self.dtype, self.dk, self.dv, self.H, self.T = rule, dtype, dk, dv, H, T
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tin = torch.bfloat16 if dtype == "bf16" else torch.float32
        zero = lambda n: torch.zeros(T, H, n, device="cuda", dtype=self.tin)
        self.q, self.k, self.v = zero(dk), zero(dk), zero(dv)
        self.decay = torch.ones((T, H, dk) if rule == "kda" else (T, H), device="cuda")
        self.beta = None if rule == "mamba2" else torch.ones(T, H, device="cuda")
        self.state = torch.zeros(1, H, dk, dv, device="cuda")
        self.dy = torch.zeros(T, H, dv, device="cuda")
        self.dstate = torch.zeros(1, H, dk, dv, device="cuda")
        self.d = ssm.Dims.make(rule, dtype, 1, H, dk, dv, 4, 4)
        self.plan = torch.empty(ssm.scan_sizes(self.d, T)[0], dtype=torch.int32, device="cuda")
        ssm.scan_plan(torch.tensor([T], dtype=torch.int32, device="cuda"), T, self.plan)

    def full(self, *shape):
        """Random values with all 24 bits in use, of either sign."""
        x = torch.randn(*shape, device="cuda", generator=self.gen)
        return (x.view(torch.int32) | 1).view(torch.float32)

    def args(self):
        return self.d, self.T, self.plan, self.q, self.k, self.v, self.decay, self.beta

    def forward(self):
        y, s = torch.empty(self.T, self.H, self.dv, device="cuda"), torch.empty_like(self.state)
        ssm.scan_forward(*self.args(), s, y, state_in=self.state)
        return y, s[0]

    def backward(self):
        o = {"dq": torch.empty_like(self.q), "dk": torch.empty_like(self.k), "dv": torch.empty_like(self.v),
             "dlog": torch.empty_like(self.decay), "dbeta": None if self.beta is None else torch.empty_like(self.beta),
             "dS": torch.empty_like(self.state)}
        ssm.scan_backward(*self.args(), self.dy, o["dq"], o["dk"], o["dv"], o["dlog"], o["dbeta"],
                          state_in=self.state, dstate=self.dstate, dstate_in=o["dS"])
        o["dS"] = o["dS"][0]
        return o


def places(T, n):
    """A channel for every token, each of them named when there are tokens enough."""
    return (torch.arange(T, device="cuda") * 7 + 3) % n


def cases(f):
    for name, values in (("shape", SHAPES), ("dtype", ["bf16", "f32"]), ("rule", RULES)):
        f = pytest.mark.parametrize(name, values, ids=str)(f)
    return f


@cases
def test_state_read_and_kept(rule, dtype, shape):
    dk, dv, H = shape
    x = Layer(rule, dtype, dk, dv, H, 37)
    x.state = x.full(1, H, dk, dv)
    at = places(37, dk)
    x.q[torch.arange(37), :, at] = 1
    y, s = x.forward()
    assert torch.equal(y, x.state[0][:, at].transpose(0, 1))
    assert torch.equal(s, x.state[0])


@cases
def test_write_and_read_within_a_block(rule, dtype, shape):
    """y = P w and S' = (O k)^T w with one writer: the value, and a gate of 24 bits, come back whole."""
    dk, dv, H = shape
    x = Layer(rule, dtype, dk, dv, H, 19)
    c, z = dk - 3, 2
    x.k[z, :, c] = 1
    x.v[z] = x.full(H, dv).to(x.tin)
    x.q[:, :, c] = 1
    y, s = x.forward()
    assert (y[:z] == 0).all() and torch.equal(y[z:], x.v[z].float().expand(17, H, dv))
    assert torch.equal(s[:, c], x.v[z].float()) and s.count_nonzero() == x.v[z].count_nonzero()
    x.v[z] = 1
    gate = torch.rand(H, dk if rule == "kda" else 1, device="cuda", generator=x.gen)
    x.decay[z + 1] = gate if rule == "kda" else gate[:, 0]
    y, s = x.forward()
    want = gate[:, c if rule == "kda" else 0, None].expand(H, dv)
    assert torch.equal(y[z + 1:], want.expand(16, H, dv)) and torch.equal(s[:, c], want)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule", ["gdn", "kda"])
def test_delta_rule_erases(rule, dtype, shape):
    """With beta = 1 and a value of zero a key's row leaves the state exactly: r = -(D S)^T k has
    all of its 24 bits, through the product with the inverse and the write."""
    dk, dv, H = shape
    x = Layer(rule, dtype, dk, dv, H, 21)
    x.state = x.full(1, H, dk, dv)
    c, z = 5, 18
    x.k[z, :, c] = 1
    x.q[:, :, c] = 1
    y, s = x.forward()
    assert torch.equal(y[:z], x.state[0][:, c].expand(z, H, dv)) and (y[z:] == 0).all()
    assert (s[:, c] == 0).all()
    rest = [i for i in range(dk) if i != c]
    assert torch.equal(s[:, rest], x.state[0][:, rest])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule", RULES)
def test_fp32_keys_and_queries(rule, shape):
    dk, dv, H = shape
    x = Layer(rule, "f32", dk, dv, H, 40)
    at = places(40, dk)
    x.state += 1.0
    value = x.full(40, H)
    x.q[torch.arange(40), :, at] = value
    y, _ = x.forward()
    assert torch.equal(y, value[..., None].expand(40, H, dv))
    x.state.zero_()
    x.q.zero_()
    z, c = 7, dk - 1
    x.k[z, :, c] = value[0]
    x.v[z] = 1
    x.q[z + 1:, :, c] = 1
    y, s = x.forward()
    assert torch.equal(s[:, c], value[0][:, None].expand(H, dv))
    assert torch.equal(y[z + 1:], value[0][:, None].expand(39 - z, H, dv))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule,dtype", [("mamba2", "f32"), ("gdn", "f32"), ("kda", "f32"), ("kda", "bf16")])
def test_products_of_two_full_values(rule, dtype, shape):
    """q S with one channel: queries of 24 bits (fp32, or KDA's decayed by a gate of 24 bits; with
    scalar gates bf16 ones are exact operands)."""
    dk, dv, H = shape
    x = Layer(rule, dtype, dk, dv, H, 33)
    x.state = x.full(1, H, dk, dv)
    at = places(33, dk)
    if dtype == "f32":
        value = x.full(33, H)
        x.q[torch.arange(33), :, at] = value
        value = value.double()
    else:
        gate = 0.5 + torch.rand(H, dk, device="cuda", generator=x.gen) / 2  # of the first token, so of all
        x.decay[0] = gate
        x.q[torch.arange(33), :, at] = 1
        value = gate.double()[:, at].transpose(0, 1)
    y, _ = x.forward()
    want = value[..., None] * x.state[0].double()[:, at].transpose(0, 1)
    err = (y.double() - want).abs() / want.abs()
    # KDA's state after the first block has taken the gate itself: one rounding more
    assert err.max() <= (14 + (rule == "kda")) * U, float(err.max() / U)


@cases
def test_gradients_of_states(rule, dtype, shape):
    """dL/dS passes back whole; q dy^T adds whole values; the values' gradient is a row of it."""
    dk, dv, H = shape
    x = Layer(rule, dtype, dk, dv, H, 35)
    x.dstate = x.full(1, H, dk, dv)
    o = x.backward()
    assert torch.equal(o["dS"], x.dstate[0])
    z, c = 9, dk // 2
    x.dstate.zero_()
    x.q[z, :, c] = 1
    x.dy[z] = x.full(H, dv)
    o = x.backward()
    assert torch.equal(o["dS"][:, c], x.dy[z]) and o["dS"].count_nonzero() == x.dy[z].count_nonzero()
    x.q.zero_()
    x.dy.zero_()
    x.dstate = x.full(1, H, dk, dv)
    x.k[z, :, c] = 1
    o = x.backward()
    assert torch.equal(o["dv"][z], x.dstate[0][:, c].to(x.tin))
    if rule != "mamba2":  # dL/dS0 = G - k (beta k^T G): the key's row leaves exactly
        assert (o["dS"][:, c] == 0).all()
        col = dv - 2
        x.v[z, :, col] = 1
        assert torch.equal(x.backward()["dbeta"][z], x.dstate[0][:, c, col])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule", RULES)
def test_fp32_gradients_of_tokens(rule, shape):
    """dq = S dy, the writer's dk = G w, and dP's and dK's pairs, with one product each."""
    dk, dv, H = shape
    x = Layer(rule, "f32", dk, dv, H, 80)
    col = dv // 2
    x.state = x.full(1, H, dk, dv)
    x.dy[:, :, col] = 1
    o = x.backward()
    assert torch.equal(o["dq"], x.state[0][:, :, col].expand(80, H, dk))
    x.state.zero_()
    x.dstate = x.full(1, H, dk, dv)
    x.dy.zero_()
    x.v[:, :, col] = 1
    assert torch.equal(x.backward()["dk"], x.dstate[0][:, :, col].expand(80, H, dk))
    # dq_i = (dy_i . w_j) k_j for one writer j: in its block, in a later one, in the next chunk
    x.dstate.zero_()
    x.v.zero_()
    c, z = dk - 4, 3
    value = x.full(80, H)
    x.k[z, :, c] = 1
    x.v[z, :, col] = 1
    x.dy[:, :, col] = value
    o = x.backward()
    assert torch.equal(o["dq"][z:, :, c], value[z:]) and (o["dq"][:z] == 0).all()
    # the writer's dk_j = sum_i (dy_i . w_j) q_i for one reader i
    for i in (z + 1, 20, 70):
        x.dy.zero_()
        x.q.zero_()
        x.dy[i, :, col] = value[i]
        x.q[i, :, c - 1] = 1
        got = x.backward()["dk"][z]
        assert torch.equal(got[:, c - 1], value[i]) and (got[:, [j for j in range(dk) if j != c - 1]] == 0).all()
