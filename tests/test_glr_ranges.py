"""GPU tests of the gated linear recurrence where products of decays leave fp32's range: states as large
as fp32 holds them, over stretches whose decays' product is far below 2^-126."""
import pytest
import torch
from glr_ref import backward, forward
from test_glr import DT, assert_within, gen_of, inputs, randn, run_bwd, run_fwd, spans_of

pytestmark = pytest.mark.gpu

# tokens of one row or packed sequences, channels: one block a row, clusters of blocks, odd rows, borders
SHAPES = [((32,), False, 8), ((200, 200), False, 64), ((1500,), False, 64), ((600, 600), False, 33),
          ((37, 0, 150, 1, 400), True, 64), ((1100, 90), True, 31)]


def case(lens, packed, D, dt, gate, large):
    """Every second channel starts (and, backwards, ends) in a large state, half of those without any input;
    each channel's gate stays where products of 16, 64 or some hundred decays underflow."""
    z, cu = inputs(lens, packed, D, dt, gate, True)
    log = torch.tensor([-3.0, -0.3, -9.0, -30.0, -0.05, -1.5, -5.5], device="cuda")
    log = log[torch.arange(D, device="cuda") // 4 % 7] * (0.9 + 0.2 * torch.rand(D, generator=gen_of(9), device="cuda"))
    if gate == "log":
        z["g"][:] = log.to(dt)
    elif gate == "sigmoid":  # log sigmoid(g)
        z["g"][:] = -torch.log(torch.expm1(-log)).to(dt)
    else:
        z["rate"][:] = 2 * log
        z["g"][:] = 0
    sign = torch.where(randn(gen_of(3), D) < 0, -1.0, 1.0)
    some = torch.arange(D, device="cuda") % 2 == 0
    none = torch.arange(D, device="cuda") % 4 == 0
    z["x"][..., none] = 0
    z["h0"] = torch.where(some, large * sign, z["h0"])
    return z, cu, some, none


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", [("log", None), ("sigmoid", "linear"), ("rate", "sqrt")])
@pytest.mark.parametrize("lens,packed,D", SHAPES)
def test_large_states_decay_as_token_by_token(cuda_lib, dtype, gate, norm, lens, packed, D):
    z, cu, _, _ = case(lens, packed, D, DT[dtype], gate, 3e38)
    y, hT, states = run_fwd(cuda_lib, z, cu, gate, norm, output_states=True)
    ry, ey, rh, eh, *_ = forward(z["x"], z["g"], z["rate"], z["h0"], gate, norm, spans_of(lens, packed))
    assert_within(y, ry, ey, "y")
    assert_within(hT, rh, eh, "hT")
    for i in range(1, states.shape[1]):
        assert_within(states[:, i], ry[:, 64 * i - 1], ey[:, 64 * i - 1], "states")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", [("log", None), ("sigmoid", "linear"), ("rate", "sqrt")])
@pytest.mark.parametrize("lens,packed,D", SHAPES)
def test_large_gradients_decay_as_token_by_token(cuda_lib, dtype, gate, norm, lens, packed, D):
    # (products of a state and a gradient stay in range: one of them is large in a channel)
    z, cu, some, none = case(lens, packed, D, DT[dtype], gate, 1e35)
    z["dy"][..., none] = 0
    z["dhT"] = torch.where(some, z["dhT"], 1e35 * torch.sign(z["dhT"]))
    z["dy"][..., 1::4] = 0
    _, _, states = run_fwd(cuda_lib, z, cu, gate, norm, output_states=True)
    got = run_bwd(cuda_lib, z, states, cu, gate, norm)
    want = backward(z["dy"], z["x"], z["g"], z["rate"], z["h0"], z["dhT"], gate, norm, spans_of(lens, packed))
    # A gradient m that has decayed below 2^-126 meets a state of 1e35 in dg = m h_{t-1}, and a decayed state such a
    # gradient: numbers with fewer bits, also token by token.  m and h take up to four roundings a token, each off by
    # 2^-150 there, and pass them on undiminished at most: by T 2^-148 both.  The other factor is at most 1.01e35 (its
    # large start, and inputs far below), a rate's gate has a factor of |rate| more, and the rate's gradient sums T.
    T = max(lens)
    off = 2 * T * 2.0 ** -148 * 1.01e35 * (1 + z["rate"].abs().double() if gate == "rate" else 1)
    for a, b, what in zip(got, want, ("dx", "dg", "drate", "dh0")):
        if a is not None:
            more = 0 if what in ("dx", "dh0") else off * (sum(lens) if what == "drate" else 1)
            assert_within(a, b[0], b[1] + more, what)


def test_a_large_state_as_a_prompt_and_by_steps(cuda_lib):
    T, D = 80, 4
    g = torch.full((1, T, D), -3.0, device="cuda")
    x = torch.zeros(1, T, D, device="cuda")
    h = torch.tensor([[3e38, -3e38, 1e36, 1e30]], device="cuda")
    y, hT, _ = cuda_lib.gdn_glr_chunk_fwd(x, g, h0=h)
    steps = [cuda_lib.gdn_glr_recurrent_step(x[:, t], g[:, t], h) for t in range(T)]
    steps = torch.stack(steps, 1)
    # a token is two roundings and a decay that is off by the same amount on both sides.  A product of decays below
    # 2^-234 is held with 2^-149 / 2^108 as its last bit: half of that times a state below 2^128 is 2^-130 a product,
    # and a token has at most two of them
    assert ((y - steps).abs() <= 4 * T * 2.0 ** -24 * steps.abs() + T * 2.0 ** -129).all()
    assert torch.equal(hT, y[:, -1])
