"""GPU tests of the gated linear recurrence on operands at odd places: the same bits as on aligned ones, over
several rounds of a cluster too (the rate's gradient, whose order is the launch's, within its bound)."""
import pytest
import torch
from test_glr import DT, check, inputs, randn, run_bwd, run_fwd, sliced  # noqa: F401

pytestmark = pytest.mark.gpu
SHAPES = [((130,), False), ((2500,), False), ((1400, 1400), False), ((700, 0, 900, 3), True)]


def odd(t):
    """The same values, contiguous, one element into a buffer."""
    if t is None:
        return None
    buffer = torch.full((t.numel() + 2,), float("nan"), dtype=t.dtype, device=t.device)
    v = buffer[1:1 + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def rate_bound(z, grads, other, gate, norm):
    """A thread adds at most every fourth token of its row, then come 4 warps, and the partial sums of rows and blocks
    by 32 warps: at most tokens / 4 + 4 + rows * 16 / 32 + 32 + 1 roundings, of each side."""
    if grads is None:
        assert other is None
        return
    # |d sig| summed: dg = d rate sig (1 - sig), from the fp32 call
    g = z["g"].float()
    size = (z["dg32"].abs() / (z["rate"].abs() * torch.sigmoid(-g))).double().sum((0, 1))
    n = g.shape[0] * g.shape[1] / 4 + g.shape[0] / 2 + 40
    assert ((grads - other).double().abs() <= 2 * n * 2.0 ** -24 * size).all()


def bits(a, b):
    return a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", [("log", None), ("sigmoid", "linear"), ("rate", "sqrt")])
@pytest.mark.parametrize("D", [64, 130, 1111])
@pytest.mark.parametrize("lens,packed", SHAPES)
def test_same_bits_at_odd_places(cuda_lib, dtype, gate, norm, lens, packed, D):
    dt = DT[dtype]
    z, cu = inputs(lens, packed, D, dt, gate, True)
    fwd = run_fwd(cuda_lib, z, cu, gate, norm, output_states=True)
    grads = run_bwd(cuda_lib, z, fwd[2], cu, gate, norm)
    if gate == "rate":
        f = {k: v.float() if k in ("x", "g", "dy") else v for k, v in z.items()}
        st = run_fwd(cuda_lib, f, cu, gate, norm, output_states=True)[2]
        z["dg32"] = run_bwd(cuda_lib, f, st, cu, gate, norm)[1]

    def same(z, states=fwd[2], out=(None,) * 3, back=(None,) * 4):
        y, hT, st = out
        dx, dg, drate, dh0 = back
        again = run_fwd(cuda_lib, z, cu, gate, norm, output_states=True, y=y, hT=hT, states=st)
        assert all(bits(a, b) for a, b in zip(again, fwd))
        for a, b in zip((y, hT, st), again):
            assert a is None or a.data_ptr() == b.data_ptr()
        got = run_bwd(cuda_lib, z, states, cu, gate, norm, dx=dx, dg=dg, drate=drate, dh0=dh0)
        assert all(bits(a, b) for a, b in zip(got[:2] + got[3:], grads[:2] + grads[3:]))
        rate_bound(z, got[2], grads[2], gate, norm)

    # rows of slices, by 16 bytes, 4 bytes and elements
    for shift in (8, 2, 1):
        same(dict(z, **{k: sliced(z[k], shift * (i + 1), 8 - shift) for i, k in enumerate(("x", "g", "dy"))}))
    # aligned rows beside one other operand off its pairs, on the way in and out
    for k in ("h0", "rate", "dhT"):
        if z[k] is not None:
            same(dict(z, **{k: odd(z[k])}))
    same(z, states=odd(fwd[2]))
    for i in range(3):
        same(z, out=tuple(odd(torch.empty_like(t)) if j == i else None for j, t in enumerate(fwd)))
    for i in range(4):
        if grads[i] is not None:
            same(z, back=tuple(odd(torch.empty_like(t)) if j == i else None for j, t in enumerate(grads)))
    # and all together
    same({k: odd(v) if k != "dg32" else v for k, v in z.items()}, odd(fwd[2]),
         tuple(odd(torch.empty_like(t)) for t in fwd),
         tuple(odd(torch.empty_like(t)) if t is not None else None for t in grads))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 130, 1111])
def test_step_at_odd_places(cuda_lib, dtype, D):
    z, _ = inputs((1,) * 5, False, D, DT[dtype], "rate")
    x, g, h = z["x"][:, 0], z["g"][:, 0], z["h0"].clone()
    form = dict(gate="rate", input_norm="sqrt")
    y = cuda_lib.gdn_glr_recurrent_step(x, g, h, z["rate"], **form)
    for which in range(6):
        a, b, r, s, o = (odd(t) if which in (i, 5) else t.clone()
                         for i, t in enumerate((x, g, z["rate"], z["h0"], torch.empty_like(y))))
        again = cuda_lib.gdn_glr_recurrent_step(a, b, s, r, o, **form)
        assert torch.equal(again, y) and torch.equal(s, h)


def one_row(T, D):
    z, _ = inputs((T,), False, D, torch.float32, "rate", False, 3)
    return z


@pytest.mark.parametrize("T,D", [(50, 64), (640, 64), (9000, 64), (3000, 2560)])
def test_rate_gradient_of_long_rows(cuda_lib, T, D):
    """Against a sum in 64 bits of the same fp32 terms: a thread adds every fourth token of its block's share, at most
    T / 4 of them, then 4 warps, 16 blocks and the columns' 32 warps follow."""
    z = one_row(T, D)
    _, _, st = run_fwd(cuda_lib, z, None, "rate", None, output_states=True)
    _, dg, drate, _ = run_bwd(cuda_lib, z, st, None, "rate", None)
    g = z["g"].double()
    # dg = dL rate sig (1 - sig) in fp32: dL sig comes back with the roundings of dg, sig (3 + 2 |g| of e^-g, 3 more)
    # and 1 - sig, four products and the quotient
    term = dg.double() / (z["rate"].double() * torch.sigmoid(-g))
    each = (2 * (3 + 2 * g.abs()) + 16) * 2.0 ** -24
    bound = ((T / 4 + 4 + 16 + 32) * 2.0 ** -24 + each) * term.abs()
    assert ((drate.double() - term.sum((0, 1))).abs() <= bound.sum((0, 1))).all()
