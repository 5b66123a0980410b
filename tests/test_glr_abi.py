"""The C entry points of the gated recurrence, layer norm and rotary positions on the CPU: bad
arguments are rejected before any CUDA call, calls without work return GDN_OK, and the workspace
sizes follow their layout."""
import pytest
from test_layer_abi import at


@pytest.fixture(scope="module")
def lib():
    from linear_attention_prefill_gb300 import _build, binding
    _build.build()
    return binding.load_library()


GLR = dict(x=at(0), g=at(1), rate=None, h0=at(3), y=at(4), hT=at(5), states=at(6), N=1, T=100, D=16, xs=16, gs=16,
           gate=0, norm=0, cu=None)


def glr(lib, f32=False, **kw):
    a = dict(GLR, **kw)
    return (lib.gdn_glr_chunk_fwd_f32 if f32 else lib.gdn_glr_chunk_fwd)(*a.values(), None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(g=None), 1), (dict(y=None), 1), (dict(N=-1), 1), (dict(T=-1), 1), (dict(D=0), 1),
    (dict(D=2 ** 30 + 1, xs=2 ** 31, gs=2 ** 31), 1), (dict(xs=15), 1), (dict(gs=1), 1), (dict(gate=3), 1),
    (dict(gate=-1), 1), (dict(norm=3), 1), (dict(norm=-1), 1), (dict(gate=2), 1), (dict(rate=at(2)), 1),
    (dict(x=at(0, 1)), 1), (dict(g=at(1, 1)), 1), (dict(y=at(4, 1)), 1), (dict(rate=at(2, 2), gate=2), 1),
    (dict(h0=at(3, 2)), 1), (dict(hT=at(5, 1)), 1), (dict(states=at(6, 2)), 1), (dict(cu=at(7, 2)), 1),
    (dict(cu=at(7), N=0), 1), (dict(N=1 << 30, T=1 << 30), 1), (dict(N=2 ** 31 - 1, T=1, D=200, xs=200, gs=200), 1),
    (dict(y=at(0)), 1), (dict(y=at(1, 8)), 1), (dict(hT=at(0)), 1), (dict(states=at(1)), 1), (dict(y=at(3)), 1),
    (dict(hT=at(3, 16)), 1), (dict(states=at(3)), 1), (dict(hT=at(4)), 1), (dict(states=at(5)), 1),
    (dict(states=at(4)), 1), (dict(rate=at(2), gate=2, y=at(2)), 1), (dict(cu=at(5)), 1), (dict(cu=at(6, 4)), 1),
])
def test_glr_rejects(lib, case, status, f32):
    assert glr(lib, f32, **case) == status
    assert lib.gdn_last_error() != b""


def test_glr_without_work(lib):
    assert glr(lib, N=0) == 0 and glr(lib, T=0, hT=None, x=None, g=None, y=None) == 0


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", [dict(x=None), dict(h=None), dict(y=None), dict(N=-1), dict(xs=3), dict(gate=2),
                                  dict(h=at(3, 2)), dict(y=at(3)), dict(y=at(0)), dict(h=at(1)), dict(norm=9),
                                  dict(rate=at(2), gate=2, h=at(2))])
def test_glr_step_rejects(lib, case, f32):
    a = dict(dict(x=at(0), g=at(1), rate=None, h=at(3), y=at(4), N=2, D=16, xs=16, gs=16, gate=0, norm=0), **case)
    fn = lib.gdn_glr_recurrent_step_f32 if f32 else lib.gdn_glr_recurrent_step
    assert fn(*a.values(), None) == 1
    assert fn(None, None, None, None, None, 0, 16, 16, 16, 0, 0, None) == 0


BWD = dict(dy=at(0), x=at(1), g=at(2), rate=at(3), h0=at(4), states=at(5), dhT=at(6), dx=at(7), dg=at(8), drate=at(9),
           dh0=at(10), N=1, T=100, D=16, ds=16, xs=16, gs=16, gate=2, norm=2, cu=None, ws=at(12), nws=1 << 20)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", [
    dict(dy=None), dict(x=None), dict(g=None), dict(states=None), dict(dx=None), dict(dg=None), dict(drate=None),
    dict(rate=None), dict(rate=None, gate=0), dict(gate=0), dict(ds=15), dict(dy=at(0, 1)), dict(dx=at(7, 1)),
    dict(dg=at(8, 1)), dict(drate=at(9, 2)), dict(dh0=at(10, 2)), dict(dhT=at(6, 1)), dict(states=at(5, 2)),
    dict(dx=at(0)), dict(dx=at(1, 16)), dict(dg=at(2)), dict(dg=at(7)), dict(drate=at(3)), dict(dh0=at(6)),
    dict(dh0=at(4)), dict(dh0=at(5)), dict(drate=at(8)), dict(dh0=at(9)), dict(cu=at(10)), dict(ws=at(12, 16)),
    dict(nws=8), dict(N=-1), dict(cu=at(11), N=0),
])
def test_glr_bwd_rejects(lib, case, f32):
    a = dict(BWD, **case)
    fn = lib.gdn_glr_chunk_bwd_f32 if f32 else lib.gdn_glr_chunk_bwd
    assert fn(*a.values(), None) == 1 and lib.gdn_last_error() != b""


def test_workspace_sizes(lib):
    size = lib.gdn_glr_chunk_bwd_workspace_size
    for gate in (0, 1):
        assert size(2, 1000, 64, gate, 0) == 0
    for N, T, D, packed in ((1, 1, 64, 0), (3, 700, 100, 0), (8, 2048, 2560, 0), (5, 10007, 1111, 1), (1000, 3, 5000, 0)):
        got, rows = size(N, T, D, 2, packed), 1 if packed else N
        assert got in [4 * rows * k * D for k in range(1, 17)]  # a sum a block of a cluster
    assert size(-1, 4, 4, 2, 0) == size(1, -4, 4, 2, 0) == size(1, 4, 0, 2, 0) == size(0, 4, 4, 2, 1) == 0
    assert size(1, 4, 4, 5, 0) == 0 and size(0, 0, 4, 2, 0) == 0
    size = lib.gdn_layer_norm_bwd_workspace_size
    assert size(3, 100) == 3 * 2 * 100 * 4 and size(0, 100) == 0 and size(-1, 100) == 0 and size(1, 32769) == 0
    assert size(10 ** 6, 100) == 8 * 152 * 2 * 100 * 4 and size(10 ** 6, 5120) == 2 * 152 * 2 * 5120 * 4


LN = dict(x=at(0), w=at(1), b=at(2), res=None, y=at(4), out=None, rows=4, D=64, xs=64, eps=1e-5)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(D=32769, xs=32769), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(xs=63), 1), (dict(res=at(3)), 1), (dict(out=at(3)), 1),
    (dict(x=at(0, 1)), 1), (dict(w=at(1, 2)), 1), (dict(b=at(2, 1)), 1), (dict(y=at(4, 1)), 1), (dict(y=at(0)), 1),
    (dict(y=at(1)), 1), (dict(y=at(2, 8)), 1), (dict(res=at(3), out=at(0)), 1), (dict(res=at(3), out=at(3, 16)), 1),
    (dict(res=at(3), out=at(4)), 1), (dict(res=at(4), out=at(4)), 1), (dict(res=at(3, 1), out=at(5)), 1),
    (dict(rows=1 << 32), 1),
])
def test_layer_norm_rejects(lib, case, status, f32):
    a = dict(LN, **case)
    assert (lib.gdn_layer_norm_fwd_f32 if f32 else lib.gdn_layer_norm_fwd)(*a.values(), None) == status
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(dy=None), 1), (dict(x=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(db=None), 1), (dict(ds=3), 1),
    (dict(xs=63), 1), (dict(D=40000, ds=40000, xs=40000), 2), (dict(eps=-1.0), 1), (dict(dx=at(0)), 1), (dict(dx=at(1)), 1),
    (dict(dw=at(2)), 1), (dict(db=at(5)), 1), (dict(dres=at(4, 16)), 1), (dict(dw=at(3)), 1), (dict(dw=at(6)), 1),
    (dict(ws=at(12, 4)), 1), (dict(nws=100), 1), (dict(dw=at(5, 2)), 1), (dict(dx=at(4, 1)), 1),
])
def test_layer_norm_bwd_rejects(lib, case, status, f32):
    a = dict(dict(dy=at(0), x=at(1), w=at(2), dres=at(3), dx=at(4), dw=at(5), db=at(6), rows=4, D=64, ds=64, xs=64, eps=1e-5,
                  ws=at(12), nws=1 << 20), **case)
    assert (lib.gdn_layer_norm_bwd_f32 if f32 else lib.gdn_layer_norm_bwd)(*a.values(), None) == status
    assert lib.gdn_last_error() != b""


def test_layer_norm_without_work(lib):
    assert lib.gdn_layer_norm_fwd(None, None, None, None, None, None, 0, 64, 64, 1e-5, None) == 0
    assert lib.gdn_layer_norm_bwd(None, None, None, None, None, None, None, 0, 64, 64, 64, 1e-5, None, 0, None) == 0


ROT = dict(q=at(0), k=at(1), turns=at(2), positions=None, offsets=None, cu=None, qo=at(6), ko=at(7), N=2, T=5, Hq=4, Hk=2,
           D=16, R=8, qs=64, ks=32, qos=64, kos=32, inter=0, mag=1.0)


@pytest.mark.parametrize("name", ["gdn_rotary_fwd", "gdn_rotary_fwd_f32", "gdn_rotary_bwd", "gdn_rotary_bwd_f32"])
@pytest.mark.parametrize("case,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(turns=None), 1), (dict(N=-1), 1),
    (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(Hk=0), 1), (dict(R=7), 1), (dict(R=0), 1), (dict(R=18), 1),
    (dict(D=1025, R=8), 2), (dict(D=0), 1), (dict(qs=63), 1), (dict(ks=31), 1), (dict(qos=3), 1), (dict(kos=0), 1),
    (dict(q=at(0, 1)), 1), (dict(ko=at(7, 1)), 1), (dict(turns=at(2, 4)), 1), (dict(positions=at(3, 2)), 1),
    (dict(offsets=at(4, 1)), 1), (dict(cu=at(5, 2)), 1), (dict(positions=at(3), offsets=at(4)), 1),
    (dict(positions=at(3), cu=at(5)), 1), (dict(qo=at(0, 8)), 1), (dict(qo=at(0), qos=128), 1), (dict(qo=at(1)), 1),
    (dict(ko=at(0)), 1), (dict(ko=at(6)), 1), (dict(qo=at(2)), 1), (dict(ko=at(3), positions=at(3)), 1),
    (dict(Hq=2 ** 30), 1), (dict(N=2 ** 20, T=2 ** 20), 1), (dict(cu=at(5), N=0), 1),
])
def test_rotary_rejects(lib, name, case, status):
    a = dict(ROT, **case)
    assert getattr(lib, name)(*a.values(), None) == status
    assert lib.gdn_last_error() != b""


def test_rotary_without_work(lib):
    assert lib.gdn_rotary_fwd(*dict(ROT, T=0, q=None, k=None, qo=None, ko=None, turns=None).values(), None) == 0


def test_binding_refuses_what_is_not_on_a_gpu(lib):
    import torch

    import linear_attention_prefill_gb300 as lap
    x, h, st = torch.zeros(1, 4, 8), torch.zeros(1, 8), torch.zeros(1, 1, 8)
    turns, _ = lap.gdn_rotary_turns(8, device="cpu")
    for call in (lambda **k: lap.gdn_glr_chunk_fwd(x, x, **k), lambda **k: lap.gdn_glr_recurrent_step(x[:, 0], x[:, 0], h, **k),
                 lambda **k: lap.gdn_glr_chunk_bwd(x, x, x, st, **k), lambda **k: lap.gdn_layer_norm_fwd(x, **k),
                 lambda **k: lap.gdn_layer_norm_bwd(x, x, **k),
                 lambda **k: lap.gdn_rotary_fwd(x[:, :, None], None, turns, **k),
                 lambda **k: lap.gdn_rotary_bwd(x[:, :, None], None, turns, **k)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(ValueError, match="CUDA"):
            call(stream=1)


def test_gradient_formula_against_autograd_and_differences():
    """The formula that the GPU's gradient is held against, on the CPU in 64 bits."""
    import torch
    from glr_ref import backward, forward
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    spans, D = [(0, 0, 5), (0, 5, 5), (0, 5, 14)], 3
    for gate in ("log", "sigmoid", "rate"):
        for norm in (None, "linear", "sqrt"):
            z = dict(x=rand(1, 14, D), g=-rand(1, 14, D).abs() - 0.1 if gate == "log" else rand(1, 14, D),
                     rate=-rand(D).abs() if gate == "rate" else None, h0=rand(3, D))
            dy, dhT = rand(1, 14, D), rand(3, D)

            def loss(v):
                y, _, hT, *_ = forward(v["x"], v["g"], v["rate"], v["h0"], gate, norm, spans)
                return (y * dy).sum() + (hT * dhT).sum()

            got = backward(dy, z["x"], z["g"], z["rate"], z["h0"], dhT, gate, norm, spans)
            for k, w in zip(("x", "g", "rate", "h0"), got):
                if z[k] is None:
                    continue
                step = rand(*z[k].shape)
                eps = 1e-5
                up, down = loss(dict(z, **{k: z[k] + eps * step})), loss(dict(z, **{k: z[k] - eps * step}))
                # the difference's own error: eps^2 times a third derivative, 2^-52 of the loss / eps
                assert abs((up - down) / (2 * eps) - (w[0] * step).sum()) <= 1e-7
