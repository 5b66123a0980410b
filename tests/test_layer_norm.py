"""GPU tests of layer norm and its gradient against the definition in 64 bits (glr_ref.py)."""
import pytest
import torch
from glr_ref import ln_backward, ln_forward
from test_glr import DT, assert_within, gen_of, randn, sliced

pytestmark = pytest.mark.gpu
EPS = 1e-5


def inputs(rows, D, dt, seed=0):
    g = gen_of(seed + D)
    lead = rows if isinstance(rows, tuple) else (rows,)
    return dict(x=(randn(g, *lead, D) + randn(g, D)).to(dt), dy=randn(g, *lead, D, dtype=dt),
                w=randn(g, D), b=randn(g, D), res=(2 * randn(g, *lead, D)).to(dt))


def check(lib, z, w, b, res):
    y, out = lib.gdn_layer_norm_fwd(z["x"], w, b, res, eps=EPS)
    ref, err, r, _ = ln_forward(z["x"], w, b, res, EPS)
    assert_within(y, ref, err, "y")
    if res is None:
        assert out is None
    else:
        assert_within(out, r, torch.zeros_like(r) + 2.0 ** -24 * r.abs(), "residual")
    dx, dw, db = lib.gdn_layer_norm_bwd(z["dy"], z["x"], w, res, eps=EPS)
    want = ln_backward(z["dy"], z["x"], w, res, EPS)
    for got, (ref, err), what in ((dx, want[0], "dx"), (dw, want[1], "dweight"), (db, want[2], "dbias")):
        assert_within(got, ref, err, what)
    only, none, none2 = lib.gdn_layer_norm_bwd(z["dy"], z["x"], w, res, eps=EPS, param_grads=False)
    assert none is None and none2 is None and torch.equal(only, dx)
    return y, out, dx, dw, db


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [
    (1, 1), (3, 2), (7, 7), (5, 31), (33, 64), (9, 65), (1000, 72), (3, 128), (70, 200), (2, 250), (17, 512), (5, 509),
    (1, 520), (400, 1111), (16, 2560), (700, 1024), (3, 4096), (5, 4100), (9, 5120), (2, 8192), (3, 8193), (320, 8200),
    (4, 16384), (3, 16390), (2, 32768), ((2, 3), 96),
])
def test_rows(cuda_lib, dtype, rows, D):
    z = inputs(rows, D, DT[dtype])
    out = check(cuda_lib, z, z["w"], z["b"], z["res"])
    check(cuda_lib, z, None, None, None)
    check(cuda_lib, z, z["w"], None, None)
    # slices give the same values; parameters and outputs at odd places too, on narrower accesses
    for shift in (8, 3):
        x, dy = sliced(z["x"], shift, 16 - shift), sliced(z["dy"], 2 * shift, 8)
        y, r = cuda_lib.gdn_layer_norm_fwd(x, z["w"], z["b"], z["res"], eps=EPS)
        dx, dw, db = cuda_lib.gdn_layer_norm_bwd(dy, x, z["w"], z["res"], eps=EPS)
        for a, b in zip((y, r, dx, dw, db), out):
            assert torch.equal(a, b)
    # in place
    res = z["res"].clone()
    y, r = cuda_lib.gdn_layer_norm_fwd(z["x"], z["w"], z["b"], res, residual_out=res, eps=EPS)
    assert r.data_ptr() == res.data_ptr() and torch.equal(r, out[1]) and torch.equal(y, out[0])
    res = z["res"].clone()
    dx, _, _ = cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"], res, dx=res, eps=EPS)
    assert dx.data_ptr() == res.data_ptr() and torch.equal(dx, out[2])


@pytest.mark.parametrize("D", [64, 384, 2560, 9000])
def test_rows_whose_mean_is_large(cuda_lib, D):
    """Their spread keeps its digits: the mean is taken off before the squares."""
    z = inputs(50, D, torch.float32)
    z["x"] = 1000 + z["x"]
    check(cuda_lib, z, z["w"], z["b"], None)


@pytest.mark.parametrize("D", [64, 100, 2560, 9000])
def test_constant_rows_infinities_and_nan(cuda_lib, D):
    z = inputs(40, D, torch.float32)
    clean = cuda_lib.gdn_layer_norm_fwd(z["x"], z["w"], z["b"])[0]
    cleang = cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"])
    z["x"][3], z["x"][7, 5], z["x"][9, 6] = 4.0, float("nan"), float("inf")
    y = cuda_lib.gdn_layer_norm_fwd(z["x"], z["w"], z["b"])[0]
    dx, _, db = cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"])
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 7, 9]] = False
    assert torch.equal(y[keep], clean[keep]) and torch.equal(dx[keep], cleang[0][keep])
    assert torch.equal(y[3], z["b"]) and torch.isnan(y[7]).all() and torch.isnan(y[9]).all()
    assert torch.isfinite(dx[3]).all() and torch.isnan(dx[7]).all() and torch.equal(db, cleang[2])
    assert torch.isnan(cuda_lib.gdn_layer_norm_fwd(z["x"][3:4], eps=0.0)[0]).all()  # 0 / 0, as the formula


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(5000, 48), (9000, 256), (2600, 2560), (1500, 6000), (700, 12000)])
def test_many_rows(cuda_lib, dtype, rows, D):
    z = inputs(rows, D, DT[dtype])
    check(cuda_lib, z, z["w"], z["b"], z["res"])


def test_bits_on_streams_graphs_and_workspaces(cuda_lib):
    zs = [inputs(900, 1280, torch.bfloat16, s) for s in (1, 2)]
    both = lambda z, **k: cuda_lib.gdn_layer_norm_fwd(z["x"], z["w"], z["b"], z["res"], **k) \
        + cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"], z["res"], **k)  # noqa: E731
    want = [both(z) for z in zs]
    torch.cuda.synchronize()
    graphs, outs, sides = [], [], [torch.cuda.Stream() for _ in zs]
    for z in zs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(z))
        graphs.append(graph)
    for _ in range(4):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    other = [both(z, stream=s) for z, s in zip(zs, sides)]
    torch.cuda.synchronize()
    for w, o, s in zip(want, outs, other):
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w, o, s))
    z, need = zs[0], cuda_lib.gdn_layer_norm_bwd_workspace_size(900, 1280)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    got = cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"], z["res"], workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0][2:]))


def test_empty_and_far(cuda_lib):
    none, w = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(16, device="cuda")
    assert cuda_lib.gdn_layer_norm_fwd(none, w, w)[0].numel() == 0
    dx, dw, db = cuda_lib.gdn_layer_norm_bwd(none, none, w)
    assert dx.numel() == 0 and (dw == 0).all() and (db == 0).all()
    D, rows = 32768, 66000  # more than 2^31 elements
    z = inputs(3, D, torch.bfloat16)
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    x[-3:] = z["x"]
    y = cuda_lib.gdn_layer_norm_fwd(x, z["w"], z["b"])[0]
    ref, err, _, _ = ln_forward(z["x"], z["w"], z["b"], None, EPS)
    assert_within(y[-3:], ref, err, "y")
    y[:] = 0
    y[-3:] = z["dy"]
    dx, dw, db = cuda_lib.gdn_layer_norm_bwd(y, x, z["w"])
    want = ln_backward(z["dy"], z["x"], z["w"], None, EPS)
    assert_within(dx[-3:], *want[0], "dx")
    assert_within(dw, *want[1], "dweight")
    assert_within(db, *want[2], "dbias")


def test_binding_refusals(cuda_lib):
    dev, bf = "cuda", torch.bfloat16
    x, w = torch.zeros(4, 16, dtype=bf, device=dev), torch.ones(16, device=dev)
    fwd, bwd, err = cuda_lib.gdn_layer_norm_fwd, cuda_lib.gdn_layer_norm_bwd, cuda_lib.GdnError
    for bad, fn in [
        (TypeError, lambda: fwd(x.half(), w)), (TypeError, lambda: fwd(x, w.to(bf))), (ValueError, lambda: fwd(x, w[:8])),
        (ValueError, lambda: fwd(x.cpu(), w)), (TypeError, lambda: fwd(x, w, w, x.float())), (err, lambda: fwd(x, w, y=x)),
        (ValueError, lambda: fwd(x, w, residual_out=x.clone())), (err, lambda: fwd(x, w, eps=-1.0)),
        (err, lambda: fwd(torch.zeros(1, 40000, device=dev))), (ValueError, lambda: fwd(x[:, ::2])),
        (ValueError, lambda: bwd(x[:2], x)), (err, lambda: bwd(x, x.clone(), w, dx=x)), (err, lambda: bwd(x, x, w, dweight=w)),
        (ValueError, lambda: bwd(x, x, w, dweight=torch.ones_like(w), param_grads=False)),
        (err, lambda: bwd(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device=dev))),
    ]:
        with pytest.raises(bad):
            fn()
