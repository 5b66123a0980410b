"""GPU tests of the gated linear recurrence, its step and its gradient against the definition in 64
bits, with bounds carried through the arithmetic (glr_ref.py)."""
import numpy as np
import pytest
import torch
from glr_ref import backward, forward

from linear_attention_prefill_gb300.workloads import cu_seqlens_of

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMS = [(g, n) for g in ("log", "sigmoid", "rate") for n in (None, "linear", "sqrt")]


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def sliced(t, before=0, after=0):
    """The same values as a slice of a wider row (``before``/``after`` extra columns of NaN)."""
    wide = torch.full(t.shape[:-1] + (before + t.shape[-1] + after,), float("nan"), dtype=t.dtype,
                      device=t.device)
    wide[..., before:before + t.shape[-1]] = t
    return wide[..., before:before + t.shape[-1]]


def assert_within(got, ref, err, what):
    """|got - ref| <= err + half a step of the storage type at |ref| + err."""
    f = torch.finfo(got.dtype)
    bound = err + f.eps / 2 * (ref.abs() + err) + f.tiny
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst " \
                          f"{(d / bound).nan_to_num(float('inf')).max().item():.3g} of the bound"


def spans_of(lens, packed):
    if packed:
        cu = np.concatenate([[0], np.cumsum(lens)])
        return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]
    return [(b, 0, lens[0]) for b in range(len(lens))]


def inputs(lens, packed, D, dt, gate, state=True, seed=0):
    g = gen_of(seed + D)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    # decays from 0.1 to 0.9999
    raw = randn(g, *lead, D)
    z = dict(x=randn(g, *lead, D, dtype=dt), dy=randn(g, *lead, D, dtype=dt),
             g=(-torch.exp(2 * raw - 3) if gate == "log" else 2 * raw + 1).to(dt),
             rate=-torch.exp(randn(g, D) - 1) if gate == "rate" else None,
             h0=randn(g, len(lens), D) if state else None, dhT=randn(g, len(lens), D) if state else None)
    return z, torch.from_numpy(cu_seqlens_of(lens)).cuda() if packed else None


def run_fwd(lib, z, cu, gate, norm, **kw):
    return lib.gdn_glr_chunk_fwd(z["x"], z["g"], z["rate"], z["h0"], gate=gate, input_norm=norm, cu_seqlens=cu, **kw)


def run_bwd(lib, z, states, cu, gate, norm, **kw):
    return lib.gdn_glr_chunk_bwd(z["dy"], z["x"], z["g"], states, z["rate"], z["h0"], z["dhT"], gate=gate,
                                 input_norm=norm, cu_seqlens=cu, **kw)


def check(lib, lens, packed, D, dt, gate, norm, state, seed=0):
    z, cu = inputs(lens, packed, D, dt, gate, state, seed)
    spans = spans_of(lens, packed)
    y, hT, states = run_fwd(lib, z, cu, gate, norm, output_states=True)
    ry, ey, rh, eh, hp, ep, _ = forward(z["x"], z["g"], z["rate"], z["h0"], gate, norm, spans)
    assert_within(y, ry, ey, "y")
    assert_within(hT, rh, eh, "hT")
    for i in range(states.shape[1]):  # the state before every 64th token; at a border the row's, from before it
        if not packed:
            assert_within(states[:, i], hp[:, 64 * i], ep[:, 64 * i], "states")
        elif i:
            assert_within(states[:, i], ry[:, 64 * i - 1], ey[:, 64 * i - 1], "states")
    got = run_bwd(lib, z, states, cu, gate, norm)
    want = backward(z["dy"], z["x"], z["g"], z["rate"], z["h0"], z["dhT"], gate, norm, spans)
    for a, b, what in zip(got, want, ("dx", "dg", "drate", "dh0")):
        if a is None:
            assert what == "drate" and b is None or what == "dh0" and not state
        else:
            assert_within(a, b[0], b[1], what)
    return z, cu, (y, hT, states), got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", FORMS)
@pytest.mark.parametrize("lens,packed,D", [
    ((1,), False, 64), ((2, 2, 2), False, 7), ((37, 37), False, 130), ((200,), False, 64),
    ((1, 0, 2, 3, 0, 70, 1), True, 72), ((0, 0, 5), True, 1), ((64, 64, 1, 127), True, 33),
])
def test_prompt_and_gradient(cuda_lib, dtype, gate, norm, lens, packed, D):
    dt = DT[dtype]
    z, cu, out, grads = check(cuda_lib, lens, packed, D, dt, gate, norm, True)
    check(cuda_lib, lens, packed, D, dt, gate, norm, False, 1)
    # slices of wider projections give the same bits, on wide and on narrow accesses
    for shift in (1, 8):
        s = dict(z, **{k: sliced(z[k], shift + i, 2 * shift - i) for i, k in enumerate(("x", "g", "dy"))})
        again = run_fwd(cuda_lib, s, cu, gate, norm, output_states=True)
        assert all(torch.equal(a, b) for a, b in zip(again[:2], out[:2]))
        for a, b in zip(run_bwd(cuda_lib, s, out[2], cu, gate, norm), grads):
            assert a is None and b is None or torch.equal(a, b)
    # in place
    h = z["h0"].clone()
    y, hT, st = run_fwd(cuda_lib, dict(z, h0=h), cu, gate, norm, hT=h)
    assert hT.data_ptr() == h.data_ptr() and st is None and torch.equal(h, out[1]) and torch.equal(y, out[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", [("log", None), ("sigmoid", "linear"), ("rate", "sqrt")])
@pytest.mark.parametrize("lens,packed,D", [
    ((1605,), False, 64), ((700, 700, 700), False, 200), ((130,), False, 5000), ((9,) * 300, False, 100),
    ((513, 0, 1, 600, 511), True, 96), (tuple((7 * i) % 41 for i in range(60)), True, 31), ((300, 300), False, 9000),
])
def test_many_blocks_in_time(cuda_lib, dtype, gate, norm, lens, packed, D):
    """Rounds of clusters, of single blocks, of blocks with few warps."""
    check(cuda_lib, lens, packed, D, DT[dtype], gate, norm, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,norm", FORMS)
@pytest.mark.parametrize("N,D", [(1, 64), (5, 129), (300, 40), (3, 1)])
def test_step(cuda_lib, dtype, gate, norm, N, D):
    z, _ = inputs((1,) * N, False, D, DT[dtype], gate)
    ry, ey, rh, eh, *_ = forward(z["x"], z["g"], z["rate"], z["h0"], gate, norm, [(n, 0, 1) for n in range(N)])
    for x, g in ((z["x"], z["g"]), (sliced(z["x"], 1, 2), sliced(z["g"], 4, 0))):
        h = z["h0"].clone()
        y = cuda_lib.gdn_glr_recurrent_step(x[:, 0], g[:, 0], h, z["rate"], gate=gate, input_norm=norm)
        assert_within(y[:, None], ry, ey, "y")
        assert_within(h, rh, eh, "h")
        # a prompt of one token is the step
        y1, h1, _ = run_fwd(cuda_lib, z, None, gate, norm)
        assert torch.equal(y1[:, 0], y) and torch.equal(h1, h)


def test_prompt_then_steps_and_split_prompts(cuda_lib):
    z, _ = inputs((150, 150), False, 136, torch.float32, "sigmoid")
    ry, ey, rh, eh, *_ = forward(z["x"], z["g"], None, z["h0"], "sigmoid", "linear", spans_of((150, 150), False))
    part = lambda lo, hi, h: run_fwd(cuda_lib, dict(z, x=z["x"][:, lo:hi].contiguous(),  # noqa: E731
                                                    g=z["g"][:, lo:hi].contiguous(), h0=h), None, "sigmoid", "linear")
    y, h, _ = part(0, 77, z["h0"])
    y2, h, _ = part(77, 140, h)
    parts = [y, y2] + [cuda_lib.gdn_glr_recurrent_step(z["x"][:, t], z["g"][:, t], h, gate="sigmoid",
                                                       input_norm="linear")[:, None] for t in range(140, 150)]
    assert_within(torch.cat(parts, 1), ry, ey, "y")
    assert_within(h, rh, eh, "h")


def test_leaves_rows_behind_the_last_sequence(cuda_lib):
    for T, borders, D in ((100, [0, 33, 60], 64), (4000, [0, 1500, 1501, 3100], 32), (300, [0, 0, 0], 8)):
        n, end = len(borders) - 1, borders[-1]
        z, _ = inputs((T,), False, D, torch.bfloat16, "rate")
        z["h0"], z["dhT"] = randn(gen_of(1), n, D), randn(gen_of(2), n, D)
        for k in ("x", "g", "dy"):
            z[k][:, end:] = float("nan")
        cu = torch.tensor(borders, dtype=torch.int32, device="cuda")
        y, dx, dg = (torch.full_like(z["x"], 7.0) for _ in range(3))
        st = torch.full((1, -(-T // 64), D), float("nan"), device="cuda")
        _, hT, _ = run_fwd(cuda_lib, z, cu, "rate", "sqrt", y=y, states=st)
        _, _, drate, dh0 = run_bwd(cuda_lib, z, st, cu, "rate", "sqrt", dx=dx, dg=dg)
        short = {k: v[:, :end].contiguous() if k in ("x", "g", "dy") else v for k, v in z.items()}
        spans = [(0, a, b) for a, b in zip(borders[:-1], borders[1:])]
        ry, ey, rh, eh, *_ = forward(short["x"], short["g"], z["rate"], z["h0"], "rate", "sqrt", spans)
        want = backward(short["dy"], short["x"], short["g"], z["rate"], z["h0"], z["dhT"], "rate", "sqrt", spans)
        assert_within(y[:, :end], ry, ey, "y")
        assert_within(hT, rh, eh, "hT")
        for got, (ref, err), what in ((dx[:, :end], want[0], "dx"), (dg[:, :end], want[1], "dg"),
                                      (drate, want[2], "drate"), (dh0, want[3], "dh0")):
            assert_within(got, ref, err, what)
        for t in (y, dx, dg):
            assert (t[:, end:] == 7).all()
        assert torch.isnan(st[:, -(-end // 64):]).all()


def test_clamps_a_broken_border_table(cuda_lib):
    """Borders outside [0, T] or out of order: no access outside the tensors, sane tables kept."""
    for T, D in ((64, 64), (1200, 33)):
        z, _ = inputs((T,), False, D, torch.bfloat16, "log")
        z["h0"], z["dhT"] = randn(gen_of(1), 2, D), randn(gen_of(2), 2, D)
        st = torch.zeros(1, -(-T // 64), D, device="cuda")
        for borders in ([0, 1 << 30, 1 << 30], [-5, 70, 20], [40, 10, 64], [64, 64, 0], [5, 9, T]):
            cu = torch.tensor(borders, dtype=torch.int32, device="cuda")
            run_fwd(cuda_lib, z, cu, "log", None)
            run_bwd(cuda_lib, z, st, cu, "log", None)
        z["h0"], z["dhT"] = z["h0"][:1], z["dhT"][:1]
        y, hT, _ = run_fwd(cuda_lib, z, torch.tensor([0, 1 << 30], dtype=torch.int32, device="cuda"), "log", None)
        ry, ey, rh, eh, *_ = forward(z["x"], z["g"], None, z["h0"], "log", None, [(0, 0, T)])
        assert_within(y, ry, ey, "y")
        assert_within(hT, rh, eh, "hT")


def test_infinities_and_nan_stay_in_their_channel_and_sequence(cuda_lib):
    """Also where decays' products underflow between them and the tokens behind."""
    T = 1400
    z, _ = inputs((T,), False, 64, torch.float32, "log")
    z["g"][..., 20:30] = -3.0  # e^-600 within 200 tokens
    cu = torch.tensor([0, 500, 900, T], dtype=torch.int32, device="cuda")
    z["h0"], z["dhT"] = randn(gen_of(1), 3, 64), randn(gen_of(2), 3, 64)
    clean = run_fwd(cuda_lib, z, cu, "log", None, output_states=True)
    cleang = run_bwd(cuda_lib, z, clean[2], cu, "log", None)
    bad = dict(z, x=z["x"].clone(), dy=z["dy"].clone())
    bad["x"][0, 510, 3], bad["x"][0, 520, 25] = float("nan"), float("inf")
    bad["dy"][0, 800, 5], bad["dy"][0, 810, 26] = float("nan"), float("inf")
    y, hT, st = run_fwd(cuda_lib, bad, cu, "log", None, output_states=True)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 510:900, 3] = hit[0, 520:900, 25] = True
    assert torch.equal(y[~hit], clean[0][~hit]) and torch.isnan(y[0, 510:900, 3]).all()
    assert (y[0, 520:900, 25] == float("inf")).all()
    assert torch.equal(hT[[0, 2]], clean[1][[0, 2]]) and torch.isnan(hT[1, 3]) and torch.isinf(hT[1, 25])
    dx, dg, _, dh0 = run_bwd(cuda_lib, bad, st, cu, "log", None)
    hit[:] = False
    hit[0, 500:801, 5] = hit[0, 500:811, 26] = True
    assert torch.equal(dx[~hit], cleang[0][~hit]) and torch.isnan(dx[0, 500:801, 5]).all()
    assert (dx[0, 500:811, 26] == float("inf")).all()
    assert torch.equal(dh0[[0, 2]], cleang[3][[0, 2]])


@pytest.mark.parametrize("gate,norm", FORMS)
def test_gates_at_their_ends(cuda_lib, gate, norm):
    """Open and closed gates, decays next to 1 and underflown ones: no NaN, the weights keep their digits."""
    ends = {"log": [-0.0, -1e-7, -1e-5, -1e-3, -0.4999, -0.25, -0.2501, -0.5, -20.0, -100.0, -1e4],
            "sigmoid": [-1e4, -100.0, -87.0, -20.0, -1.0, 0.0, 1.0, 16.0, 40.0, 100.0, 1e4],
            "rate": [-1e4, -100.0, -87.0, -20.0, -1.0, 0.0, 1.0, 16.0, 40.0, 100.0, 1e4]}[gate]
    D = len(ends)
    g = torch.tensor(ends, device="cuda").expand(1, 70, D).contiguous()
    z = dict(x=randn(gen_of(1), 1, 70, D), dy=randn(gen_of(2), 1, 70, D), g=g, h0=randn(gen_of(3), 1, D),
             dhT=randn(gen_of(4), 1, D), rate=-torch.linspace(0.001, 3, D, device="cuda") if gate == "rate" else None)
    y, hT, st = run_fwd(cuda_lib, z, None, gate, norm, output_states=True)
    ry, ey, rh, eh, *_ = forward(z["x"], g, z["rate"], z["h0"], gate, norm, [(0, 0, 70)])
    # (decays below 2^-126 are flushed)
    assert_within(y, ry, ey + 1e-37, "y")
    assert_within(hT, rh, eh + 1e-37, "hT")
    got = run_bwd(cuda_lib, z, st, None, gate, norm)
    want = backward(z["dy"], z["x"], g, z["rate"], z["h0"], z["dhT"], gate, norm, [(0, 0, 70)])
    for a, b, what in zip(got, want, ("dx", "dg", "drate", "dh0")):
        if a is not None:
            # (weights of flushed decays, and what they divide, are below 1e-18)
            assert_within(a, b[0], b[1] + 1e-17, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_its_bits_on_streams_threads_and_graphs(cuda_lib, dtype):
    import threading
    cases = [inputs((900, 900), False, 192, DT[dtype], "rate", seed=s)[0] for s in (1, 2)]

    def both(z, **kw):
        y, hT, st = run_fwd(cuda_lib, z, None, "rate", "sqrt", output_states=True, **kw)
        return (y, hT, st) + run_bwd(cuda_lib, z, st, None, "rate", "sqrt", **kw)

    want = [both(z) for z in cases]
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(s, t) for s, t in zip(a, b))  # noqa: E731
    graphs, outs = [], []
    for z in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(z))
        graphs.append(graph)
    sides = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))
    bad = []

    def work(i):
        for _ in range(20):
            out = both(cases[i], stream=sides[i])
            sides[i].synchronize()
            if not same(out, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    # the caller's workspace, filled with NaN first
    need = cuda_lib.gdn_glr_chunk_bwd_workspace_size(2, 900, 192, "rate")
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    assert need > 0 and same(run_bwd(cuda_lib, cases[0], want[0][2], None, "rate", "sqrt", workspace=ws), want[0][3:])


def test_empty_batches(cuda_lib):
    bf = torch.bfloat16
    x, rate = torch.empty(2, 0, 16, dtype=bf, device="cuda"), -torch.ones(16, device="cuda")
    h0, dhT = torch.ones(2, 16, device="cuda"), 2 * torch.ones(2, 16, device="cuda")
    y, hT, st = cuda_lib.gdn_glr_chunk_fwd(x, x, rate, h0, gate="rate", output_states=True)
    assert y.numel() == st.numel() == 0 and torch.equal(hT, h0)
    assert (cuda_lib.gdn_glr_chunk_fwd(x, x)[1] == 0).all()
    _, _, drate, dh0 = cuda_lib.gdn_glr_chunk_bwd(x, x, x, st, rate, h0, dhT, gate="rate")
    assert (drate == 0).all() and torch.equal(dh0, dhT)
    _, _, drate, dh0 = cuda_lib.gdn_glr_chunk_bwd(x, x, x, st, rate, gate="rate")
    assert (drate == 0).all() and dh0 is None
    none = torch.empty(0, 5, 16, dtype=bf, device="cuda")
    y, hT, st = cuda_lib.gdn_glr_chunk_fwd(none, none, rate, gate="rate", output_states=True)
    assert y.shape == none.shape and hT.shape == (0, 16)
    assert (cuda_lib.gdn_glr_chunk_bwd(none, none, none, st, rate, gate="rate")[2] == 0).all()
    assert cuda_lib.gdn_glr_recurrent_step(none[:, 0], none[:, 0], h0[:0]).numel() == 0
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    _, hT, _ = cuda_lib.gdn_glr_chunk_fwd(x[:1], x[:1], None, h0, cu_seqlens=cu)
    assert torch.equal(hT, h0)


def test_many_empty_sequences(cuda_lib):
    """2^18 of them amid a few tokens: right, and searched, not walked."""
    k = 2 ** 18
    lens = [5, 1] + [0] * k + [7] + [0] * 3 + [2, 0, 1, 80] + [0] * k
    z, cu = inputs(lens, True, 8, torch.float32, "sigmoid")
    y, hT, st = run_fwd(cuda_lib, z, cu, "sigmoid", None, output_states=True)
    dx, dg, _, dh0 = run_bwd(cuda_lib, z, st, cu, "sigmoid", None)
    some = [i for i, n in enumerate(lens) if n]
    spans = spans_of([lens[i] for i in some], True)
    f = dict(z, h0=z["h0"][some], dhT=z["dhT"][some])
    ry, ey, rh, eh, *_ = forward(z["x"], z["g"], None, f["h0"], "sigmoid", None, spans)
    want = backward(z["dy"], z["x"], z["g"], None, f["h0"], f["dhT"], "sigmoid", None, spans)
    assert_within(y, ry, ey, "y")
    assert_within(hT[some], rh, eh, "hT")
    assert_within(dx, *want[0], "dx")
    assert_within(dg, *want[1], "dg")
    assert_within(dh0[some], *want[3], "dh0")
    rest = torch.ones(len(lens), dtype=torch.bool, device="cuda")
    rest[some] = False
    assert torch.equal(hT[rest], z["h0"][rest]) and torch.equal(dh0[rest], z["dhT"][rest])


def test_offsets_beyond_32_bits(cuda_lib):
    """Tensors of more than 2^31 elements: the last rows against the definition."""
    D, T, bf = 32768, 66016, torch.bfloat16
    z, _ = inputs((40,), False, D, bf, "log")
    x = torch.zeros(1, T, D, dtype=bf, device="cuda")
    x[:, -40:] = z["x"]
    g = torch.full_like(x, float("-inf"))  # nothing of the state is kept
    g[:, -40:] = z["g"]
    y, hT, st = cuda_lib.gdn_glr_chunk_fwd(x, g, output_states=True)
    ry, ey, rh, eh, *_ = forward(z["x"], z["g"], None, None, "log", None, [(0, 0, 40)])
    assert_within(y[:, -40:], ry, ey, "y")
    assert_within(hT, rh, eh, "hT")
    x[:, -40:], y[:, :-40] = z["x"], 0
    y[:, -40:] = z["dy"]  # y as dy
    dx, dg, _, _ = cuda_lib.gdn_glr_chunk_bwd(y, x, g, st)
    want = backward(z["dy"], z["x"], z["g"], None, None, None, "log", None, [(0, 0, 40)])
    assert_within(dx[:, -40:], *want[0], "dx")
    assert_within(dg[:, -40:], *want[1], "dg")
    del y, st, dx, dg, x, g
    n = 70000
    h = torch.zeros(n, D, device="cuda")
    x, g = torch.zeros(n, D, dtype=bf, device="cuda"), torch.zeros(n, D, dtype=bf, device="cuda")
    x[-1], g[-1], h[-1] = z["x"][0, 0], z["g"][0, 0], z["h0"][0]
    y = cuda_lib.gdn_glr_recurrent_step(x, g, h)
    ry, ey, rh, eh, *_ = forward(z["x"][:, :1], z["g"][:, :1], None, z["h0"], "log", None, [(0, 0, 1)])
    assert_within(y[-1:, None], ry, ey, "step")
    assert_within(h[-1:], rh, eh, "state")


def test_binding_refusals(cuda_lib):
    dev, bf = "cuda", torch.bfloat16
    x, h, rate = torch.zeros(1, 8, 16, dtype=bf, device=dev), torch.zeros(1, 16, device=dev), -torch.ones(16, device=dev)
    st = torch.zeros(1, 1, 16, device=dev)
    fwd, bwd, step = cuda_lib.gdn_glr_chunk_fwd, cuda_lib.gdn_glr_chunk_bwd, cuda_lib.gdn_glr_recurrent_step
    err = cuda_lib.GdnError
    for bad, fn in [
        (TypeError, lambda: fwd(x.half(), x)), (TypeError, lambda: fwd(x, x.float())), (ValueError, lambda: fwd(x, x[:, :4])),
        (ValueError, lambda: fwd(x.cpu(), x)), (ValueError, lambda: fwd(x[0], x[0])), (ValueError, lambda: fwd(x, x, gate="tanh")),
        (ValueError, lambda: fwd(x, x, input_norm="cube")), (err, lambda: fwd(x, x, rate)), (err, lambda: fwd(x, x, gate="rate")),
        (ValueError, lambda: fwd(x, x, h0=h[:, :8].contiguous())), (TypeError, lambda: fwd(x, x, h0=h.to(bf))),
        (err, lambda: fwd(x, x.clone(), y=x)), (ValueError, lambda: fwd(x[..., ::2], x[..., ::2])),
        (ValueError, lambda: fwd(x, x, states=st[..., :8].contiguous())), (ValueError, lambda: fwd(x.expand(2, 8, 16), x)),
        (ValueError, lambda: fwd(x, x, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=dev))),
        (ValueError, lambda: step(x[0], x[0], h)), (err, lambda: step(x[:, 0], x[:, 0], h, rate)),
        (ValueError, lambda: bwd(x[:, :4], x, x, st)), (ValueError, lambda: bwd(x, x, x, st[:, :0])),
        (ValueError, lambda: bwd(x, x, x, st, drate=rate)), (err, lambda: bwd(x, x.clone(), x.clone(), st, dx=x)),
        (err, lambda: bwd(x, x, x, st, h0=h, dhT=h, dh0=h)),
        (err, lambda: bwd(x, x, x, st, rate, gate="rate", workspace=torch.empty(16, dtype=torch.uint8, device=dev))),
    ]:
        with pytest.raises(bad):
            fn()
