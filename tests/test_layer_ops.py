"""GPU tests of the layer operators (short causal convolution, S6 scan, RMS norm) against
their definitions in 64 bits, with bounds carried through the arithmetic.

Half a unit of rounding is u = 2^-24 in fp32.  Every bound below counts the roundings of the
fp32 arithmetic on the magnitudes that it works on, and one rounding of the result to its
storage type (half a step: finfo.eps / 2 of the value).
"""
import numpy as np
import pytest
import torch

from linear_attention_prefill_gb300.workloads import cu_seqlens_of

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


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


def assert_within(got, ref, err, dtype, what):
    """|got - ref| <= err + half a step of the storage type at |ref| + err."""
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny
    bound = err + half * (ref.abs() + err) + tiny
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst " \
                          f"{(d / bound).nan_to_num(float('inf')).max().item():.3g} of the bound"


def dsilu(v):
    return v * torch.sigmoid(v)


def spans_of(lens, packed, batch):
    if packed:
        cu = np.concatenate([[0], np.cumsum(lens)])
        return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]
    return [(b, 0, lens[0]) for b in range(batch)]


# ---- short convolution ---------------------------------------------------------------


def conv_ref(x, w, bias, s0, act, spans):
    """(y, error of y, states): sum in 64 bits; error = roundings of W products and sums."""
    W = w.shape[1]
    y, err = torch.zeros_like(x, dtype=torch.float64), torch.zeros_like(x, dtype=torch.float64)
    states = []
    for n, (b, lo, hi) in enumerate(spans):
        past = s0[n].double() if s0 is not None else x.new_zeros(W - 1, x.shape[2], dtype=torch.float64)
        full = torch.cat([past, x[b, lo:hi].double()])
        terms = [full[j:j + hi - lo] * w[:, j].double() for j in range(W)]
        v, mag = sum(terms), sum(t.abs() for t in terms)
        if bias is not None:
            v, mag = v + bias.double(), mag + bias.double().abs()
        e = (W + 1) * U * mag
        if act:  # |silu'| <= 1.1; its own arithmetic: 2^x, a sum, a reciprocal, two products
            e = 1.1 * e + (8 + 2 * v.abs()) * U * dsilu(v).abs()
            v = dsilu(v)
        y[b, lo:hi], err[b, lo:hi] = v, e
        states.append(full[full.shape[0] - (W - 1):])
    return y, err, torch.stack(states)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens,packed,D,state", [
    ((1,), False, 64, True), ((2, 2, 2), False, 8, True), ((37, 37), False, 129, False),
    ((1, 0, 2, 3, 0, 70, 1), True, 72, True), ((0, 0, 5), True, 7, False), ((65,), False, 1032, True),
    ((31, 33, 1, 64), True, 200, True),
])
def test_conv_prompt(cuda_lib, dtype, W, lens, packed, D, state):
    dt, g = DT[dtype], gen_of(11 * W + D)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    x = randn(g, B, T, D, dtype=dt)
    w, bias = randn(g, D, W), randn(g, D)
    s0 = randn(g, len(lens), W - 1, D, dtype=dt) if state else None
    cu = torch.from_numpy(cu_seqlens_of(lens)).cuda() if packed else None
    for act, b, xx in (("silu", bias, sliced(x, 8, 8)), (None, None, sliced(x, 3, 2)), ("silu", None, x)):
        y, sT = cuda_lib.gdn_short_conv_fwd(xx, w, b, s0, activation=act, cu_seqlens=cu)
        ref, err, st = conv_ref(x, w, b, s0, act, spans_of(lens, packed, B))
        assert_within(y, ref, err, dt, "y")
        assert torch.equal(sT.double(), st)
    # in place: the same state, and nothing written twice
    if state:
        s = s0.clone()
        y2, s2 = cuda_lib.gdn_short_conv_fwd(x, w, None, s, sT=s, cu_seqlens=cu)
        assert s2.data_ptr() == s.data_ptr() and torch.equal(s.double(), st) and torch.equal(y2, y)


def test_conv_leaves_rows_behind_the_last_sequence(cuda_lib):
    g = gen_of(3)
    x, w = randn(g, 1, 100, 64, dtype=torch.bfloat16), randn(g, 64, 4)
    x[:, 60:] = float("nan")
    y = torch.full_like(x, 7.0)
    cu = torch.tensor([0, 33, 60], dtype=torch.int32, device="cuda")
    _, sT = cuda_lib.gdn_short_conv_fwd(x, w, y=y, cu_seqlens=cu)
    ref, err, st = conv_ref(x[:, :60], w, None, None, "silu", [(0, 0, 33), (0, 33, 60)])
    assert_within(y[:, :60], ref, err, torch.bfloat16, "y")
    assert torch.equal(y[:, 60:], torch.full_like(y[:, 60:], 7.0)) and torch.equal(sT.double(), st)


def test_conv_clamps_a_broken_border_table(cuda_lib):
    """Borders outside [0, T] or out of order: no access outside the tensors, sane tokens kept."""
    g = gen_of(4)
    x, w = randn(g, 1, 64, 64, dtype=torch.bfloat16), randn(g, 64, 4)
    for borders in ([0, 1 << 30], [-5, 70, 20], [40, 10, 64], [64, 64, 0]):
        cu = torch.tensor(borders, dtype=torch.int32, device="cuda")
        cuda_lib.gdn_short_conv_fwd(x, w, cu_seqlens=cu)
    y, _ = cuda_lib.gdn_short_conv_fwd(x, w, cu_seqlens=torch.tensor([0, 1 << 30], dtype=torch.int32,
                                                                    device="cuda"))
    assert torch.equal(y, cuda_lib.gdn_short_conv_fwd(x, w)[0])


def test_conv_nan_and_inf_stay_in_their_window(cuda_lib):
    g = gen_of(5)
    x, w = randn(g, 1, 40, 16, dtype=torch.float32), randn(g, 16, 4)
    clean, _ = cuda_lib.gdn_short_conv_fwd(x, w)
    x[0, 10, 3], x[0, 20, 5] = float("nan"), float("inf")
    y, _ = cuda_lib.gdn_short_conv_fwd(x, w)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 10:14, 3] = True
    hit[0, 20:24, 5] = True
    assert torch.equal(y[~hit], clean[~hit]) and torch.isnan(y[0, 10:14, 3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,W", [(1, 64, 4), (5, 129, 4), (33, 8, 2), (3, 1032, 3), (257, 72, 4)])
def test_conv_step(cuda_lib, dtype, N, D, W):
    dt, g = DT[dtype], gen_of(N + D)
    x, w, bias = randn(g, N, D, dtype=dt), randn(g, D, W), randn(g, D)
    s0 = randn(g, N, W - 1, D, dtype=dt)
    for act, b, xx in (("silu", bias, sliced(x, 16, 8)), (None, None, sliced(x, 1, 0)), ("silu", None, x)):
        s = s0.clone()
        y = cuda_lib.gdn_short_conv_step(xx, w, s, b, activation=act)
        ref, err, st = conv_ref(x[:, None], w, b, s0, act, [(n, 0, 1) for n in range(N)])
        assert_within(y[:, None], ref, err, dt, "y")
        assert torch.equal(s.double(), st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_prompt_then_steps_is_one_prompt(cuda_lib, dtype):
    dt, g = DT[dtype], gen_of(6)
    x, w, bias = randn(g, 2, 50, 136, dtype=dt), randn(g, 136, 4), randn(g, 136)
    whole, end = cuda_lib.gdn_short_conv_fwd(x, w, bias)
    y, s = cuda_lib.gdn_short_conv_fwd(x[:, :20].contiguous(), w, bias)
    y2, s = cuda_lib.gdn_short_conv_fwd(x[:, 20:21].contiguous(), w, bias, s)
    parts = [y, y2] + [cuda_lib.gdn_short_conv_step(x[:, t], w, s, bias)[:, None] for t in range(21, 50)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, end)


# ---- S6 scan -------------------------------------------------------------------------


def s6_inputs(g, lead, N, dim, Ns, dt, softplus=True, state=True):
    step = torch.exp(torch.rand(dim, generator=g, device="cuda") * 4.6 - 6.9)
    x = dict(x=randn(g, *lead, dim, dtype=dt), z=randn(g, *lead, dim, dtype=dt),
             B=randn(g, *lead, Ns, dtype=dt), C=randn(g, *lead, Ns, dtype=dt),
             A=-(1 + torch.arange(Ns, device="cuda")) * torch.exp(0.1 * randn(g, dim, Ns)),
             D=randn(g, dim), h0=randn(g, N, dim, Ns) if state else None)
    if softplus:
        x.update(dt=randn(g, *lead, dim, dtype=dt), dt_bias=torch.log(torch.expm1(step)))
    else:
        x.update(dt=(step * torch.exp(randn(g, *lead, dim))).to(dt), dt_bias=None)
    return x


def s6_ref(x, softplus, spans, gate=True, skip=True):
    """(y, error of y, hT, error of hT) of the recurrence, token by token in 64 bits.

    The errors follow the fp32 arithmetic: a step D = softplus(v) is off by at most
    (3 |v| + 8) u relative (the rounding of v and of its scaled copy, both of which softplus
    passes on relative to itself at most |v| times; 2^x, a quotient and the series); a decay
    2^(D A log2 e) by 3 u (2^x: 1.4e-7) plus |D A| (the step's error + 3 u); a state adds
    two roundings a token, and y one for each of its Ns terms.
    """
    f = {k: v.double() if v is not None else None for k, v in x.items()}
    dim, Ns = f["A"].shape
    y = torch.zeros_like(f["x"])
    ey = torch.zeros_like(y)
    hs, es = [], []
    for n, (b, lo, hi) in enumerate(spans):
        h = f["h0"][n].clone() if f["h0"] is not None else f["x"].new_zeros(dim, Ns)
        mag, e = h.abs(), torch.zeros_like(h)
        for t in range(lo, hi):
            v = f["dt"][b, t] + (f["dt_bias"] if f["dt_bias"] is not None else 0.0)
            d = torch.logaddexp(v, torch.zeros_like(v)) if softplus else v
            ed = (3 * v.abs() + 8) * U
            arg = d[:, None] * f["A"]
            a = torch.exp(arg)
            ea = 3 * U + arg.abs() * (ed[:, None] + 3 * U)
            u = (d * f["x"][b, t])[:, None] * f["B"][b, t]
            e = a * e + a * mag * ea + u.abs() * (ed[:, None] + 3 * U)
            h = a * h + u
            mag = a * mag + u.abs()
            e = e + 2 * U * mag
            c = f["C"][b, t]
            o, eo = h @ c, e @ c.abs() + (Ns + 2) * U * (mag @ c.abs())
            if skip:
                o, eo = o + f["D"] * f["x"][b, t], eo + 2 * U * (f["D"] * f["x"][b, t]).abs()
            if gate:
                z = f["z"][b, t]
                s = dsilu(z)
                o, eo = o * s, eo * s.abs() + (8 + 2 * z.abs()) * U * (o * s).abs()
            y[b, t], ey[b, t] = o, eo
        hs.append(h)
        # a chunk's decay is 2^(A log2 e times the sum of its steps): a sum of n positive
        # terms is off by at most n u relative, and |a log a| <= 1/e
        es.append(2 * e + (hi - lo) * U * 0.37 * mag)
    return y, 2 * ey, torch.stack(hs), torch.stack(es)


def s6_run(lib, x, softplus, cu=None, gate=True, skip=True, hT=None, **kw):
    return lib.gdn_s6_chunk_fwd(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"] if skip else None,
                                x["z"] if gate else None, x["dt_bias"], x["h0"], hT=hT,
                                dt_softplus=softplus, cu_seqlens=cu, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,dim,Ns", [
    ((1,), False, 32, 16), ((70, 70), False, 100, 16), ((33,), False, 33, 5), ((64,), False, 16, 64),
    ((40, 0, 1, 95, 0), True, 72, 16), ((31, 65), True, 40, 8), ((17,), False, 34, 4),
    ((3, 3, 3), False, 65, 1), ((32,), False, 64, 32), ((45,), False, 31, 23), ((50,), False, 64, 6),
    (tuple((7 * i) % 41 for i in range(170)), True, 40, 16),  # several CTAs on every SM
])
def test_s6_prompt(cuda_lib, dtype, lens, packed, dim, Ns):
    dt, g = DT[dtype], gen_of(dim + Ns)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    cu = torch.from_numpy(cu_seqlens_of(lens)).cuda() if packed else None
    for i, (softplus, state, gate, skip) in enumerate([(True, True, True, True), (False, False, False, False),
                                                       (True, False, False, True)]):
        x = s6_inputs(g, (B, T), len(lens), dim, Ns, dt, softplus, state)
        y, hT = s6_run(cuda_lib, x, softplus, cu, gate, skip)
        ry, ey, rh, eh = s6_ref(x, softplus, spans_of(lens, packed, B), gate, skip)
        assert_within(y, ry, ey, dt, "y")
        assert_within(hT, rh, eh, torch.float32, "hT")
        # slices of wider projections give the same bits
        s = dict(x)
        for j, k in enumerate(("x", "dt", "z", "B", "C")):
            s[k] = sliced(x[k], j + i, 8 - j)
        y2, h2 = s6_run(cuda_lib, s, softplus, cu, gate, skip)
        assert torch.equal(y2, y) and torch.equal(h2, hT)
        if state:  # in place
            h = x["h0"].clone()
            y3, h3 = s6_run(cuda_lib, dict(x, h0=h), softplus, cu, gate, skip, hT=h)
            assert h3.data_ptr() == h.data_ptr() and torch.equal(h, hT) and torch.equal(y3, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,dim,Ns", [
    ((2085,), False, 64, 16), ((1300, 0, 2, 1700), True, 40, 16), ((1111, 1111), False, 33, 7),
    ((1500,), False, 16, 64), ((1100,), False, 4900, 16),  # the last: whole channels beside split ones
    ((1100,), False, 4900, 8), ((8950,), False, 32, 16), ((4500, 7, 4400), True, 31, 32),
])
def test_s6_split_over_time(cuda_lib, dtype, lens, packed, dim, Ns):
    """Few channels, many tokens: the split over time, with states and in place."""
    dt, g = DT[dtype], gen_of(dim)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    assert cuda_lib.gdn_s6_chunk_fwd_workspace_size(len(lens), T, dim, Ns, packed) > 0
    cu = torch.from_numpy(cu_seqlens_of(lens)).cuda() if packed else None
    x = s6_inputs(g, (B, T), len(lens), dim, Ns, dt)
    y, hT = s6_run(cuda_lib, x, True, cu)
    ry, ey, rh, eh = s6_ref(x, True, spans_of(lens, packed, B))
    assert_within(hT, rh, eh, torch.float32, "hT")
    # y reads states with the chunk sums' error too
    cm = x["C"].double().abs().amax() * Ns * rh.abs().amax() * 4
    assert_within(y, ry, ey + max(lens) * U * 0.37 * cm * (dsilu(x["z"].double())).abs(), dt, "y")
    h = x["h0"].clone()
    y2, _ = s6_run(cuda_lib, dict(x, h0=h), True, cu, hT=h)
    assert torch.equal(h, hT) and torch.equal(y2, y)
    # the caller's workspace, filled with NaN first, gives the same bits
    need = cuda_lib.gdn_s6_chunk_fwd_workspace_size(len(lens), T, dim, Ns, packed)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    y3, h3 = s6_run(cuda_lib, x, True, cu, workspace=ws)
    assert torch.equal(y3, y) and torch.equal(h3, hT)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,dim,Ns", [
    ((700,) + (5,) * 15, 40, 16),             # one CTA an SM
    ((3,) * 60 + (1400, 0, 33), 96, 16),      # several
    ((1, 900) + (20,) * 30, 64, 24), ((900, 40) + (9,) * 40, 33, 19),
])
def test_s6_one_long_sequence_among_short_ones(cuda_lib, dtype, lens, dim, Ns):
    dt, g = DT[dtype], gen_of(dim + Ns)
    T = sum(lens)
    assert cuda_lib.gdn_s6_chunk_fwd_workspace_size(len(lens), T, dim, Ns, True) > 0
    cu = torch.from_numpy(cu_seqlens_of(lens)).cuda()
    x = s6_inputs(g, (1, T), len(lens), dim, Ns, dt)
    y, hT = s6_run(cuda_lib, x, True, cu)
    ry, ey, rh, eh = s6_ref(x, True, spans_of(lens, True, 1))
    assert_within(hT, rh, eh, torch.float32, "hT")
    # y reads states with the chunk sums' error too, as above
    cm = x["C"].double().abs().amax() * Ns * rh.abs().amax() * 4
    assert_within(y, ry, ey + max(lens) * U * 0.37 * cm * (dsilu(x["z"].double())).abs(), dt, "y")
    h = x["h0"].clone()
    y2, _ = s6_run(cuda_lib, dict(x, h0=h), True, cu, hT=h)
    assert torch.equal(h, hT) and torch.equal(y2, y)


@pytest.mark.parametrize("Ns", [8, 16])
def test_s6_repeats_its_bits_beside_other_work(cuda_lib, Ns):
    """Chunks beside whole sequences, and a copy that keeps the memory busy: every wait is needed."""
    x = s6_inputs(gen_of(Ns), (1, 4064), 1, 5088, Ns, torch.bfloat16)
    other, a = torch.cuda.Stream(), torch.empty(1 << 28, device="cuda", dtype=torch.uint8)
    y, hT = s6_run(cuda_lib, x, True)
    ends = []
    for i in range(6):
        with torch.cuda.stream(other):
            b = a.clone()
        y2, h2 = s6_run(cuda_lib, x, True)
        ends.append((torch.equal(y2, y), torch.equal(h2, hT)))
        del b
    assert ends == [(True, True)] * 6


def test_s6_leaves_rows_behind_the_last_sequence(cuda_lib):
    for T, borders, dim in ((100, [0, 33, 60], 64), (4000, [0, 1500, 3100], 32)):
        x = s6_inputs(gen_of(T), (1, T), 2, dim, 16, torch.bfloat16)
        end = borders[-1]
        for k in ("x", "dt", "z", "B", "C"):
            x[k][:, end:] = float("nan")
        y = torch.full_like(x["x"], 7.0)
        cu = torch.tensor(borders, dtype=torch.int32, device="cuda")
        _, hT = s6_run(cuda_lib, x, True, cu, y=y)
        short = {k: v[:, :end].contiguous() if k in ("x", "dt", "z", "B", "C") else v for k, v in x.items()}
        ry, ey, rh, eh = s6_ref(short, True, [(0, borders[0], borders[1]), (0, borders[1], end)])
        assert_within(hT, rh, eh, torch.float32, "hT")
        assert torch.equal(y[:, end:], torch.full_like(y[:, end:], 7.0))
        assert torch.isfinite(y[:, :end].float()).all()


def test_s6_clamps_a_broken_border_table(cuda_lib):
    for T, dim in ((64, 64), (2048, 32)):
        x = s6_inputs(gen_of(T), (1, T), 2, dim, 16, torch.bfloat16)
        for borders in ([0, 1 << 30, 1 << 30], [-5, 70, 20], [40, 10, 64], [64, 64, 0]):
            cu = torch.tensor(borders, dtype=torch.int32, device="cuda")
            s6_run(cuda_lib, x, True, cu)
    x["h0"] = x["h0"][:1]
    want = s6_run(cuda_lib, x, True)
    got = s6_run(cuda_lib, x, True, torch.tensor([0, 1 << 30], dtype=torch.int32, device="cuda"))
    for a, b in zip(got, want):
        assert torch.allclose(a.float(), b.float(), rtol=1e-2, atol=1e-2)


def test_s6_infinite_and_nan_inputs_stay_in_their_channel(cuda_lib):
    for Ns in (16, 5):
        x = s6_inputs(gen_of(8), (1, 50), 1, 64, Ns, torch.float32)
        clean, hc = s6_run(cuda_lib, x, True)
        x["x"][0, 10, 3], x["x"][0, 20, 7] = float("nan"), float("inf")
        x["dt"][0, 30, 9] = float("inf")  # an infinite step forgets the state
        y, h = s6_run(cuda_lib, x, True)
        keep = torch.ones(64, dtype=torch.bool, device="cuda")
        keep[[3, 7, 9]] = False
        assert torch.equal(y[..., keep], clean[..., keep]) and torch.equal(h[:, keep], hc[:, keep])
        assert torch.isnan(y[0, 10:, 3]).all() and torch.equal(y[0, :10, 3], clean[0, :10, 3])
        assert not torch.isfinite(y[0, 20, 7])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,dim,Ns", [(1, 64, 16), (5, 100, 16), (33, 33, 5), (3, 24, 64), (2, 50, 8),
                                      (130, 17, 1), (2, 40, 32), (2, 9, 3)])
def test_s6_step(cuda_lib, dtype, N, dim, Ns):
    dt, g = DT[dtype], gen_of(N + dim + Ns)
    for softplus, gate, skip in ((True, True, True), (False, False, False)):
        x = s6_inputs(g, (N, 1), N, dim, Ns, dt, softplus)
        ry, ey, rh, eh = s6_ref(x, softplus, [(n, 0, 1) for n in range(N)], gate, skip)
        one = {k: v[:, 0] if k in ("x", "dt", "z", "B", "C") else v for k, v in x.items()}
        for cut in (False, True):
            s = {k: sliced(v, 4, 8) if cut and k in ("x", "dt", "z", "B", "C") else v for k, v in one.items()}
            h = x["h0"].clone()
            y = cuda_lib.gdn_s6_recurrent_step(s["x"], s["dt"], s["A"], s["B"], s["C"], h,
                                               s["D"] if skip else None, s["z"] if gate else None,
                                               s["dt_bias"], dt_softplus=softplus)
            assert_within(y[:, None], ry, ey, dt, "y")
            assert_within(h, rh, eh, torch.float32, "h")


def test_s6_prompt_then_steps(cuda_lib):
    """A prompt and single tokens after it against one prompt: every state within the bound."""
    x = s6_inputs(gen_of(9), (2, 60), 2, 72, 16, torch.float32)
    seq = ("x", "dt", "z", "B", "C")
    ry, ey, rh, eh = s6_ref(x, True, [(0, 0, 60), (1, 0, 60)])
    y, h = s6_run(cuda_lib, {k: v[:, :40].contiguous() if k in seq else v for k, v in x.items()}, True)
    parts = [y]
    for t in range(40, 60):
        parts.append(cuda_lib.gdn_s6_recurrent_step(
            x["x"][:, t], x["dt"][:, t], x["A"], x["B"][:, t], x["C"][:, t], h, x["D"], x["z"][:, t],
            x["dt_bias"], dt_softplus=True)[:, None])
    assert_within(torch.cat(parts, 1), ry, ey, torch.float32, "y")
    assert_within(h, rh, eh, torch.float32, "h")


# ---- RMS norm ------------------------------------------------------------------------


def norm_ref(x, w, residual, gate, eps):
    """(y, relative error of y before its rounding, r): D squares added in fp32 by at most 64
    in a row and a tree, a square root's reciprocal (2 u), three products, SiLU."""
    r = x.double() if residual is None else x.double() + residual.double()
    y = r / (r.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    rel = torch.full_like(y, 48 * U)
    if gate is not None:
        z = gate.double()
        y, rel = y * dsilu(z), rel + (8 + 2 * z.abs()) * U
    return y, rel, r


NORM_ROWS = [(1, 64), (3, 8), (17, 129), (5, 128), (130, 72), (2, 1032), (9, 2560), (3, 5123), (2, 16392),
             (1, 32768), (4, 1000), (6, 500), (1300, 520), (2500, 2560), (1217, 8192), (1216, 1001),
             (5000, 952), (1217, 4096), (1216, 12288), (70, 12900), (40, 250), (33, 1330), (9, 36), (5, 22)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", NORM_ROWS)
def test_norm(cuda_lib, dtype, rows, D):
    dt, g = DT[dtype], gen_of(rows + D)
    x, w = randn(g, rows, D, dtype=dt), randn(g, D)
    for residual, gate, cut in ((None, None, False), (randn(g, rows, D, dtype=dt), None, True),
                                (None, randn(g, rows, D, dtype=dt), True),
                                (randn(g, rows, D, dtype=dt), randn(g, rows, D, dtype=dt), False)):
        xx = sliced(x, 8, 8) if cut else x
        gg = sliced(gate, 3, 1) if cut and gate is not None else gate
        y, scales, out = cuda_lib.gdn_rms_norm_fwd(xx, w, residual, gg, eps=1e-5)
        ref, rel, r = norm_ref(x, w, residual, gate, 1e-5)
        assert scales is None and (out is None) == (residual is None)
        assert_within(y, ref, rel * ref.abs(), dt, "y")
        if residual is not None:
            assert_within(out, r, U * r.abs(), dt, "residual_out")
            res = residual.clone()  # in place
            y2, _, out2 = cuda_lib.gdn_rms_norm_fwd(x, w, res, gate, residual_out=res, eps=1e-5)
            assert out2.data_ptr() == res.data_ptr() and torch.equal(out2, out) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [None, 32, 64, 128])
@pytest.mark.parametrize("rows,D", NORM_ROWS)
def test_norm_e4m3(cuda_lib, dtype, group, rows, D):
    dt, g = DT[dtype], gen_of(rows * 3 + D)
    x, w = randn(g, rows, D, dtype=dt), randn(g, D)
    w[D // 2:] *= 1e-3
    for residual, gate in ((randn(g, rows, D, dtype=dt), None), (None, randn(g, rows, D, dtype=dt))):
        q, scales, out = cuda_lib.gdn_rms_norm_fwd(x, w, residual, gate, out_dtype=E4M3, group=group)
        ref, rel, r = norm_ref(x, w, residual, gate, 1e-6)
        width = group or D
        pad = torch.nn.functional.pad(ref, (0, -D % width)).reshape(rows, -1, width)
        top = pad.abs().amax(-1)
        rs = top / 448
        most = rel.amax()
        assert q.dtype == E4M3 and scales.shape == (rows, -(-D // width))
        assert ((scales.double() - rs).abs() <= (most + 2 * U) * rs).all()
        # q = y / scale to half a step: 2^-4 relative, 2^-10 below the normals; the value
        # itself is off by y's, the scale's and the quotient's errors
        v = (pad / rs[..., None]).reshape(rows, -1)[:, :D]
        off = (2 * most + 4 * U) * v.abs()
        assert ((q.double() - v).abs() <= off + 2.0 ** -4 * (v.abs() + off) + 2.0 ** -10).all()
        if residual is not None:
            assert_within(out, r, U * r.abs(), dt, "residual_out")


def test_norm_zero_huge_and_nan_rows(cuda_lib):
    for D in (128, 2560):
        x = torch.zeros(4, D, device="cuda")
        x[1], x[2, 3], x[3] = 1e-30, float("nan"), 3e4
        w = torch.ones(D, device="cuda")
        y, _, _ = cuda_lib.gdn_rms_norm_fwd(x, w, eps=1e-6)
        assert (y[0] == 0).all() and torch.isnan(y[2]).all() and (y[3] - 1).abs().max() < 1e-5
        for group in (None, 64):
            q, s, _ = cuda_lib.gdn_rms_norm_fwd(x, w, out_dtype=E4M3, group=group, eps=1e-6)
            assert (q[0].float() == 0).all() and (s[0] == 1).all()
            assert torch.isnan(q[2].float()).all() and torch.isnan(s[2]).all()
            assert (q[3].float() == 448).all() and torch.isfinite(s[1]).all()
            # y = 1e-30 / 1e-3: its own scale, full range
            assert (q[1].float() == 448).all() and (s[1] > 0).all()


@pytest.mark.parametrize("B,T,H,D", [(2, 7, 3, 128), (1, 700, 2, 1024), (3, 5, 7, 40)])
def test_norm_of_heads_with_a_sliced_gate(cuda_lib, B, T, H, D):
    """[B, T, H, D] with the gate a slice of the projection: tokens strided, heads dense."""
    g = gen_of(12)
    x = randn(g, B, T, H, D, dtype=torch.bfloat16)
    proj = randn(g, B, T, 2 * H * D + 16, dtype=torch.bfloat16)
    gate = proj[..., H * D:2 * H * D].unflatten(-1, (H, D))
    w = randn(g, D)
    y, _, _ = cuda_lib.gdn_rms_norm_fwd(x, w, gate=gate)
    ref, rel, _ = norm_ref(x, w, None, gate, 1e-6)
    assert_within(y, ref, rel * ref.abs(), torch.bfloat16, "y")
    z, _, _ = cuda_lib.gdn_rms_norm_fwd(x, w, gate=gate.contiguous())
    assert torch.equal(y, z)


# ---- together, and how calls behave ------------------------------------------------------


def test_a_gdn_layer(cuda_lib):
    """Norm with residual, projection, convolution, GDN with the fused prologue, gated norm:
    a prompt of 96 tokens in one call, and the first 90 with 6 decode steps behind them."""
    g = gen_of(20)
    T, M, H, d, W = 96, 256, 2, 128, 4
    x, res = randn(g, 1, T, M, dtype=torch.bfloat16), randn(g, 1, T, M, dtype=torch.bfloat16)
    wn, wo = 1 + 0.1 * randn(g, M), 1 + 0.1 * randn(g, d)
    wp = (randn(g, M, 4 * H * d) * M ** -0.5).to(torch.bfloat16)
    wg = randn(g, M, 2 * H) * M ** -0.5
    wc = randn(g, 3 * H * d, W) * 0.5

    def layer(x, res, conv, h, step):
        y, _, r = cuda_lib.gdn_rms_norm_fwd(x, wn, res)
        p = y @ wp
        ab = y.float() @ wg
        qkv, gate = p[..., :3 * H * d], p[..., 3 * H * d:]
        if step:
            qkv, s = cuda_lib.gdn_short_conv_step(qkv, wc, conv), conv
            q, k, v = (t.unflatten(-1, (H, d)).contiguous() for t in qkv.chunk(3, -1))
            o = cuda_lib.gdn_recurrent_step_prologue(q, k, v, ab[..., :H].contiguous(),
                                                     ab[..., H:].contiguous(), h)
        else:
            qkv, s = cuda_lib.gdn_short_conv_fwd(qkv, wc, s0=conv)
            q, k, v = (t.unflatten(-1, (H, d)).contiguous() for t in qkv.chunk(3, -1))
            o, h = cuda_lib.gdn_chunk_fwd_prologue(q, k, v, ab[..., :H].contiguous(),
                                                   ab[..., H:].contiguous(), h0=h)
        o, _, _ = cuda_lib.gdn_rms_norm_fwd(o, wo, gate=gate.unflatten(-1, (H, d)))
        return o, r, s, h

    o, r, s, h = layer(x, res, None, None, False)
    o1, _, s1, h1 = layer(x[:, :90].contiguous(), res[:, :90].contiguous(), None, None, False)
    outs = [o1]
    for t in range(90, T):
        ot, _, s1, h1 = layer(x[:, t].contiguous(), res[:, t].contiguous(), s1, h1, True)
        outs.append(ot[:, None])
    got = torch.cat(outs, 1).float()
    # two routes through 16-bit products: the forward's own tolerance, 2e-2 of the RMS, on
    # either side of the norm
    rms = o.float().square().mean().sqrt()
    assert torch.equal(r, (x.float() + res.float()).to(torch.bfloat16))
    assert (got - o.float()).abs().max() <= 2 * 2e-2 * rms + 2.0 ** -7 * o.float().abs().max()
    assert (h1 - h).abs().max() <= 2 * 2e-2 * h.square().mean().sqrt()
    cuda_lib.gdn_device_status()


def test_an_s6_layer_captured_and_replayed(cuda_lib):
    """Convolution, scan and norm in one CUDA graph, replayed on new inputs, against eager."""
    g = gen_of(21)
    T, dim, Ns = 1500, 64, 16  # split over time: a workspace inside the graph
    x = s6_inputs(g, (1, T), 1, dim, Ns, torch.bfloat16)
    w, wn = randn(g, dim, 4), randn(g, dim)

    def run():
        c, s = cuda_lib.gdn_short_conv_fwd(x["x"], w)
        y, h = cuda_lib.gdn_s6_chunk_fwd(c, x["dt"], x["A"], x["B"], x["C"], x["D"], x["z"], x["dt_bias"],
                                         x["h0"], dt_softplus=True)
        q, sc, r = cuda_lib.gdn_rms_norm_fwd(y, wn, c, out_dtype=E4M3, group=32)
        t = cuda_lib.gdn_s6_recurrent_step(c[:, -1], x["dt"][:, 0], x["A"], x["B"][:, 0], x["C"][:, 0],
                                           h, dt_softplus=False)
        u = cuda_lib.gdn_short_conv_step(x["x"][:, 0], w, s)
        return c, s, y, h, q.view(torch.uint8), sc, r, t, u

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (1, 2):
        fresh = s6_inputs(gen_of(seed), (1, T), 1, dim, Ns, torch.bfloat16)
        for k in x:
            x[k].copy_(fresh[k])
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_a_stream_by_its_handle(cuda_lib):
    g = gen_of(23)
    x, w = randn(g, 1, 40, 64, dtype=torch.bfloat16), randn(g, 64, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    want, _ = cuda_lib.gdn_short_conv_fwd(x, w)
    for handle in (side.cuda_stream, 0):
        y, _ = cuda_lib.gdn_short_conv_fwd(x, w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_calls_on_a_side_stream(cuda_lib):
    g = gen_of(22)
    x = s6_inputs(g, (1, 1500), 1, 64, 16, torch.bfloat16)
    w, wn = randn(g, 64, 4), randn(g, 64)
    torch.cuda.synchronize()
    want = s6_run(cuda_lib, x, True), cuda_lib.gdn_short_conv_fwd(x["x"], w), \
        cuda_lib.gdn_rms_norm_fwd(x["x"], wn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = s6_run(cuda_lib, x, True, stream=side), cuda_lib.gdn_short_conv_fwd(x["x"], w, stream=side), \
        cuda_lib.gdn_rms_norm_fwd(x["x"], wn, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        for s, t in zip(a, b):
            assert s is None and t is None or torch.equal(s, t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 3, 5, 31, 33])
def test_narrow_rows(cuda_lib, dtype, D):
    dt, g = DT[dtype], gen_of(D)
    x, w = randn(g, 2, 9, D, dtype=dt), randn(g, D, 3)
    s0 = randn(g, 2, 2, D, dtype=dt)
    y, sT = cuda_lib.gdn_short_conv_fwd(x, w, s0=s0)
    ref, err, st = conv_ref(x, w, None, s0, "silu", spans_of((9, 9), False, 2))
    assert_within(y, ref, err, dt, "convolution")
    assert torch.equal(sT.double(), st)
    for Ns in (1, 2, 16):
        z = s6_inputs(g, (2, 9), 2, D, Ns, dt)
        y, hT = s6_run(cuda_lib, z, True)
        ry, ey, rh, eh = s6_ref(z, True, spans_of((9, 9), False, 2))
        assert_within(y, ry, ey, dt, "scan")
        assert_within(hT, rh, eh, torch.float32, "state")
    wn, gate = randn(g, D), randn(g, 2, 9, D, dtype=dt)
    ref, rel, _ = norm_ref(x, wn, None, gate, 1e-6)
    assert_within(cuda_lib.gdn_rms_norm_fwd(x, wn, gate=gate)[0], ref, rel * ref.abs(), dt, "norm")
    for group in (None, 32, 128):
        q, scales, _ = cuda_lib.gdn_rms_norm_fwd(x, wn, gate=gate, out_dtype=E4M3, group=group)
        width = group or D
        rs = torch.nn.functional.pad(ref, (0, -D % width)).unflatten(-1, (-1, width)).abs().amax(-1) / 448
        assert ((scales.double() - rs).abs() <= (rel.amax() + 2 * U) * rs).all()
        v = ref / rs.repeat_interleave(width, -1)[..., :D]
        off = (2 * rel.amax() + 4 * U) * v.abs()
        assert ((q.double() - v).abs() <= off + 2.0 ** -4 * (v.abs() + off) + 2.0 ** -10).all()


def test_offsets_beyond_32_bits(cuda_lib):
    """Tensors of more than 2^31 elements: the last rows against the definition."""
    g, bf = gen_of(31), torch.bfloat16
    D, T = 32768, 66016
    x = torch.zeros(1, T, D, dtype=bf, device="cuda")
    x[:, -40:] = randn(g, 1, 40, D, dtype=bf)
    assert x.numel() > 2 ** 31
    w, wn = randn(g, D, 4), randn(g, D)
    y, sT = cuda_lib.gdn_short_conv_fwd(x, w)
    ref, err, st = conv_ref(x[:, -40:], w, None, None, "silu", [(0, 0, 40)])
    assert_within(y[:, -40:], ref, err, bf, "convolution")
    assert torch.equal(sT.double(), st)
    del y
    y = cuda_lib.gdn_rms_norm_fwd(x, wn, x)[0]
    ref, rel, _ = norm_ref(x[:, -40:], wn, x[:, -40:], None, 1e-6)
    assert_within(y[:, -40:], ref, rel * ref.abs(), bf, "norm")
    del y
    n, d = T // 32, 16  # the same memory as sequences of 32 tokens; B, C and dt far apart too
    z = s6_inputs(g, (1, 32), 1, D, 8, bf)
    rows = x.view(-1)[:n * 32 * D].view(n, 32, D)
    rows[-1] = z["x"][0]
    bc = torch.zeros(n, 32, D, dtype=bf, device="cuda")[..., D - d:]
    bc[-1, :, :8], bc[-1, :, 8:] = z["B"][0], z["C"][0]
    h0 = torch.zeros(n, D, 8, device="cuda")
    h0[-1] = z["h0"][0]
    step = dict(z, x=rows, dt=rows, z=None, B=bc[..., :8], C=bc[..., 8:], h0=h0)
    y, hT = s6_run(cuda_lib, step, True, gate=False)
    ry, ey, rh, eh = s6_ref(dict(z, dt=z["x"], z=None), True, [(0, 0, 32)], gate=False)
    assert_within(y[-1:], ry, ey, bf, "scan")
    assert_within(hT[-1:], rh, eh, torch.float32, "state")
    del y, hT, rows, step, bc, x, h0
    N, dim, Ns = 2200, 16384, 64
    h = torch.zeros(N, dim, Ns, device="cuda")
    assert h.numel() > 2 ** 31
    z = s6_inputs(g, (1, 1), 1, dim, Ns, bf)
    h[-1] = z["h0"][0]
    many = {k: z[k][0].expand(N, -1).contiguous() for k in ("x", "dt", "z", "B", "C")}
    y = cuda_lib.gdn_s6_recurrent_step(many["x"], many["dt"], z["A"], many["B"], many["C"], h, z["D"], many["z"],
                                       z["dt_bias"], dt_softplus=True)
    ry, ey, rh, eh = s6_ref(z, True, [(0, 0, 1)])
    assert_within(y[-1:, None], ry, ey, bf, "step")
    assert_within(h[-1:], rh, eh, torch.float32, "state")
    del h, many
    s = torch.zeros(22000, 3, D, dtype=bf, device="cuda")
    assert s.numel() > 2 ** 31
    s[-1] = randn(g, 3, D, dtype=bf)
    last, x1 = s[-1:].clone(), randn(g, 1, D, dtype=bf)
    y = cuda_lib.gdn_short_conv_step(x1.expand(22000, -1).contiguous(), w, s)
    ref, err, st = conv_ref(x1[:, None], w, None, last, "silu", [(0, 0, 1)])
    assert_within(y[-1:, None], ref, err, bf, "step")
    assert torch.equal(s[-1:].double(), st)


def test_two_graphs_replayed_in_turn_and_two_threads(cuda_lib):
    """Each graph has its own workspace, each thread its own stream."""
    import threading
    xs = [s6_inputs(gen_of(40 + i), (1, 1500), 1, 64, 16, torch.bfloat16) for i in range(2)]
    want = [s6_run(cuda_lib, x, True) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(s6_run(cuda_lib, x, True))
        graphs.append(graph)
    sides = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
    bad = []

    def work(i):
        for _ in range(50):
            y, hT = s6_run(cuda_lib, xs[i], True, stream=sides[i])
            sides[i].synchronize()
            if not (torch.equal(y, want[i][0]) and torch.equal(hT, want[i][1])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_empty_batches(cuda_lib):
    dev, bf = "cuda", torch.bfloat16
    w, A = torch.ones(16, 4, device=dev), -torch.ones(16, 8, device=dev)
    s0, h0 = torch.ones(2, 3, 16, dtype=bf, device=dev), torch.ones(2, 16, 8, device=dev)
    x, bc = torch.empty(2, 0, 16, dtype=bf, device=dev), torch.empty(2, 0, 8, dtype=bf, device=dev)
    y, sT = cuda_lib.gdn_short_conv_fwd(x, w, s0=s0)
    assert y.numel() == 0 and torch.equal(sT, s0)
    assert (cuda_lib.gdn_short_conv_fwd(x, w)[1] == 0).all()
    y, hT = cuda_lib.gdn_s6_chunk_fwd(x, x, A, bc, bc, h0=h0)
    assert y.numel() == 0 and torch.equal(hT, h0)
    assert (cuda_lib.gdn_s6_chunk_fwd(x, x, A, bc, bc)[1] == 0).all()
    none = torch.empty(0, 16, dtype=bf, device=dev)
    assert cuda_lib.gdn_short_conv_step(none, w, s0[:0]).numel() == 0
    assert cuda_lib.gdn_s6_recurrent_step(none, none, A, none[:, :8], none[:, :8], h0[:0]).numel() == 0
    assert cuda_lib.gdn_rms_norm_fwd(none, w[:, 0].contiguous())[0].numel() == 0


def test_binding_refusals(cuda_lib):
    dev, bf = "cuda", torch.bfloat16
    x, w, s = torch.zeros(1, 8, 16, dtype=bf, device=dev), torch.ones(16, 4, device=dev), \
        torch.zeros(1, 3, 16, dtype=bf, device=dev)
    A, bc, h = -torch.ones(16, 8, device=dev), torch.zeros(1, 8, 8, dtype=bf, device=dev), \
        torch.zeros(1, 16, 8, device=dev)
    conv, scan, norm = cuda_lib.gdn_short_conv_fwd, cuda_lib.gdn_s6_chunk_fwd, cuda_lib.gdn_rms_norm_fwd
    err = cuda_lib.GdnError
    for bad, fn in [
        (TypeError, lambda: conv(x.half(), w)), (TypeError, lambda: conv(x, w.to(bf))),
        (ValueError, lambda: conv(x.cpu(), w)), (ValueError, lambda: conv(x[..., ::2], w[:8])),
        (ValueError, lambda: conv(x[0], w)), (ValueError, lambda: conv(x, w, activation="relu")),
        (ValueError, lambda: conv(x, w, s0=s[:, :2].contiguous())),
        (ValueError, lambda: conv(x.expand(2, 8, 16), w)),
        (err, lambda: conv(x, torch.ones(16, 5, device=dev))), (err, lambda: conv(x, w, y=x)),
        (err, lambda: conv(x, torch.ones(16, 1, device=dev))),
        (ValueError, lambda: conv(x, w, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=dev))),
        (TypeError, lambda: conv(x, w, cu_seqlens=torch.zeros(2, dtype=torch.int64, device=dev))),
        (ValueError, lambda: conv(x.view(2, 4, 16), w, cu_seqlens=torch.zeros(2, dtype=torch.int32, device=dev))),
        (ValueError, lambda: cuda_lib.gdn_short_conv_step(x[0], w, s)),
        (ValueError, lambda: scan(x, x[:, :4], A, bc, bc)), (TypeError, lambda: scan(x, x.float(), A, bc, bc)),
        (ValueError, lambda: scan(x, x, A, bc[..., :4], bc)), (err, lambda: scan(x, x, A, bc, bc, y=x)),
        (err, lambda: scan(x, x, torch.ones(16, 65, device=dev), x.new_zeros(1, 8, 65), x.new_zeros(1, 8, 65))),
        (ValueError, lambda: scan(x, x, A, bc, bc, h0=h[:, :8].contiguous())),
        (ValueError, lambda: cuda_lib.gdn_s6_recurrent_step(x[0], x[0], A, bc[0], bc[0], h)),
        (TypeError, lambda: norm(x, w[:, 0].contiguous(), x.float())), (err, lambda: norm(x, w[:, 0].contiguous(), y=x)),
        (ValueError, lambda: norm(x, w[:8, 0].contiguous())),
        (ValueError, lambda: norm(x, w[:, 0].contiguous(), group=32)),
        (ValueError, lambda: norm(x, w[:, 0].contiguous(), out_dtype=E4M3, group=48)),
        (TypeError, lambda: norm(x, w[:, 0].contiguous(), out_dtype=torch.float16)),
        (ValueError, lambda: norm(x, w[:, 0].contiguous(), residual_out=x.clone())),
        (err, lambda: norm(x, w[:, 0].contiguous(), eps=-1.0)),
        (err, lambda: norm(torch.zeros(1, 40000, device=dev), torch.zeros(40000, device=dev))),
    ]:
        with pytest.raises(bad):
            fn()
    big = torch.zeros(1, 2048, 32, dtype=bf, device=dev)
    bb = torch.zeros(1, 2048, 16, dtype=bf, device=dev)
    with pytest.raises(err, match="workspace"):
        scan(big, big, -torch.ones(32, 16, device=dev), bb, bb,
             workspace=torch.empty(256, dtype=torch.uint8, device=dev))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("end", [1, 7, 2049, 2050, 4095])
def test_conv_blocks_behind_the_last_sequence_leave_nothing_in_flight(cuda_lib, dtype, end):
    """Most blocks find their rows behind the last sequence (or meet its end within a round) and leave
    early; other kernels take their shared memory at once, on the same and on another stream."""
    dt, g, T, D = DT[dtype], gen_of(end), 4096, 2048
    x, w = randn(g, 1, T, D, dtype=dt), randn(g, D, 4)
    cu = torch.tensor([0, end], dtype=torch.int32, device="cuda")
    ref, err, st = conv_ref(x[:, :end], w, None, None, "silu", [(0, 0, end)])
    s = s6_inputs(gen_of(1), (1, 256), 1, 512, 16, torch.bfloat16)
    torch.cuda.synchronize()
    other, want, ends = torch.cuda.Stream(), s6_run(cuda_lib, s, True), []
    torch.cuda.synchronize()
    for _ in range(8):
        y = torch.full_like(x, 7.0)
        with torch.cuda.stream(other):
            beside = s6_run(cuda_lib, s, True)
        _, sT = cuda_lib.gdn_short_conv_fwd(x, w, y=y, cu_seqlens=cu)
        ends.append((y, sT, s6_run(cuda_lib, s, True), beside))
    torch.cuda.synchronize()
    for y, sT, *scans in ends:
        assert_within(y[:, :end], ref, err, dt, "y")
        assert (y[:, end:] == 7).all() and torch.equal(sT.double(), st)
        assert all(torch.equal(a, b) for scan in scans for a, b in zip(scan, want))


def test_conv_of_more_than_2_30_sequences(cuda_lib):
    """All empty but the last: the search for a token's sequence ends at numbers whose sum passes 31 bits."""
    g, N, T, bf = gen_of(17), 2 ** 30 + 5, 64, torch.bfloat16
    x, w = randn(g, 1, T, 8, dtype=bf), randn(g, 8, 4)
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    cu[-1] = T
    y, sT = cuda_lib.gdn_short_conv_fwd(x, w, cu_seqlens=cu, output_final_state=False)
    ref, err, _ = conv_ref(x, w, None, None, "silu", [(0, 0, T)])
    assert sT is None
    assert_within(y, ref, err, bf, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 7])
def test_conv_passes_many_empty_sequences_at_once(cuda_lib, dtype, D):
    """Empty sequences amid a run of tokens: right, and not walked through one by one (65536 of them took
    5.4 ms that way, 2^19 43 ms)."""
    dt, g, k = DT[dtype], gen_of(19), 2 ** 19
    lens = [5, 1] + [0] * k + [7] + [0] * 3 + [2, 0, 1, 4] + [0] * k
    x, w = randn(g, 1, sum(lens), D, dtype=dt), randn(g, D, 4)
    cu = torch.from_numpy(cu_seqlens_of(lens)).cuda()
    some = [n for n in lens if n]
    want, _ = cuda_lib.gdn_short_conv_fwd(x, w, cu_seqlens=torch.from_numpy(cu_seqlens_of(some)).cuda())
    ref, err, _ = conv_ref(x, w, None, None, "silu", spans_of(some, True, 1))
    times = []
    for _ in range(5):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        y, _ = cuda_lib.gdn_short_conv_fwd(x, w, cu_seqlens=cu, output_final_state=False)
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
        assert_within(y, ref, err, dt, "y")
        assert torch.equal(y, want)
    assert min(times) < 5.0  # ms


def test_channels_beyond_31_bits_are_refused(cuda_lib):
    """Never cut down to their low bits."""
    D, w, A = 2 ** 32 + 64, torch.ones(64, 4, device="cuda"), -torch.ones(64, 16, device="cuda")
    x = torch.empty(1, 1, D, dtype=torch.bfloat16, device="cuda")
    s, h = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 64, 16, device="cuda")
    for call in (lambda: cuda_lib.gdn_short_conv_fwd(x, w), lambda: cuda_lib.gdn_short_conv_step(x[0], w, s)):
        with pytest.raises(ValueError, match=f"D = {D}"):
            call()
    bc = x[..., :16].contiguous()
    for call in (lambda: cuda_lib.gdn_s6_chunk_fwd(x, x, A, bc, bc),
                 lambda: cuda_lib.gdn_s6_recurrent_step(x[0], x[0], A, bc[0], bc[0], h),
                 lambda: cuda_lib.gdn_rms_norm_fwd(x, w[:, 0].contiguous())):
        with pytest.raises(ValueError):
            call()
