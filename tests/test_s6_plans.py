"""GPU tests of how the S6 scan divides a batch (whole sequences, chunks with summaries, both side
by side) against the recurrence in 64 bits, at batches that are hard on the division.

The bounds are those of tests/test_layer_ops.py, carried through the recurrence: u = 2^-24 is half
a unit of fp32 rounding, outputs are rounded once more to their storage type.
"""
import numpy as np
import pytest
import torch

from test_layer_ops import DT, U, assert_within, gen_of, s6_inputs, s6_ref, s6_run, spans_of

from linear_attention_prefill_gb300.workloads import cu_seqlens_of

pytestmark = pytest.mark.gpu


def borders_of(lens):
    return torch.from_numpy(cu_seqlens_of(lens)).cuda()


# ---- more sequences than tokens ------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,Ns", [(8, 16), (64, 5), (1250, 16)])  # the last: above 38 tiles of channels
@pytest.mark.parametrize("lens", [(0, 1), (0, 1, 0, 0, 1, 0), (0, 0, 0, 1), (1, 0, 2, 0, 0, 0, 0, 0),
                                  (0,) * 198 + (150, 0)])
def test_more_sequences_than_tokens(cuda_lib, dtype, dim, Ns, lens):
    dt, g, T = DT[dtype], gen_of(dim + len(lens)), sum(lens)
    x = s6_inputs(g, (1, T), len(lens), dim, Ns, dt)
    ry, ey, rh, eh = s6_ref(x, True, spans_of(lens, True, 1))
    y, hT = s6_run(cuda_lib, x, True, borders_of(lens))
    assert_within(y, ry, ey, dt, "y")
    assert_within(hT, rh, eh, torch.float32, "hT")
    empty = torch.from_numpy(np.asarray(lens) == 0).cuda()
    assert torch.equal(hT[empty], x["h0"][empty])
    h = x["h0"].clone()
    y2, _ = s6_run(cuda_lib, dict(x, h0=h), True, borders_of(lens), hT=h)
    assert torch.equal(h, hT) and torch.equal(y2, y)


def test_packed_batch_without_tokens(cuda_lib):
    x = s6_inputs(gen_of(1), (1, 0), 3, 40, 16, torch.bfloat16)
    y, hT = s6_run(cuda_lib, x, True, borders_of((0, 0, 0)))
    assert y.numel() == 0 and torch.equal(hT, x["h0"])


def test_convolution_of_more_sequences_than_tokens(cuda_lib):
    from test_layer_ops import conv_ref, randn
    for lens in ((0, 1, 0, 0, 1, 0), (0, 0, 0, 1), (0,) * 198 + (50, 0)):
        g = gen_of(len(lens))
        x, w = randn(g, 1, sum(lens), 72, dtype=torch.bfloat16), randn(g, 72, 4)
        s0 = randn(g, len(lens), 3, 72, dtype=torch.bfloat16)
        y, sT = cuda_lib.gdn_short_conv_fwd(x, w, s0=s0, cu_seqlens=borders_of(lens))
        ref, err, st = conv_ref(x, w, None, s0, "silu", spans_of(lens, True, 1))
        assert_within(y, ref, err, torch.bfloat16, "y")
        assert torch.equal(sT.double(), st)


# ---- infinite inputs -----------------------------------------------------------------


def positive_inputs(T, dim, Ns, dt):
    """Every term of every sum positive: an infinity stays one in the definition, it never meets its opposite."""
    g = gen_of(T + Ns)
    r = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.5  # noqa: E731
    return dict(x=r(1, T, dim).to(dt), dt=(0.01 * r(1, T, dim)).to(dt), A=-0.01 * r(dim, Ns), B=r(1, T, Ns).to(dt),
                C=r(1, T, Ns).to(dt), D=None, z=None, dt_bias=None, h0=None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [50, 1100])  # whole sequences, and split over time
@pytest.mark.parametrize("Ns", [1, 3, 4, 5, 8, 12, 16, 20, 24, 28, 30, 32, 40, 60, 64])
def test_infinities_stay_infinite_for_every_state_count(cuda_lib, dtype, T, Ns):
    """Lanes that hold no state, or fewer than four, add nothing, whatever the step."""
    for name in ("x", "dt"):
        x = positive_inputs(T, 64, Ns, DT[dtype])
        clean, hc = s6_run(cuda_lib, x, False)
        x[name][0, 20, 3] = float("inf")
        y, h = s6_run(cuda_lib, x, False)
        assert (y[0, 20:, 3] == float("inf")).all() and (h[0, 3] == float("inf")).all()
        y[0, 20:, 3], h[0, 3] = clean[0, 20:, 3], hc[0, 3]
        assert torch.equal(y, clean) and torch.equal(h, hc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Ns", [8, 12, 16])
def test_infinite_states_outlive_chunks_that_decay_to_nothing(cuda_lib, dtype, Ns):
    """exp(A times a chunk's steps) underflows where no token's decay does: infinity stays infinity."""
    dt, T = DT[dtype], 1500
    assert cuda_lib.gdn_s6_chunk_fwd_workspace_size(1, T, 64, Ns) > 0
    x = positive_inputs(T, 64, Ns, dt)
    x["A"], x["dt"] = 1000 * x["A"], 10 * x["dt"]  # decays of e^-0.25 to e^-2.25 a token, e^-32 or less over 128
    clean, hc = s6_run(cuda_lib, x, False)
    assert torch.isfinite(clean.float()).all() and torch.isfinite(hc).all()
    x["x"][0, 20, 3] = float("inf")
    y, h = s6_run(cuda_lib, x, False)
    assert (y[0, 20:, 3] == float("inf")).all() and (h[0, 3] == float("inf")).all()
    x["h0"] = torch.full((1, 64, Ns), float("-inf"), device="cuda")
    x["x"][0, 20, 3] = 0.5
    y, h = s6_run(cuda_lib, x, False)
    assert (y == float("-inf")).all() and (h == float("-inf")).all()
    x["dt"][0, 700, 5] = float("inf")  # a decay that is 0 for one token: 0 times infinity has no value
    y, h = s6_run(cuda_lib, x, False)
    assert torch.isnan(y[0, 700:, 5]).all() and torch.isnan(h[0, 5]).all()
    y[0, 700:, 5], h[0, 5] = float("-inf"), float("-inf")
    assert (y == float("-inf")).all() and (h == float("-inf")).all()


# ---- split scans, y and hT to the roundings of their own arithmetic ------------------


def plan_of(lib, N, T, dim, Ns, packed):
    """(channels that are split, most tokens of a chunk) of the plan whose workspace the library asks for:
    per slot of a chunk a sum and Ns states a split channel, and N copies of h0, in pieces of 64 floats;
    32-channel tiles that are not split come first.  A packed batch has T / chunk + N + 1 slots, rows
    have N ceil(T / chunk); no chunk is shorter than 128 tokens."""
    need = lib.gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, packed)
    up = lambda v: -(-v // 64) * 64  # noqa: E731
    found = []
    for w in range(dim, 0, -32):
        for slots in range(max(1, need // (4 * w * (Ns + 1)) - N - 130), need // (4 * w * (Ns + 1)) + 1):
            if 4 * (up(slots * w) + up(slots * w * Ns) + N * w * Ns) != need:
                continue
            chunks = slots - N - 1 if packed else slots // N - 1  # T / chunk, rounded down
            if 1 <= chunks <= T // 128 and (packed or slots % N == 0):
                found.append((w, T // chunks))
    assert found, need
    assert len({w for w, _ in found}) == 1, found
    return found[0][0], max(c for _, c in found)


def s6_ref_of_chunks(x, spans, chunk):
    """(y, bound of y, hT, bound of hT) of the recurrence in 64 bits, with dt_softplus, gate and skip.

    The bounds are s6_ref's, for every channel, state and token by itself.  A decay over a chunk is
    2^(A log2 e times the sum of its steps).  A thread adds up a quarter of the chunk's steps, all
    positive, and four such sums are added, so a sum is off by at most n = chunk / 4 + 4 roundings
    relative; that is n u |D_t A| on the decay of each of its tokens.  What else happens at a chunk's
    end (one product, 2^x, one multiply-add) a token's own bound has counted once for every token of
    the chunk."""
    f = {k: v.double() if v is not None else None for k, v in x.items()}
    y, ey = torch.zeros_like(f["x"]), torch.zeros_like(f["x"])
    hs, es, n = [], [], chunk / 4 + 4
    v = f["dt"] + f["dt_bias"]
    step, estep = torch.logaddexp(v, torch.zeros_like(v)), (3 * v.abs() + 8) * U
    Ns = f["A"].shape[1]
    for i, (b, lo, hi) in enumerate(spans):
        h = f["h0"][i].clone()
        mag, e = h.abs(), torch.zeros_like(h)
        for t in range(lo, hi):
            d, ed = step[b, t][:, None], estep[b, t][:, None]
            arg = d * f["A"]
            a = torch.exp(arg)
            u = d * f["x"][b, t][:, None] * f["B"][b, t]
            e = a * e + a * mag * (3 * U + arg.abs() * (ed + (3 + n) * U)) + u.abs() * (ed + 3 * U)
            h, mag = a * h + u, a * mag + u.abs()
            e = e + 2 * U * mag
            c = f["C"][b, t]
            y[b, t], ey[b, t] = h @ c, e @ c.abs() + (Ns + 2) * U * (mag @ c.abs())
        hs.append(h)
        es.append(e)
    skip, s = f["D"] * f["x"], f["z"] * torch.sigmoid(f["z"])
    y, ey = y + skip, ey + 2 * U * skip.abs()
    ey = ey * s.abs() + (8 + 2 * f["z"].abs()) * U * (y * s).abs()
    return y * s, 2 * ey, torch.stack(hs), 2 * torch.stack(es)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,dim,Ns,whole", [
    # every channel split
    ((2085,), False, 64, 16, False), ((1300, 0, 2, 1700), True, 40, 16, False), ((1111, 1111), False, 33, 7, False),
    ((1500,), False, 16, 64, False), ((8950,), False, 32, 16, False), ((4500, 7, 4400), True, 31, 32, False),
    ((1600,), False, 40, 24, False), ((1600,), False, 36, 12, False),
    # one long sequence among short ones, empty ones before, between and behind
    ((700,) + (5,) * 15, True, 40, 16, False), ((0,) * 9 + (3,) * 30 + (1400, 0, 0, 33, 0), True, 96, 16, False),
    ((900, 40) + (9,) * 40, True, 33, 19, False),
    # whole channels beside split ones: one sequence, several rows, packed ones with empty ones among them
    ((1100,), False, 4900, 16, True), ((1100, 1100), False, 2460, 16, True), ((1100, 1100), False, 2433, 8, True),
    ((1500, 0, 700), True, 1630, 16, True), ((0, 1200, 1000), True, 1625, 24, True),
    ((800, 700, 0, 900), True, 1230, 5, True),
])
def test_split_scans_to_their_roundings(cuda_lib, dtype, lens, packed, dim, Ns, whole):
    dt, g = DT[dtype], gen_of(dim + Ns + len(lens))
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    split, chunk = plan_of(cuda_lib, len(lens), T, dim, Ns, packed)
    assert (split < dim) == whole and chunk < max(lens)
    cu = borders_of(lens) if packed else None
    x = s6_inputs(g, (B, T), len(lens), dim, Ns, dt)
    ry, ey, rh, eh = s6_ref_of_chunks(x, spans_of(lens, packed, B), chunk)
    y, hT = s6_run(cuda_lib, x, True, cu)
    assert_within(y, ry, ey, dt, "y")
    assert_within(hT, rh, eh, torch.float32, "hT")
    h = x["h0"].clone()  # in place: whole channels, first and last chunks and empty sequences at once
    y2, h2 = s6_run(cuda_lib, dict(x, h0=h), True, cu, hT=h)
    assert h2.data_ptr() == h.data_ptr() and torch.equal(h, hT) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_split_scan_is_its_pieces(cuda_lib, dtype):
    """One split call against the same tokens in calls too short to be split, each from the last one's state."""
    dt, T, dim, Ns, n = DT[dtype], 2000, 48, 16, 125
    x = s6_inputs(gen_of(5), (1, T), 1, dim, Ns, dt)
    _, chunk = plan_of(cuda_lib, 1, T, dim, Ns, False)
    assert cuda_lib.gdn_s6_chunk_fwd_workspace_size(1, n, dim, Ns) == 0
    y, hT = s6_run(cuda_lib, x, True)
    parts, h = [], x["h0"]
    for t in range(0, T, n):
        piece = {k: v[:, t:t + n].contiguous() if k in ("x", "dt", "z", "B", "C") else v for k, v in x.items()}
        part, h = s6_run(cuda_lib, dict(piece, h0=h), True)
        parts.append(part)
    _, ey, _, eh = s6_ref_of_chunks(x, [(0, 0, T)], chunk)
    # either side is within the bound and one rounding of the definition
    assert_within(y, torch.cat(parts, 1).double(), 2 * ey + torch.finfo(dt).eps / 2 * y.double().abs(), dt, "y")
    assert_within(hT, h.double(), 2 * eh, torch.float32, "hT")
