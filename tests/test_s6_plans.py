"""GPU tests of how the S6 scan divides a batch (whole sequences, chunks with summaries, both side
by side) against the recurrence in 64 bits, at batches that are hard on the division.

The bounds are those of tests/test_layer_ops.py, carried through the recurrence: u = 2^-24 is half
a unit of fp32 rounding, outputs are rounded once more to their storage type.
"""
import numpy as np
import pytest
import torch

from test_layer_ops import DT, assert_within, gen_of, s6_inputs, s6_ref, s6_run, spans_of

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
