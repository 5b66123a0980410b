"""The gated recurrence, layer norm and rotary positions as a layer runs them together: a block forwards and
backwards against 64 bits, and a rotated decayed attention from its prompt into decoding."""
import pytest
import torch
from glr_ref import frequencies, rotate
from test_glr import gen_of, randn

pytestmark = pytest.mark.gpu


def layer64(p, x, res, cu):
    """norm(x + res) -> a projection of inputs, gates and an output gate -> recurrence -> out, in 64 bits."""
    r = x + res
    h = torch.nn.functional.layer_norm(r, r.shape[-1:], p["w"], p["b"], 1e-5)
    u, g, z = (h @ p["in"]).split(p["rate"].numel(), -1)
    a = torch.exp(p["rate"] * torch.sigmoid(g))
    s = torch.sqrt(1 - a * a)
    ys = []
    for i in range(len(cu) - 1):
        state = p["h0"][i]
        for t in range(cu[i], cu[i + 1]):
            state = a[0, t] * state + s[0, t] * u[0, t]
            ys.append(state)
    y = torch.stack(ys)[None]
    return r + (y * z) @ p["out"]


def test_block_and_its_gradients(cuda_lib):
    """Layer norm, the recurrence (of slices of one projection) and their gradients, with the products
    around them by torch, in fp32.

    Bound: a result is a chain of three operators and two products of 64 and 96 terms, over a memory of some
    tens of tokens: fewer than 1500 roundings of U = 2^-24, each of at most the largest magnitude of its
    tensor, so 1e-4 of that.
    """
    gen, D, C, cu = gen_of(1), 64, 96, [0, 70, 71, 200]
    T = cu[-1]
    p = dict(w=1 + 0.1 * randn(gen, D), b=0.1 * randn(gen, D), rate=-torch.exp(0.5 * randn(gen, C) - 2),
             h0=randn(gen, 3, C), out=randn(gen, C, D) * C ** -0.5)
    p["in"] = randn(gen, D, 3 * C) * D ** -0.5
    x, res, dout = randn(gen, 1, T, D), randn(gen, 1, T, D), randn(gen, 1, T, D)
    f = {k: v.double().requires_grad_() for k, v in p.items()}
    x64, res64 = x.double().requires_grad_(), res.double().requires_grad_()
    want = layer64(f, x64, res64, cu)
    (want * dout.double()).sum().backward()
    # forwards
    borders = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h, r = cuda_lib.gdn_layer_norm_fwd(x, p["w"], p["b"], res)
    proj = h @ p["in"]
    u, g, z = proj.split(C, -1)
    y, hT, states = cuda_lib.gdn_glr_chunk_fwd(u, g, p["rate"], p["h0"], gate="rate", input_norm="sqrt",
                                               cu_seqlens=borders, output_states=True)
    got = r + (y * z) @ p["out"]
    # backwards: the gradient arrives at r and at the branch
    dyz = dout @ p["out"].t()
    du, dg, drate, dh0 = cuda_lib.gdn_glr_chunk_bwd(dyz * z, u, g, states, p["rate"], p["h0"], gate="rate",
                                                    input_norm="sqrt", cu_seqlens=borders)
    dproj = torch.cat([du, dg, dyz * y], -1)
    dr, dw, db = cuda_lib.gdn_layer_norm_bwd(dproj @ p["in"].t(), r, p["w"], dout)
    pairs = dict(out=(got, want), dx=(dr, x64.grad), dres=(dr, res64.grad), dw=(dw, f["w"].grad), db=(db, f["b"].grad),
                 drate=(drate, f["rate"].grad), dh0=(dh0, f["h0"].grad),
                 din=(torch.einsum("btd,btc->dc", h, dproj), f["in"].grad),
                 dout=(torch.einsum("btc,btd->cd", y * z, dout), f["out"].grad))
    for name, (a, b) in pairs.items():
        b = b.detach()
        assert (a.double() - b).abs().max() <= 1e-4 * b.abs().max(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotated_prompt_goes_on_into_decoding(cuda_lib, dtype):
    """Rotary q and k before the decayed linear attention (ssd_chunk_fwd), a packed prompt resumed at offsets and
    then one token at a time, against the sum over pairs of positions in 64 bits (tolerance of the forwards:
    2e-2 of the RMS for bf16, 1e-4 for fp32; the rotation adds its rounding of q and k: 2^-8 each in
    bf16, within it)."""
    dt, gen, H, d, lens = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype], gen_of(2), 2, 64, [130, 67]
    cu = torch.tensor([0, 130, 197], dtype=torch.int32, device="cuda")
    T, steps = 197, 3
    unit = lambda *s: torch.nn.functional.normalize(randn(gen, *s), dim=-1).to(dt)  # noqa: E731
    q, k, v = unit(1, T, H, d), unit(1, T, H, d), randn(gen, 1, T, H, d, dtype=dt)
    q1, k1, v1 = unit(steps, 2, H, d), unit(steps, 2, H, d), randn(gen, steps, 2, H, d, dtype=dt)
    g = -0.05 * torch.ones(1, T, H, device="cuda")
    beta, g1, beta1 = torch.ones_like(g), -0.05 * torch.ones(2, H, device="cuda"), torch.ones(2, H, device="cuda")
    offsets = torch.tensor([100000, 3], dtype=torch.int32, device="cuda")
    turns, mag = cuda_lib.gdn_rotary_turns(32)  # half of each head
    freq, _ = frequencies(32)
    qr, kr = cuda_lib.gdn_rotary_fwd(q, k, turns, cu_seqlens=cu, offsets=offsets)
    o, h = cuda_lib.ssd_chunk_fwd(qr, kr, v, g, beta, cu_seqlens=cu)
    outs = []
    for i in range(steps):
        at = offsets + torch.tensor(lens, dtype=torch.int32, device="cuda") + i
        a, b = cuda_lib.gdn_rotary_fwd(q1[i], k1[i], turns, at)
        outs.append(cuda_lib.ssd_recurrent_step(a, b, v1[i], g1, beta1, h))
    tol = 2e-2 if dtype == "bf16" else 1e-4
    for n, (lo, hi) in enumerate(zip([0, 130], [130, 197])):
        qs, ks, vs = (torch.cat([t[0, lo:hi], t1[:, n]]).double() for t, t1 in ((q, q1), (k, k1), (v, v1)))
        m = qs.shape[0]
        pos = torch.arange(m, device="cuda") + int(offsets[n])
        qs, ks = rotate(qs, pos, freq, 1.0, False)[0], rotate(ks, pos, freq, 1.0, False)[0]
        i = torch.arange(m, device="cuda")
        decay = torch.where(i[:, None] >= i, torch.exp(-0.05 * (i[:, None] - i).double()), 0.0)
        want = torch.einsum("ihd,jhd,ij,jhe->ihe", qs, ks, decay, vs)
        got = torch.cat([o[0, lo:hi], torch.stack([t[n] for t in outs])]).double()
        half = torch.finfo(dt).eps / 2 * want.abs() if dtype == "bf16" else 0.0  # o's own rounding
        err = ((got - want).abs() - half).clamp(min=0).max() / want.square().mean().sqrt()
        assert err <= tol, (n, err)
