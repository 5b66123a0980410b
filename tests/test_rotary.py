"""Rotary positions: the table of frequencies on the CPU, the operator on the GPU, against the definition
in 64 bits (glr_ref.py)."""
import math

import pytest
import torch
from glr_ref import frequencies, rotate

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=32.0, original_length=4096)]


@pytest.fixture(scope="module")
def lap():
    import linear_attention_prefill_gb300 as lap
    from linear_attention_prefill_gb300 import _build
    _build.build()
    return lap


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("R", [2, 4, 10, 64, 128, 1024])
@pytest.mark.parametrize("base", [10000.0, 5e5, 100.0])
def test_turns(lap, scaling, R, base):
    turns, magnitude = lap.gdn_rotary_turns(R, base, device="cpu", **scaling)
    freq, mag = frequencies(R, base, **scaling)
    # a frequency is a 64-bit number with 53 bits, from a power that is within a few of its last ones
    want = freq / (2 * math.pi) * 2.0 ** 64
    assert turns.shape == (R // 2,) and turns.dtype == torch.int64
    assert ((turns.double() - want).abs() <= 2.0 ** -50 * want + 4).all()
    assert abs(magnitude - mag) <= 2.0 ** -23


def test_turns_refusals(lap):
    for kw in (dict(dim=0), dict(dim=1 << 21), dict(dim=8, scaling="cube")):
        with pytest.raises(ValueError):
            lap.gdn_rotary_turns(**{"device": "cpu", **kw})
    for kw in (dict(dim=7), dict(dim=1026), dict(dim=8, base=1.0), dict(dim=8, base=float("nan")),
               dict(dim=8, scaling="linear", factor=0.5), dict(dim=8, scaling="yarn", factor=2.0),
               dict(dim=8, scaling="yarn", factor=2.0, original_length=64, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(lap.GdnError):
            lap.gdn_rotary_turns(**{"device": "cpu", **kw})


def _gpu():
    from test_glr import DT, assert_within, gen_of, randn, sliced
    return DT, assert_within, gen_of, randn, sliced


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk,D,R", [(1, 0, 2, 2), (3, 1, 8, 4), (16, 4, 128, 128), (5, 5, 64, 32), (2, 1, 80, 40),
                                       (7, 3, 33, 10), (40, 8, 96, 24), (1, 1, 1024, 1024), (2, 2, 1023, 2),
                                       (3, 2, 256, 64), (4, 1, 24, 12)])
def test_prompt_and_gradient(cuda_lib, dtype, interleaved, Hq, Hk, D, R):
    DT, assert_within, gen_of, randn, sliced = _gpu()
    dt, gen = DT[dtype], gen_of(D + R)
    turns, mag = cuda_lib.gdn_rotary_turns(R, **SCALINGS[(Hq + D) % 4])
    freq, _ = frequencies(R, **SCALINGS[(Hq + D) % 4])
    for B, T, lens in ((1, 1, None), (3, 37, None), (1, 90, [3, 0, 50, 30])):
        q = randn(gen, B, T, Hq * D, dtype=dt)
        k = randn(gen, B, T, Hk * D, dtype=dt) if Hk else None
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda") if lens else None
        n = len(lens) if lens else B
        offsets = torch.randint(0, 1 << 30, (n,), generator=gen, device="cuda").to(torch.int32)
        if lens:
            pos = torch.cat([torch.arange(m) for m in lens] + [torch.zeros(T - sum(lens), dtype=torch.int64)])[None].cuda()
            far = pos + torch.cat([offsets.long().repeat_interleave(torch.tensor(lens, device="cuda")),
                                   torch.zeros(T - sum(lens), dtype=torch.int64, device="cuda")])
        else:
            pos = torch.arange(T, device="cuda").expand(B, T)
            far = pos + offsets.long()[:, None]
        end = sum(lens) if lens else T
        heads = lambda t, H: t if t is None else t.unflatten(-1, (H, D))  # noqa: E731
        for shift, off in ((0, None), (8, offsets), (3, offsets)):
            a = heads(sliced(q, shift, 8) if shift else q, Hq)
            b = heads(sliced(k, 2 * shift, 16) if shift and Hk else k, Hk)
            at = far if off is not None else pos
            for bwd in (False, True):
                call = cuda_lib.gdn_rotary_bwd if bwd else cuda_lib.gdn_rotary_fwd
                outs = call(a, b, turns, magnitude=mag, interleaved=interleaved, cu_seqlens=cu, offsets=off)
                for o, x in zip(outs, (heads(q, Hq), heads(k, Hk))):
                    if x is None:
                        assert o is None
                        continue
                    ref, err = rotate(x, at, freq, mag, interleaved, bwd)
                    assert_within(o[:, :end], ref[:, :end], err[:, :end], "rotated")
                    assert torch.equal(o[:, :end, :, R:], x[:, :end, :, R:])
                # positions say the same
                if end == T:
                    same = call(a, b, turns, at.to(torch.int32).contiguous(), magnitude=mag, interleaved=interleaved)
                    assert all(s is None or torch.equal(s, o) for s, o in zip(same, outs))
        # in place, q and k beside each other in one projection
        if Hk:
            proj = torch.cat([q, k, q], -1)
            a, b = heads(proj[..., :Hq * D], Hq), heads(proj[..., Hq * D:(Hq + Hk) * D], Hk)
            want = cuda_lib.gdn_rotary_fwd(a, b, turns, interleaved=interleaved, cu_seqlens=cu)
            qo, ko = cuda_lib.gdn_rotary_fwd(a, b, turns, q_out=a, k_out=b, interleaved=interleaved, cu_seqlens=cu)
            assert torch.equal(a[:, :end], want[0][:, :end]) and torch.equal(b[:, :end], want[1][:, :end])
            assert qo.data_ptr() == a.data_ptr() and ko.data_ptr() == b.data_ptr()
            assert torch.equal(a[:, end:], heads(q, Hq)[:, end:]) and torch.equal(proj[..., (Hq + Hk) * D:], q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_positions(cuda_lib, dtype):
    """Far, negative and repeated positions of single tokens."""
    DT, assert_within, gen_of, randn, _ = _gpu()
    gen, R = gen_of(3), 128
    turns, mag = cuda_lib.gdn_rotary_turns(R, **SCALINGS[3])
    freq, _ = frequencies(R, **SCALINGS[3])
    at = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9, 131072, 131072, 7], dtype=torch.int32, device="cuda")
    q, k = randn(gen, 9, 16, R, dtype=DT[dtype]), randn(gen, 9, 2, R, dtype=DT[dtype])
    for o, x in zip(cuda_lib.gdn_rotary_fwd(q, k, turns, at, magnitude=mag), (q, k)):
        assert_within(o, *rotate(x, at, freq, mag, False), "rotated")


@pytest.mark.gpu
def test_prompt_in_blocks_is_decode_and_undoes_itself(cuda_lib):
    DT, assert_within, gen_of, randn, _ = _gpu()
    gen = gen_of(4)
    turns, _ = cuda_lib.gdn_rotary_turns(64)
    q, k = randn(gen, 1, 2000, 8, 64), randn(gen, 1, 2000, 2, 64)
    off = torch.tensor([100000], dtype=torch.int32, device="cuda")
    qo, ko = cuda_lib.gdn_rotary_fwd(q, k, turns, offsets=off)
    at = (torch.arange(2000, device="cuda") + 100000).to(torch.int32)
    q1, k1 = cuda_lib.gdn_rotary_fwd(q[0], k[0], turns, at)
    assert torch.equal(q1, qo[0]) and torch.equal(k1, ko[0])
    back, _ = cuda_lib.gdn_rotary_bwd(qo, None, turns, offsets=off)
    # two turns of pairs, each with 8 roundings of its two terms (the angle is the same)
    assert ((back - q).abs() <= 24 * 2.0 ** -24 * (q.abs() + torch.cat([q[..., 32:], q[..., :32]], -1).abs())).all()


@pytest.mark.gpu
def test_streams_graphs_empty_and_far(cuda_lib):
    DT, assert_within, gen_of, randn, _ = _gpu()
    gen, bf = gen_of(5), torch.bfloat16
    turns, _ = cuda_lib.gdn_rotary_turns(128)
    q, k = randn(gen, 2, 300, 8, 128, dtype=bf), randn(gen, 2, 300, 2, 128, dtype=bf)
    want = cuda_lib.gdn_rotary_fwd(q, k, turns)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    got = cuda_lib.gdn_rotary_fwd(q, k, turns, stream=side)
    side.synchronize()
    with torch.cuda.graph(graph):
        replayed = cuda_lib.gdn_rotary_fwd(q, k, turns)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, replayed))
    assert cuda_lib.gdn_rotary_fwd(q[:, :0], None, turns)[0].numel() == 0
    x = torch.zeros(1, 131200, 128, 128, dtype=bf, device="cuda")  # more than 2^31 elements
    x[:, -2:] = q[:1, :2, :1]
    y, _ = cuda_lib.gdn_rotary_fwd(x, None, turns)
    freq, _ = frequencies(128)
    at = torch.tensor([[131198, 131199]], device="cuda")
    assert_within(y[:, -2:], *rotate(x[:, -2:], at, freq, 1.0, False), "rotated")


@pytest.mark.gpu
def test_binding_refusals(cuda_lib):
    dev, bf = "cuda", torch.bfloat16
    turns, _ = cuda_lib.gdn_rotary_turns(16)
    q, k = torch.zeros(1, 8, 4, 16, dtype=bf, device=dev), torch.zeros(1, 8, 2, 16, dtype=bf, device=dev)
    at = torch.zeros(1, 8, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 8], dtype=torch.int32, device=dev)
    f, err = cuda_lib.gdn_rotary_fwd, cuda_lib.GdnError
    for bad, fn in [
        (TypeError, lambda: f(q.half(), k, turns)), (TypeError, lambda: f(q, k.float(), turns)),
        (ValueError, lambda: f(q.cpu(), k, turns)), (ValueError, lambda: f(q, k[:, :4], turns)),
        (TypeError, lambda: f(q, k, turns.int())), (ValueError, lambda: f(q, k, turns[None])),
        (TypeError, lambda: f(q, k, turns, at.long())), (ValueError, lambda: f(q, k, turns, at[:, :4])),
        (ValueError, lambda: f(q, k, turns, at, cu_seqlens=cu)), (ValueError, lambda: f(q, k, turns, at, offsets=cu[:1])),
        (ValueError, lambda: f(q[0], k[0], turns)), (ValueError, lambda: f(q[0, 0], None, turns)),
        (ValueError, lambda: f(q, None, turns, k_out=k)), (ValueError, lambda: f(q, k[:, :, :0], turns)),
        (ValueError, lambda: f(q.transpose(1, 2), None, turns)), (err, lambda: f(q[..., :8].contiguous(), None, turns)),
        (err, lambda: f(q, k, turns, q_out=q.view(-1)[:512].view(1, 8, 4, 16), k_out=q.view(-1)[:256].view(1, 8, 2, 16))),
        (ValueError, lambda: f(q, k, turns, offsets=cu)), (err, lambda: f(q, k, turns[:0])),
    ]:
        with pytest.raises(bad):
            fn()
