"""The layer operators' C entry points on the CPU: bad arguments are rejected before any
CUDA call, calls without work return GDN_OK, and the workspace size follows its layout."""
import pytest

A = 0x10000          # aligned fake addresses, far apart: never dereferenced
STEP = 0x100000000


def at(i, off=0):
    return A + i * STEP + off


@pytest.fixture(scope="module")
def lib():
    from linear_attention_prefill_gb300 import _build, binding
    _build.build()
    return binding.load_library()


def conv(lib, x=at(0), w=at(1), bias=None, s0=None, y=at(2), sT=None, N=1, T=8, D=16, W=4, stride=16,
         act=1, cu=None, f32=False):
    fn = lib.gdn_short_conv_fwd_f32 if f32 else lib.gdn_short_conv_fwd
    return fn(x, w, bias, s0, y, sT, N, T, D, W, stride, act, cu, None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(N=-1), 1), (dict(T=-1), 1),
    (dict(D=0), 1), (dict(W=1), 2), (dict(W=5), 2), (dict(act=2), 1), (dict(stride=15), 1),
    (dict(x=at(0, 1)), 1), (dict(w=at(1, 4)), 1), (dict(bias=at(3, 2)), 1), (dict(s0=at(3, 1)), 1),
    (dict(sT=at(3, 1)), 1), (dict(cu=at(4, 2)), 1), (dict(cu=at(4), N=0), 1),
    (dict(y=at(0)), 1), (dict(y=at(0, 128)), 1), (dict(s0=at(3), sT=at(3, 16)), 1),
    (dict(sT=at(0, 64)), 1), (dict(sT=at(2)), 1), (dict(s0=at(2)), 1),
    (dict(N=1 << 30, T=1 << 30), 1),
])
def test_conv_rejects(lib, case, status, f32):
    assert conv(lib, f32=f32, **case) == status
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", [
    dict(w=at(2)), dict(w=at(2, 16)), dict(bias=at(2, 4)), dict(cu=at(2)), dict(cu=at(2, 8), N=3),
    dict(sT=at(1)), dict(sT=at(1, 16)), dict(bias=at(3), sT=at(3)), dict(cu=at(4, 4), sT=at(4)),
    dict(cu=at(4), sT=at(4, 4), s0=at(5)),
])
def test_conv_outputs_on_parameters_or_borders(lib, case, f32):
    """y and sT may overlap no input: the filter, the bias and the borders are inputs too."""
    assert conv(lib, f32=f32, **case) == 1
    assert b"overlap" in lib.gdn_last_error()


def test_conv_step_outputs_on_parameters(lib):
    for fn in (lib.gdn_short_conv_step, lib.gdn_short_conv_step_f32):
        for w, bias, s, y in ((2, None, 3, 2), (1, 2, 3, 2), (3, None, 3, 2), (1, 3, 3, 2)):
            assert fn(at(0), at(w), bias and at(bias), at(s), at(y), 2, 16, 4, 16, 1, None) == 1
            assert b"overlap" in lib.gdn_last_error()


def test_conv_without_work(lib):
    assert conv(lib, N=0, T=0, x=None, y=None, w=None) == 0
    assert conv(lib, N=3, T=0, x=None, y=None, w=None) == 0


@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(s=None), 1), (dict(y=None), 1), (dict(N=-1), 1), (dict(W=6), 2),
    (dict(stride=4), 1), (dict(y=at(3)), 1), (dict(act=-1), 1),
])
def test_conv_step_rejects(lib, case, status):
    a = dict(x=at(0), w=at(1), s=at(3), y=at(2), N=2, D=16, W=4, stride=16, act=1)
    a.update(case)
    for fn in (lib.gdn_short_conv_step, lib.gdn_short_conv_step_f32):
        assert fn(a["x"], a["w"], None, a["s"], a["y"], a["N"], a["D"], a["W"], a["stride"], a["act"],
                  None) == status
    assert lib.gdn_short_conv_step(None, None, None, None, None, 0, 16, 4, 16, 1, None) == 0


S6 = dict(x=at(0), dt=at(1), A=at(2), B=at(3), C=at(4), D=at(5), z=at(6), bias=at(7), h0=at(8), y=at(9),
          hT=at(10), N=1, T=8, dim=32, Ns=16, xs=32, ds=32, bs=16, cs=16, zs=32, cu=None, ws=None, nws=0)


def s6(lib, f32=False, **kw):
    a = dict(S6, **kw)
    fn = lib.gdn_s6_chunk_fwd_f32 if f32 else lib.gdn_s6_chunk_fwd
    return fn(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["h0"], a["y"], a["hT"],
              a["N"], a["T"], a["dim"], a["Ns"], a["xs"], a["ds"], a["bs"], a["cs"], a["zs"], 1, a["cu"],
              a["ws"], a["nws"], None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1),
    (dict(y=None), 1), (dict(N=-1), 1), (dict(T=-1), 1), (dict(dim=0), 1), (dict(Ns=0), 1), (dict(Ns=65), 2),
    (dict(xs=31), 1), (dict(ds=1), 1), (dict(bs=15), 1), (dict(cs=0), 1), (dict(zs=-32), 1),
    (dict(x=at(0, 1)), 1), (dict(A=at(2, 8)), 1), (dict(h0=at(8, 4)), 1), (dict(hT=at(10, 8)), 1),
    (dict(D=at(5, 2)), 1), (dict(bias=at(7, 1)), 1), (dict(cu=at(11, 1)), 1), (dict(cu=at(11), N=0), 1),
    (dict(y=at(0)), 1), (dict(y=at(1, 64)), 1), (dict(y=at(8)), 1), (dict(hT=at(9)), 1), (dict(hT=at(2)), 1),
    (dict(hT=at(8, 16)), 1),
    (dict(T=4096, ws=at(12), nws=16), 1), (dict(T=4096, ws=at(12, 16), nws=1 << 40), 1),
])
def test_s6_rejects(lib, case, status, f32):
    assert s6(lib, f32=f32, **case) == status
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", [dict(cu=at(9)), dict(cu=at(9, 64)), dict(cu=at(10)), dict(cu=at(10, 16), N=2)])
def test_s6_outputs_on_borders(lib, case, f32):
    assert s6(lib, f32=f32, **case) == 1
    assert b"overlap" in lib.gdn_last_error()


def test_s6_without_work(lib):
    assert s6(lib, N=0, T=0) == 0
    assert s6(lib, N=2, T=0, hT=None, h0=None) == 0


@pytest.mark.parametrize("case,status", [(dict(h=None), 1), (dict(x=None), 1), (dict(Ns=100), 2),
                                         (dict(h=at(8, 4)), 1), (dict(y=at(8)), 1), (dict(N=-2), 1)])
def test_s6_step_rejects(lib, case, status):
    a = dict(S6, h=at(8), N=2)
    a.update(case)
    for fn in (lib.gdn_s6_recurrent_step, lib.gdn_s6_recurrent_step_f32):
        assert fn(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["h"], a["y"], a["N"],
                  a["dim"], a["Ns"], a["xs"], a["ds"], a["bs"], a["cs"], a["zs"], 1, None) == status


def test_s6_workspace_size(lib):
    size = lib.gdn_s6_chunk_fwd_workspace_size
    assert size(1, 4096, 4864, 16, 0) == 0 and size(64, 64, 64, 16, 0) == 0  # whole sequences
    for N, T, dim, Ns, packed in ((1, 65536, 2048, 16, 0), (2, 3000, 33, 7, 0), (3, 9001, 100, 16, 1),
                                  (1, 4096, 5120, 16, 0)):
        got = size(N, T, dim, Ns, packed)
        # of the split channels (all, or those behind whole 32-channel tiles): slots x (steps' sum,
        # states) and a copy of the states, each piece 256-byte aligned
        up = lambda v: -(-v // 64) * 64  # noqa: E731
        assert got > 0 and got % 4 == 0 and any(
            got == 4 * (up(s * d) + up(s * d * Ns) + N * d * Ns)
            for s in range(N, 32 * N + N + 2) for d in {dim, dim - 32 * 152} if d > 0)
    assert size(-1, 64, 64, 16, 0) == 0 and size(1, 4096, 64, 65, 0) == 0


def test_s6_workspace_size_of_more_sequences_than_tokens(lib):
    """Packed batches may hold empty sequences, any number of them: every size has an answer."""
    size = lib.gdn_s6_chunk_fwd_workspace_size
    for packed in (0, 1):
        for dim in (1, 64, 1216, 1217):
            for N in list(range(1, 20)) + [31, 64, 127, 152, 200, 299, 1000]:
                for T in list(range(0, 20)) + [31, 64, 127, 128, 129, 150, 255, 257, 300]:
                    got = size(N, T, dim, 16, packed)
                    assert got >= 0
                    if N > T and T <= 128:  # no sequence is longer than a chunk
                        assert got == 0
    # 150 tokens among 200 sequences, in chunks of 128: 1 + 200 + 1 slots
    assert size(200, 150, 64, 16, 1) == 4 * (202 * 64 + 202 * 64 * 16 + 200 * 64 * 16)


NORM = dict(x=at(0), w=at(1), res=None, gate=None, y=at(2), out=None, scales=at(3), tokens=4, heads=1, D=64,
            xs=64, gs=64, group=32, eps=1e-6)


def norm(lib, fp8=False, f32=False, **kw):
    a = dict(NORM, **kw)
    head = (a["x"], a["w"], a["res"], a["gate"], a["y"])
    size = (a["tokens"], a["heads"], a["D"], a["xs"], a["gs"])
    if fp8:
        fn = lib.gdn_rms_norm_fwd_e4m3_f32 if f32 else lib.gdn_rms_norm_fwd_e4m3
        return fn(*head, a["scales"], a["out"], *size, a["group"], a["eps"], None)
    fn = lib.gdn_rms_norm_fwd_f32 if f32 else lib.gdn_rms_norm_fwd
    return fn(*head, a["out"], *size, a["eps"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(tokens=-1), 1), (dict(heads=0), 1),
    (dict(D=0), 1), (dict(D=32769, xs=32769), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(xs=63), 1), (dict(gate=at(5), gs=10), 1), (dict(res=at(4)), 1), (dict(out=at(4)), 1),
    (dict(x=at(0, 1)), 1), (dict(w=at(1, 2)), 1), (dict(res=at(4, 1), out=at(5)), 1),
    (dict(y=at(0)), 1), (dict(res=at(4), out=at(4, 32)), 1), (dict(res=at(4), out=at(0)), 1),
    (dict(res=at(2), out=at(2)), 1), (dict(tokens=1 << 40), 1), (dict(heads=1 << 20, D=32768), 1),
    (dict(tokens=1, heads=1 << 16, D=32768, xs=1 << 31), 1),
])
def test_norm_rejects(lib, case, status, fp8, f32):
    assert norm(lib, fp8, f32, **case) == status
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("f32", [False, True])
def test_sizes_next_to_31_bits(lib, f32):
    """Sizes whose roundings up pass 31 bits are refused, before any launch."""
    most = 2 ** 31 - 1
    fn = lib.gdn_short_conv_step_f32 if f32 else lib.gdn_short_conv_step
    assert fn(at(0), at(10), None, at(20), at(40), most, 1, 2, 1, 1, None) == 1
    a = [at(8 * i) for i in range(12)]
    fn = lib.gdn_s6_recurrent_step_f32 if f32 else lib.gdn_s6_recurrent_step
    assert fn(*a[:5], None, None, None, a[8], a[9], most, 1, 1, 1, 1, 1, 1, 1, 1, None) == 1
    for dim in (most, 2 ** 30 + 1):
        assert s6(lib, f32, x=a[0], dt=a[1], A=a[2], B=a[3], C=a[4], D=None, z=None, bias=None, h0=None, y=a[9],
                  hT=a[10], T=1, dim=dim, Ns=1, xs=dim, ds=dim) == 1
    assert lib.gdn_s6_chunk_fwd_workspace_size(1, 1, most, 1, 0) == 0


def test_norm_e4m3_rejects(lib):
    assert norm(lib, True, scales=None) == 1 and norm(lib, True, group=48) == 2
    assert norm(lib, True, scales=at(2)) == 1 and norm(lib, True, scales=at(3, 2)) == 1
    assert norm(lib, True, tokens=0) == 0 and norm(lib, tokens=0, x=None, w=None, y=None) == 0


def test_binding_refuses_what_is_not_on_a_gpu(lib):
    import torch

    import linear_attention_prefill_gb300 as lap
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    A, B, h = torch.zeros(8, 16), torch.zeros(1, 4, 16), torch.zeros(1, 8, 16)
    for call in (lambda **k: lap.gdn_short_conv_fwd(x, w, **k),
                 lambda **k: lap.gdn_short_conv_step(x[:, 0], w, x[:, :3], **k),
                 lambda **k: lap.gdn_s6_chunk_fwd(x, x, A, B, B, **k),
                 lambda **k: lap.gdn_s6_recurrent_step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], h, **k),
                 lambda **k: lap.gdn_rms_norm_fwd(x, w[:, 0], **k)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(ValueError, match="CUDA"):
            call(stream=1)
    with pytest.raises(TypeError):
        lap.gdn_rms_norm_fwd([0.0], w[:, 0])
    with pytest.raises(ValueError):
        lap.gdn_short_conv_fwd(x, w, activation="relu")
    with pytest.raises(ValueError):
        lap.gdn_rms_norm_fwd(x, w[:, 0], group=32)
    with pytest.raises(TypeError):
        lap.gdn_rms_norm_fwd(x, w[:, 0], out_dtype=torch.float16)
