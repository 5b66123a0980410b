"""The layer operators around the linear-attention forwards, as measured cases.

gdn_short_conv_fwd / gdn_short_conv_step   depthwise short causal convolution with SiLU, prompts and one token
gdn_s6_chunk_fwd / gdn_s6_recurrent_step   selective state space scan (diagonal A per channel), prompts and one token
gdn_rms_norm_fwd                           RMS norm with the residual's addition or an output gate, 16-bit or e4m3 out

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is true, by
the calls of the package.  Packed batches carry sequence borders in an int32 ``cu`` as everywhere
in the package; inputs that a layer slices out of one projection are slices here too.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # q, k and v of a 16-head, 128-wide layer in one convolution over a 4K prompt, sliced out of
        # the projection that also holds the output gate's 2048 columns
        dict(name="conv_prompt_qkv", op="conv", tokens=4096, seqs=1, packed=False, D=6144, W=4, extra=2048,
             bias=False, silu=True, state=False, dtype="bf16"),
        # x, B and C of an 80-head scan layer (5120 + 2 * 128 columns), eight packed prompts that go on
        # from earlier ones
        dict(name="conv_prompt_ragged", op="conv", tokens=10007, seqs=8, packed=True, D=5376, W=4, extra=0,
             bias=True, silu=True, state=True, dtype="bf16"),
        # one user's decode token through a 16-qk-head, 32-v-head layer: latency
        dict(name="conv_step_1", op="conv_step", N=1, D=8192, W=4, extra=0, bias=False, silu=True, dtype="bf16"),
        # the same layer with 256 sequences in flight
        dict(name="conv_step_256", op="conv_step", N=256, D=8192, W=4, extra=4096, bias=False, silu=True,
             dtype="bf16"),
        # a 2.7B-class layer (5120 inner channels, 16 states each), 4K prompt
        dict(name="scan_prompt_4k", op="scan", tokens=4096, seqs=1, packed=False, D=5120, Ns=16, gate=True,
             skip=True, softplus=True, state=False, dtype="bf16"),
        # eight packed prompts of odd lengths resumed from states, in 32 bits
        dict(name="scan_prompt_ragged", op="scan", tokens=2777, seqs=8, packed=True, D=2049, Ns=16, gate=True,
             skip=True, softplus=True, state=True, dtype="f32"),
        # long context: 64K tokens of a narrow layer, where the channels alone do not fill the GPU
        dict(name="scan_prompt_64k", op="scan", tokens=65536, seqs=1, packed=False, D=2048, Ns=16, gate=True,
             skip=True, softplus=True, state=False, dtype="bf16"),
        # one decode token, one user: latency
        dict(name="scan_step_1", op="scan_step", N=1, D=5120, Ns=16, gate=True, skip=True, softplus=True,
             dtype="bf16"),
        # 128 sequences in flight: the states' traffic
        dict(name="scan_step_128", op="scan_step", N=128, D=5120, Ns=16, gate=True, skip=True, softplus=True,
             dtype="bf16"),
        # the norm before a layer's e4m3 projection while decoding 16 sequences, one scale a token
        dict(name="norm_fp8_step", op="norm", rows=16, D=2560, residual=True, gate=False, fp8=True, group=0,
             dtype="bf16"),
        # the gated norm of each 128-wide head of a 16-head layer's output, 4K prompt
        dict(name="norm_gated_heads", op="norm", rows=65536, D=128, residual=False, gate=True, fp8=False,
             group=0, dtype="bf16"),
        # the norm before a layer's e4m3 projection over two 4K prompts, a scale for every 128 columns
        dict(name="norm_fp8_prompt", op="norm", rows=8192, D=5120, residual=True, gate=False, fp8=True,
             group=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A channel count: mostly multiples of 64 as models have them, odd ones too."""
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.4 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "conv":
        D = _width(rng, 64, 8192)
        tokens = _log(rng, 1, min(65536, 67_000_000 // D))
        packed = rng.random() < 0.5
        seqs = rng.randint(1, min(16, tokens)) if packed else rng.choice([1, 1, 2, 4])
        return dict(op=op, tokens=tokens if packed else max(1, tokens // seqs) * seqs, seqs=seqs, packed=packed,
                    D=D, W=rng.choice([2, 3, 4, 4]), extra=rng.choice([0, 64, _log(rng, 1, 4096)]),
                    bias=rng.random() < 0.5, silu=rng.random() < 0.8, state=rng.random() < 0.5, dtype=dtype)
    if op == "conv_step":
        return dict(op=op, N=_log(rng, 1, 512), D=_width(rng, 64, 8192), W=rng.choice([2, 3, 4, 4]),
                    extra=rng.choice([0, 64, _log(rng, 1, 4096)]), bias=rng.random() < 0.5,
                    silu=rng.random() < 0.8, dtype=dtype)
    if op == "scan":
        Ns = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
        D = _width(rng, 64, 8192)
        tokens = _log(rng, 1, min(65536, 1_000_000_000 // (D * Ns)))
        packed = rng.random() < 0.5
        seqs = rng.randint(1, min(16, tokens)) if packed else rng.choice([1, 1, 2, 4])
        return dict(op=op, tokens=tokens if packed else max(1, tokens // seqs) * seqs, seqs=seqs, packed=packed,
                    D=D, Ns=Ns, gate=rng.random() < 0.7, skip=rng.random() < 0.7, softplus=rng.random() < 0.8,
                    state=rng.random() < 0.5, dtype=dtype)
    if op == "scan_step":
        return dict(op=op, N=_log(rng, 1, 256), D=_width(rng, 64, 8192),
                    Ns=rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)]), gate=rng.random() < 0.7,
                    skip=rng.random() < 0.7, softplus=rng.random() < 0.8, dtype=dtype)
    D = _width(rng, 64, 16384)
    fp8 = rng.random() < 0.5
    return dict(op=op, rows=_log(rng, 1, min(65536, 42_000_000 // D)), D=D, residual=rng.random() < 0.5,
                gate=rng.random() < 0.4, fp8=fp8, group=rng.choice([0, 32, 64, 128]) if fp8 else 0, dtype=dtype)


def _borders(case, seed):
    """Sequence borders of a prompt batch: random cuts for packed ones (empty sequences happen), rows else."""
    n, tokens = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [i * (tokens // n) for i in range(n + 1)]
    rng = random.Random(seed)
    return [0] + sorted(rng.randint(0, tokens) for _ in range(n - 1)) + [tokens]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, D = case["op"], case["D"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=dict(case))
    if op in ("conv", "scan"):
        borders = _borders(case, seed)
        s["cu"] = torch.tensor(borders, dtype=torch.int32, device=dev) if case["packed"] else None
        lead = (1, case["tokens"]) if case["packed"] else (case["seqs"], case["tokens"] // case["seqs"])
        n = case["seqs"]
    elif op != "norm":
        lead = (case["N"],)
        n = case["N"]
    if op in ("conv", "conv_step"):
        W = case["W"]
        # the projection's output; the convolution takes its first D columns
        s["x"] = randn(*lead, D + case["extra"], dtype=dt)[..., :D]
        s["weight"] = (rand(D, W) * 2 - 1) * W ** -0.5
        s["bias"] = (rand(D) * 2 - 1) * W ** -0.5 if case["bias"] else None
        s["s0"] = randn(n, W - 1, D, dtype=dt) if op == "conv_step" or case["state"] else None
    elif op in ("scan", "scan_step"):
        Ns, rank = case["Ns"], -(-D // 16)
        s["x"] = torch.nn.functional.silu(randn(*lead, D)).to(dt)
        s["z"] = randn(*lead, 2 * D, dtype=dt)[..., D:] if case["gate"] else None
        bc = randn(*lead, rank + 2 * Ns, dtype=dt)  # the projection that holds dt's low rank, B and C
        s["B"], s["C"] = bc[..., rank: rank + Ns], bc[..., rank + Ns:]
        # steps of 0.001 to 0.1 at dt = 0, spread evenly over the logarithm
        step = torch.exp(rand(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        if case["softplus"]:
            s["dt"], s["dt_bias"] = (0.5 * randn(*lead, D)).to(dt), step + torch.log(-torch.expm1(-step))
        else:
            s["dt"], s["dt_bias"] = (step * torch.exp(0.5 * randn(*lead, D))).to(dt), None
        s["A"] = -(1 + torch.arange(Ns, device=dev)) * torch.exp(0.1 * randn(D, Ns))
        s["D"] = 1 + 0.1 * randn(D) if case["skip"] else None
        s["h0"] = randn(n, D, Ns) * 0.1 if op == "scan_step" or case["state"] else None
    else:
        rows = case["rows"]
        s["x"] = randn(rows, D, dtype=dt)
        s["weight"] = 1 + 0.1 * randn(D)
        s["residual"] = (2 * randn(rows, D)).to(dt) if case["residual"] else None
        s["gate"] = randn(rows, D, dtype=dt) if case["gate"] else None
    return s


# ---- plain forms ---------------------------------------------------------------------


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))


def _rows_of(s, x):
    """The tokens as rows, the borders, and for each token its sequence and that sequence's first token."""
    flat = x.reshape(-1, x.shape[-1])
    cu = s["cu"]
    if cu is None:
        cu = torch.arange(x.shape[0] + 1, device=x.device) * x.shape[1]
    cu = cu.long()
    pos = torch.arange(flat.shape[0], device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), pos, right=True)
    return flat, cu, pos, seq, cu[seq]


def _plain_conv(s):
    case, x, W = s["case"], s["x"], s["case"]["W"]
    flat, cu, pos, seq, first = _rows_of(s, x)
    n, keep = cu.numel() - 1, W - 1
    s0 = s["s0"] if s["s0"] is not None else torch.zeros(n, keep, flat.shape[1], dtype=x.dtype, device=x.device)
    pool = torch.cat([s0.reshape(n * keep, -1), flat])  # states first, then the tokens
    taps = pos[:, None] - keep + torch.arange(W, device=x.device)
    src = torch.where(taps < first[:, None], seq[:, None] * keep + taps - first[:, None] + keep, n * keep + taps)
    y = (pool[src].float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["silu"]:
        y = _silu(y)
    seqs = torch.arange(n, device=x.device)[:, None]
    last = cu[1:, None] - keep + torch.arange(keep, device=x.device)
    src = torch.where(last < cu[:-1, None], seqs * keep + last - cu[:-1, None] + keep, n * keep + last)
    return y.to(x.dtype).reshape(x.shape), pool[src]


def _plain_conv_step(s):
    x, state = s["x"], s["s0"]
    window = torch.cat([state, x[:, None]], 1)  # [N, W, D]
    y = (window.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"]["silu"]:
        y = _silu(y)
    state.copy_(window[:, 1:])
    return y.to(x.dtype), state


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from h = 0, by pairs of neighbours."""
    n = a.shape[0]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = _linear_scan(a[1:m:2] * a[0:m:2], a[1:m:2] * b[0:m:2] + b[1:m:2])
    h = torch.empty_like(b)
    h[1:m:2] = odd
    h[0] = b[0]
    h[2::2] = a[2::2] * odd[: (n - 1) // 2] + b[2::2]
    return h


def _steps(s):
    d = s["dt"].float()
    if s["dt_bias"] is not None:
        d = d + s["dt_bias"]
    return _softplus(d) if s["case"]["softplus"] else d


def _plain_scan(s):
    x = s["x"]
    flat, cu, pos, seq, first = _rows_of(s, x)
    T, D = flat.shape
    u, delta = flat.float(), _steps(s).reshape(T, D)
    B, C = s["B"].float().reshape(T, -1), s["C"].float().reshape(T, -1)
    a = torch.exp(delta[:, :, None] * s["A"])
    b = (delta * u)[:, :, None] * B[:, None, :]
    starts, some = cu[:-1].clamp(max=T - 1), cu[1:] > cu[:-1]
    if s["h0"] is not None:  # a sequence's first token takes its state in, and nothing from before
        b.index_add_(0, starts, torch.where(some[:, None, None], a[starts] * s["h0"], 0.0))
    a[starts] = torch.where((first[starts] == starts)[:, None, None], 0.0, a[starts])
    h = _linear_scan(a, b)
    y = (h * C[:, None, :]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float().reshape(T, D))
    hT = h[(cu[1:] - 1).clamp(min=0)]
    hT = torch.where(some[:, None, None], hT, s["h0"] if s["h0"] is not None else torch.zeros_like(hT))
    return y.to(x.dtype).reshape(x.shape), hT


def _plain_scan_step(s):
    x, h = s["x"], s["h0"]
    u, delta = x.float(), _steps(s)
    new = torch.exp(delta[:, :, None] * s["A"]) * h + (delta * u)[:, :, None] * s["B"].float()[:, None, :]
    y = (new * s["C"].float()[:, None, :]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    h.copy_(new)
    return y.to(x.dtype), h


def _plain_norm(s):
    case, x = s["case"], s["x"]
    r = x.float()
    out = []
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out = [r.to(x.dtype)]
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    if not case["fp8"]:
        return [y.to(x.dtype)] + out
    rows, D = y.shape
    group = case["group"] or D
    parts = torch.nn.functional.pad(y, (0, -D % group)).reshape(rows, -1, group)
    amax = parts.abs().amax(-1)
    scale = torch.where(amax == 0, 1.0, amax / E4M3_MAX)
    q = (parts / scale[:, :, None]).reshape(rows, -1)[:, :D]
    return [q.to(torch.float8_e4m3fn), scale] + out


# ---- the package's calls -------------------------------------------------------------


def _own(s):
    import linear_attention_prefill_gb300 as lap
    case, op = s["case"], s["case"]["op"]
    if op == "conv":
        y, sT = lap.gdn_short_conv_fwd(s["x"], s["weight"], s["bias"], s["s0"],
                                       activation="silu" if case["silu"] else None, cu_seqlens=s["cu"])
        return y, sT
    if op == "conv_step":
        y = lap.gdn_short_conv_step(s["x"], s["weight"], s["s0"], s["bias"],
                                    activation="silu" if case["silu"] else None)
        return y, s["s0"]
    if op == "scan":
        return lap.gdn_s6_chunk_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                    s["h0"], dt_softplus=case["softplus"], cu_seqlens=s["cu"])
    if op == "scan_step":
        y = lap.gdn_s6_recurrent_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"], s["D"], s["z"],
                                      s["dt_bias"], dt_softplus=case["softplus"])
        return y, s["h0"]
    y, scale, res = lap.gdn_rms_norm_fwd(s["x"], s["weight"], s["residual"], s["gate"], eps=EPS,
                                         out_dtype=torch.float8_e4m3fn if case["fp8"] else None,
                                         group=case["group"] or None)
    return [t for t in (y, scale, res) if t is not None]


def run(state):
    if own:
        return _own(state)
    return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
            "scan_step": _plain_scan_step, "norm": _plain_norm}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    e, op, D = DTYPES[case["dtype"]].itemsize, case["op"], case["D"]
    if op in ("conv", "conv_step"):
        W = case["W"]
        t, n = (case["tokens"], case["seqs"]) if op == "conv" else (case["N"], case["N"])
        states = 1 + (op == "conv_step" or case["state"])
        return {"bytes": 2 * t * D * e + D * 4 * (W + case["bias"]) + states * n * (W - 1) * D * e,
                "flops": t * D * (2 * W + case["bias"] + 4 * case["silu"])}
    if op in ("scan", "scan_step"):
        Ns = case["Ns"]
        t, n = (case["tokens"], case["seqs"]) if op == "scan" else (case["N"], case["N"])
        states = 1 + (op == "scan_step" or case["state"])
        return {"bytes": t * D * e * (3 + case["gate"]) + 2 * t * Ns * e + states * n * D * Ns * 4
                + D * 4 * (Ns + case["skip"] + case["softplus"]),
                # per state: the exponent's product, the exponential, two multiply-adds, the input's product
                "flops": t * D * (7 * Ns + 1 + 4 * case["gate"] + 2 * case["skip"] + 4 * case["softplus"])}
    rows = case["rows"]
    out = 1 if case["fp8"] else e
    scales = rows * 4 * -(-D // (case["group"] or D)) if case["fp8"] else 0
    return {"bytes": rows * D * (e * (1 + 2 * case["residual"] + case["gate"]) + out) + scales + D * 4,
            "flops": rows * D * (4 + case["residual"] + 5 * case["gate"] + 2 * case["fp8"])}


# ---- the definitions in 64 bits ------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    x = f["x"]
    if op == "norm":
        r = x + f["residual"] if case["residual"] else x
        y = f["weight"] * r / (r.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
        if case["gate"]:
            y = y * f["gate"] * torch.sigmoid(f["gate"])
        tail = [r] if case["residual"] else []
        if not case["fp8"]:
            return [y] + tail
        width = case["group"] or case["D"]
        cols = [y[:, i: i + width] for i in range(0, case["D"], width)]
        tops = [c.abs().max(-1, keepdim=True).values / E4M3_MAX for c in cols]
        tops = [torch.where(t == 0, torch.ones_like(t), t) for t in tops]
        return [torch.cat([c / t for c, t in zip(cols, tops)], 1), torch.cat(tops, 1)] + tail  # before rounding
    if op in ("conv", "scan"):
        borders = _borders(case, seed)
        seqs = list(zip(borders[:-1], borders[1:]))
    else:
        seqs = [(i, i + 1) for i in range(case["N"])]
    x = x.reshape(-1, case["D"])
    if op in ("conv", "conv_step"):
        W, ys, lasts = case["W"], [], []
        if op == "conv_step":  # every sequence is one token
            full = torch.cat([f["s0"], x[:, None]], 1)
            ys, lasts = sum(full[:, j] * f["weight"][:, j] for j in range(W)), full[:, 1:]
        else:
            for i, (lo, hi) in enumerate(seqs):
                past = f["s0"][i] if f["s0"] is not None else x.new_zeros(W - 1, case["D"])
                full = torch.cat([past, x[lo:hi]])
                ys.append(sum(full[j: j + hi - lo] * f["weight"][:, j] for j in range(W)))
                lasts.append(full[full.shape[0] - (W - 1):])
            ys, lasts = torch.cat(ys), torch.stack(lasts)
        if case["bias"]:
            ys = ys + f["bias"]
        if case["silu"]:
            ys = ys * torch.sigmoid(ys)
        return ys.reshape(s["x"].shape), lasts
    delta = f["dt"].reshape(-1, case["D"])
    if case["softplus"]:
        delta = torch.logaddexp(delta + f["dt_bias"], torch.zeros_like(delta))
    B, C = f["B"].reshape(-1, 1, case["Ns"]), f["C"].reshape(-1, 1, case["Ns"])
    y = torch.empty_like(x)
    if op == "scan_step":
        h = torch.exp(delta[:, :, None] * f["A"]) * f["h0"] + (delta * x)[:, :, None] * B
        y, ends = (h * C).sum(-1), h
    else:
        ends = []
        for i, (lo, hi) in enumerate(seqs):  # token by token
            h = f["h0"][i] if f["h0"] is not None else x.new_zeros(case["D"], case["Ns"])
            for at in range(lo, hi, 64):
                end = min(at + 64, hi)
                a = torch.exp(delta[at:end, :, None] * f["A"])
                b = (delta[at:end] * x[at:end])[:, :, None] * B[at:end]
                for k in range(end - at):
                    h = torch.addcmul(b[k], a[k], h)
                    b[k] = h
                y[at:end] = (b * C[at:end]).sum(-1)
            ends.append(h)
        ends = torch.stack(ends)
    if case["skip"]:
        y = y + f["D"] * x
    if case["gate"]:
        z = f["z"].reshape(-1, case["D"])
        y = y * z * torch.sigmoid(z)
    return y.reshape(s["x"].shape), ends
