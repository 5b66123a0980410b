"""The gated linear recurrence, layer norm and rotary positions, as measured cases.

gdn_glr_chunk_fwd / gdn_glr_recurrent_step   h_t = a_t h_{t-1} + b_t per channel, prompts and one token
gdn_glr_chunk_bwd                            its gradient, from the states that the forward leaves
gdn_layer_norm_fwd / gdn_layer_norm_bwd      layer norm with the residual's addition, and its gradient
gdn_rotary_fwd / gdn_rotary_bwd              rotary positions of q and k, both layouts, and the gradient

``run`` computes them from elementary torch operations in 32 bits (angles in 64), or, where ``own``
is true, by the calls of the package.  Packed batches carry sequence borders in an int32 ``cu`` as
everywhere in the package; inputs that a layer slices out of one projection are slices here too.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CHUNK = 64  # tokens between the states that the recurrence's forward leaves for its backward


def listed():
    return [
        # long context: 64K tokens of a 2560-channel layer, raw gates, inputs weighted with 1 - a
        dict(name="glr_prompt_64k", op="glr", tokens=65536, seqs=1, packed=False, D=2560, gate="sigmoid",
             norm="linear", state=False, keep=False, dtype="bf16"),
        # eight packed prompts of odd lengths resumed from states, in 32 bits, states kept for a backward
        dict(name="glr_prompt_ragged", op="glr", tokens=2777, seqs=8, packed=True, D=2049, gate="log", norm="none",
             state=True, keep=True, dtype="f32"),
        # one decode token of 64 sequences: latency
        dict(name="glr_step_64", op="glr_step", N=64, D=2560, gate="rate", norm="sqrt", dtype="bf16"),
        # training: eight rows of 2048 tokens, a learned rate for each channel, inputs kept at unit variance
        dict(name="glr_train_2k", op="glr_bwd", tokens=16384, seqs=8, packed=False, D=2560, gate="rate", norm="sqrt",
             state=False, dtype="bf16"),
        # training on five packed documents of odd lengths with states in and out, an odd number of channels
        dict(name="glr_train_ragged", op="glr_bwd", tokens=10007, seqs=5, packed=True, D=1111, gate="log",
             norm="linear", state=True, dtype="bf16"),
        # the norm before a layer while decoding 16 sequences: latency
        dict(name="norm_step", op="ln", rows=16, D=2560, residual=True, affine=True, dtype="bf16"),
        # the norm before a layer over two 4K prompts, with the residual
        dict(name="norm_prompt", op="ln", rows=8192, D=5120, residual=True, affine=True, dtype="bf16"),
        # its gradient in training, added to the residual's
        dict(name="norm_train", op="ln_bwd", rows=8192, D=5120, residual=True, affine=True, dtype="bf16"),
        # odd sizes in 32 bits
        dict(name="norm_train_odd", op="ln_bwd", rows=4099, D=1111, residual=False, affine=True, dtype="f32"),
        # q and k of a 16-head, 128-wide layer over a 4K prompt, sliced out of the projection that holds v too
        dict(name="rotary_prompt", op="rotary", tokens=4096, seqs=1, packed=False, Hq=16, Hk=16, D=128, R=128,
             interleaved=False, scaling="none", extra=2048, backward=False, dtype="bf16"),
        # the gradient over two packed 4K documents, half of each head rotated, neighbours paired
        dict(name="rotary_train", op="rotary", tokens=8192, seqs=2, packed=True, Hq=16, Hk=16, D=128, R=64,
             interleaved=True, scaling="linear", extra=0, backward=True, dtype="bf16"),
        # one decode token of 128 sequences at far positions, frequencies stretched by parts
        dict(name="rotary_step", op="rotary_step", N=128, Hq=16, Hk=4, D=128, R=128, interleaved=False,
             scaling="yarn", extra=512, backward=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A channel count: mostly multiples of 64 as models have them, odd ones too."""
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.4 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["glr", "glr", "glr_bwd", "glr_bwd", "glr_step", "ln", "ln_bwd", "ln_bwd", "rotary", "rotary",
                     "rotary_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("glr", "glr_bwd"):
        D = _width(rng, 64, 8192)
        tokens = _log(rng, 1, min(65536, (80_000_000 if op == "glr" else 40_000_000) // D))
        packed = rng.random() < 0.5
        seqs = rng.randint(1, min(16, tokens)) if packed else rng.choice([1, 1, 2, 4, 8])
        c = dict(op=op, tokens=tokens if packed else max(1, tokens // seqs) * seqs, seqs=seqs, packed=packed, D=D,
                 gate=rng.choice(["log", "sigmoid", "rate"]), norm=rng.choice(["none", "linear", "sqrt"]),
                 state=rng.random() < 0.5, dtype=dtype)
        return dict(c, keep=rng.random() < 0.5) if op == "glr" else c
    if op == "glr_step":
        return dict(op=op, N=_log(rng, 1, 512), D=_width(rng, 64, 8192), gate=rng.choice(["log", "sigmoid", "rate"]),
                    norm=rng.choice(["none", "linear", "sqrt"]), dtype=dtype)
    if op in ("ln", "ln_bwd"):
        D = _width(rng, 64, 16384)
        return dict(op=op, rows=_log(rng, 1, min(65536, 42_000_000 // D)), D=D, residual=rng.random() < 0.5,
                    affine=rng.random() < 0.8, dtype=dtype)
    D = rng.choice([64, 128, 128, 256, 2 * rng.randint(8, 128)])
    R = rng.choice([D, D, D // 2 // 2 * 2, D // 4 // 2 * 2])
    Hq = rng.choice([1, 4, 8, 16, 32, rng.randint(1, 40)])
    c = dict(op=op, Hq=Hq, Hk=rng.choice([0, 1, max(1, Hq // 4), Hq]), D=D, R=R, interleaved=rng.random() < 0.5,
             scaling=rng.choice(["none", "linear", "ntk", "yarn"]), extra=rng.choice([0, 64, _log(rng, 1, 4096)]),
             backward=rng.random() < 0.4, dtype=dtype)
    if op == "rotary_step":
        return dict(c, N=_log(rng, 1, 512))
    tokens = _log(rng, 1, min(65536, 80_000_000 // (D * 2 * Hq)))
    packed = rng.random() < 0.5
    seqs = rng.randint(1, min(16, tokens)) if packed else rng.choice([1, 1, 2, 4])
    return dict(c, tokens=tokens if packed else max(1, tokens // seqs) * seqs, seqs=seqs, packed=packed)


def _borders(case, seed):
    """Sequence borders of a prompt batch: random cuts for packed ones (empty sequences happen), rows else."""
    n, tokens = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [i * (tokens // n) for i in range(n + 1)]
    rng = random.Random(seed)
    return [0] + sorted(rng.randint(0, tokens) for _ in range(n - 1)) + [tokens]


def _scaling(case):
    """The stretch of a case's frequencies: keywords of gdn_rotary_turns."""
    return {"none": dict(scaling=None), "linear": dict(scaling="linear", factor=4.0),
            "ntk": dict(scaling="ntk", factor=8.0),
            "yarn": dict(scaling="yarn", factor=32.0, original_length=4096)}[case["scaling"]]


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
    if op in ("glr", "glr_bwd", "rotary"):
        borders = _borders(case, seed)
        n = case["seqs"]
        s["cu"] = torch.tensor(borders, dtype=torch.int32, device=dev) if case["packed"] else None
        lead = (1, case["tokens"]) if case["packed"] else (n, case["tokens"] // n)
    elif op in ("glr_step", "rotary_step"):
        n = case["N"]
        lead = (n,)
    if op in ("glr", "glr_bwd", "glr_step"):
        xg = randn(*lead, 2 * D, dtype=dt)  # the projection that holds the inputs and the gates
        if case["gate"] == "log":  # decays of 0.6 to 0.999
            xg[..., D:] = -torch.nn.functional.softplus(randn(*lead, D) - 2).to(dt)
        elif case["gate"] == "sigmoid":  # forget gates that mostly keep
            xg[..., D:] = (randn(*lead, D) + 2).to(dt)
        s["x"], s["g"] = xg[..., :D], xg[..., D:]
        # a learned rate: a decay of 0.9 to 0.999 at an open gate
        s["rate"] = 8 * torch.log(0.9 + 0.099 * rand(D)) if case["gate"] == "rate" else None
        s["h0"] = randn(n, D) if op == "glr_step" or case["state"] else None
        if op == "glr_bwd":
            s["dy"] = randn(*lead, D, dtype=dt)
            s["dhT"] = randn(n, D) if case["state"] else None
            s["states"] = _every(s, _plain_states(s))
    elif op in ("ln", "ln_bwd"):
        rows = case["rows"]
        # a residual stream: channels with means of their own
        s["x"] = (randn(rows, D) + randn(D)).to(dt)
        s["weight"] = 1 + 0.1 * randn(D) if case["affine"] else None
        s["bias"] = 0.1 * randn(D) if case["affine"] else None
        s["residual"] = (2 * randn(rows, D)).to(dt) if case["residual"] else None  # backward: its gradient
        s["dy"] = randn(rows, D, dtype=dt) if op == "ln_bwd" else None
    else:
        Hq, Hk = case["Hq"], case["Hk"]
        proj = randn(*lead, (Hq + Hk) * D + case["extra"], dtype=dt)
        s["q"] = proj[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = proj[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)) if Hk else None
        # prompts go on from what their sequences hold already; decode tokens lie anywhere up to 2^20
        key = "positions" if op == "rotary_step" else "offsets"
        top = 1 << 20 if op == "rotary_step" else 1 << 15
        s[key] = torch.randint(0, top, (n,), generator=gen, device=dev).to(torch.int32)
        s["freq"], s["magnitude"] = _frequencies(case, dev)
        if own:
            import linear_attention_prefill_gb300 as lap
            s["turns"], s["magnitude"] = lap.gdn_rotary_turns(case["R"], 10000.0, device=dev, **_scaling(case))
    return s


# ---- plain forms ---------------------------------------------------------------------


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


def _layout(s, x):
    """The borders, and for each token (as one row of tokens) its sequence."""
    cu = s["cu"]
    if cu is None:
        cu = torch.arange(x.shape[0] + 1, device=x.device) * x.shape[1]
    cu = cu.long()
    pos = torch.arange(x.shape[0] * x.shape[1], device=x.device)
    return cu, pos, torch.searchsorted(cu[1:].contiguous(), pos, right=True)


def _gates(s):
    """(decay a, 1 - a or 1 - a^2, sigmoid of g, 1 - sigmoid of g), without cancellation."""
    kind, norm, g = s["case"]["gate"], s["case"]["norm"], s["g"].float()
    sig, rest = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    if kind == "sigmoid":
        return sig, rest * (1 + sig) if norm == "sqrt" else rest, sig, rest
    log = g if kind == "log" else s["rate"] * sig
    return torch.exp(log), -torch.expm1(2 * log if norm == "sqrt" else log), sig, rest


def _weights(s):
    """(a, the input's weight)."""
    a, left, _, _ = _gates(s)
    norm = s["case"]["norm"]
    return a, torch.ones_like(a) if norm == "none" else left if norm == "linear" else torch.sqrt(left)


def _cut(s, x, a, b):
    """Tokens as rows; a sequence's first token takes its state in, and nothing from before."""
    cu, pos, seq = _layout(s, x)
    D = x.shape[-1]
    a, b = a.reshape(-1, D), b.reshape(-1, D)
    first = pos == cu[seq]
    if s["h0"] is not None:
        b = torch.where(first[:, None], b + a * s["h0"][seq], b)
    return torch.where(first[:, None], 0.0, a), b, cu, seq, first


def _plain_states(s):
    x = s["x"]
    a, w = _weights(s)
    a, b, *_ = _cut(s, x, a, w * x.float())
    return _linear_scan(a, b).reshape(x.shape)


def _every(s, h):
    """The state before every 64th token of each row."""
    kept = torch.zeros(h.shape[0], -(-h.shape[1] // CHUNK), h.shape[2], device=h.device)
    kept[:, 1:] = h[:, CHUNK - 1:-1:CHUNK]
    if s["cu"] is None and s["h0"] is not None:
        kept[:, 0] = s["h0"]
    return kept


def _plain_glr(s):
    x = s["x"]
    h = _plain_states(s)
    cu, _, _ = _layout(s, x)
    hT = h.reshape(-1, x.shape[-1])[(cu[1:] - 1).clamp(min=0)]
    empty = s["h0"] if s["h0"] is not None else torch.zeros_like(hT)
    hT = torch.where((cu[1:] > cu[:-1])[:, None], hT, empty)
    out = [h.to(x.dtype), hT]
    return out + [_every(s, h)] if s["case"]["keep"] else out


def _plain_step(s):
    a, w = _weights(s)
    s["h0"].copy_(a * s["h0"] + w * s["x"].float())
    return s["h0"].to(s["x"].dtype), s["h0"]


def _plain_glr_bwd(s):
    x, norm, kind = s["x"], s["case"]["norm"], s["case"]["gate"]
    D = x.shape[-1]
    a, left, sig, rest = (t.reshape(-1, D) for t in _gates(s))
    w = torch.ones_like(a) if norm == "none" else left if norm == "linear" else torch.sqrt(left)
    xf, dy = x.float().reshape(-1, D), s["dy"].float().reshape(-1, D)
    cut, b, cu, seq, first = _cut(s, x, a, w * xf)
    h = _linear_scan(cut, b)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    start = s["h0"][seq] if s["h0"] is not None else torch.zeros_like(h)
    before = torch.where(first[:, None], start, before)
    last = torch.cat([first[1:], torch.ones_like(first[:1])])
    if s["dhT"] is not None:
        dy = torch.where(last[:, None], dy + s["dhT"][seq], dy)
    # backwards over the row: what a token gets from the next one
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
    lam = _linear_scan(torch.where(last[:, None], 0.0, nxt).flip(0), dy.flip(0)).flip(0)
    to_log = a * before
    if norm == "linear":
        to_log = to_log - a * xf
    elif norm == "sqrt":
        to_log = to_log - torch.where(w > 0, a * a / w, 0.0) * xf
    to_log = lam * to_log
    if kind == "log":
        dg, drate = to_log, None
    elif kind == "sigmoid":
        dg, drate = to_log * rest, None
    else:
        dg, drate = to_log * s["rate"] * sig * rest, (to_log * sig).double().sum(0).float()
    out = [(w * lam).to(x.dtype).reshape(x.shape), dg.to(x.dtype).reshape(x.shape)]
    if drate is not None:
        out.append(drate)
    if s["h0"] is not None:
        mu = (a * lam)[cu[:-1].clamp(max=a.shape[0] - 1)]
        out.append(torch.where((cu[1:] > cu[:-1])[:, None], mu, s["dhT"]))
    return out


def _plain_ln(s):
    x, out = s["x"], []
    r = x.float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out = [r.to(x.dtype)]
    c = r - r.mean(-1, keepdim=True)
    y = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return [y.to(x.dtype)] + out


def _plain_ln_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    xh = c * rstd
    u = dy * s["weight"] if s["weight"] is not None else dy
    dx = rstd * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    out = [dx.to(s["x"].dtype)]
    return out + [(dy * xh).double().sum(0).float(), dy.double().sum(0).float()] if s["weight"] is not None else out


def _frequencies(case, dev):
    """(radians a position for each pair in 64 bits, the factor of the rotated values)."""
    R, kw = case["R"], _scaling(case)
    base, factor = 10000.0, kw.get("factor", 1.0)
    if kw["scaling"] == "ntk":
        base = base * factor ** (R / (R - 2)) if R > 2 else base
    i = torch.arange(R // 2, dtype=torch.float64)
    freq = base ** (-2 * i / R)
    if kw["scaling"] == "linear":
        freq = freq / factor
    if kw["scaling"] != "yarn":
        return freq.to(dev), 1.0

    def pair_of(turns):  # the pair that makes so many turns within the original length
        return R * math.log(kw["original_length"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), R - 1)
    stretch = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return (freq * (1 - stretch) + freq / factor * stretch).to(dev), 0.1 * math.log(factor) + 1


def _positions(s):
    if "positions" in s:
        return s["positions"].long()
    cu, pos, seq = _layout(s, s["q"])
    return (pos - cu[seq] + s["offsets"][seq]).reshape(s["q"].shape[:2])


def _plain_rotary(s):
    case = s["case"]
    R = case["R"]
    angle = (_positions(s).double()[..., None] * s["freq"])[..., None, :]
    cos, sin = torch.cos(angle).float() * s["magnitude"], torch.sin(angle).float() * s["magnitude"]
    if case["backward"]:
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y = x.float().clone()
        if case["interleaved"]:
            a, b = x[..., 0:R:2].float(), x[..., 1:R:2].float()
            y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :R // 2].float(), x[..., R // 2:R].float()
            y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
        out.append(y.to(x.dtype))
    return out


# ---- the package's calls -------------------------------------------------------------


def _own(s):
    import linear_attention_prefill_gb300 as lap
    case, op = s["case"], s["case"]["op"]
    if op in ("glr", "glr_bwd", "glr_step"):
        form = dict(gate=case["gate"], input_norm=None if case["norm"] == "none" else case["norm"])
        if op == "glr":
            out = lap.gdn_glr_chunk_fwd(s["x"], s["g"], s["rate"], s["h0"], cu_seqlens=s["cu"],
                                        output_states=case["keep"], **form)
            return list(out if case["keep"] else out[:2])
        if op == "glr_step":
            return lap.gdn_glr_recurrent_step(s["x"], s["g"], s["h0"], s["rate"], **form), s["h0"]
        out = lap.gdn_glr_chunk_bwd(s["dy"], s["x"], s["g"], s["states"], s["rate"], s["h0"], s["dhT"],
                                    cu_seqlens=s["cu"], **form)
        return [t for t in out if t is not None]
    if op == "ln":
        out = lap.gdn_layer_norm_fwd(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS)
        return [t for t in out if t is not None]
    if op == "ln_bwd":
        out = lap.gdn_layer_norm_bwd(s["dy"], s["x"], s["weight"], s["residual"], eps=EPS,
                                     param_grads=case["affine"])
        return [t for t in out if t is not None]
    call = lap.gdn_rotary_bwd if case["backward"] else lap.gdn_rotary_fwd
    out = call(s["q"], s["k"], s["turns"], s.get("positions"), magnitude=s["magnitude"],
               interleaved=case["interleaved"], cu_seqlens=s.get("cu"), offsets=s.get("offsets"))
    return [t for t in out if t is not None]


def run(state):
    if own:
        return _own(state)
    return {"glr": _plain_glr, "glr_step": _plain_step, "glr_bwd": _plain_glr_bwd, "ln": _plain_ln,
            "ln_bwd": _plain_ln_bwd, "rotary": _plain_rotary,
            "rotary_step": _plain_rotary}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    e, op, D = DTYPES[case["dtype"]].itemsize, case["op"], case["D"]
    if op in ("glr", "glr_bwd", "glr_step"):
        t, n = (case["N"], case["N"]) if op == "glr_step" else (case["tokens"], case["seqs"])
        rate = 4 * D * (case["gate"] == "rate")
        # the gate's exponential (three operations, three more of a sigmoid, one of a rate), the weight, the state
        gate = {"log": 2, "sigmoid": 4, "rate": 7}[case["gate"]] + {"none": 0, "linear": 2, "sqrt": 4}[case["norm"]]
        kept = 4 * D * (1 if case.get("packed") else n) * -(-(t if case.get("packed") else t // n) // CHUNK)
        if op == "glr_step":
            return {"bytes": 3 * t * D * e + 8 * n * D + rate, "flops": t * D * (gate + 2)}
        if op == "glr":
            return {"bytes": 3 * t * D * e + 4 * n * D * (1 + case["state"]) + rate + kept * case["keep"],
                    "flops": t * D * (gate + 2)}
        return {"bytes": 5 * t * D * e + 12 * n * D * case["state"] + 2 * rate + kept,
                "flops": t * D * (gate + 10 + 3 * (case["gate"] != "log"))}
    if op in ("ln", "ln_bwd"):
        rows = case["rows"]
        if op == "ln":
            return {"bytes": rows * D * e * (2 + 2 * case["residual"]) + 8 * D * case["affine"],
                    "flops": rows * D * (5 + case["residual"] + 2 * case["affine"])}
        return {"bytes": rows * D * e * (3 + case["residual"]) + 12 * D * case["affine"],
                "flops": rows * D * (11 + case["residual"] + 4 * case["affine"])}
    t = case["tokens"] if op == "rotary" else case["N"]
    heads = case["Hq"] + case["Hk"]
    return {"bytes": 2 * t * heads * D * e + 4 * case["R"] + 4 * (case["N"] if op == "rotary_step" else case["seqs"]),
            "flops": t * heads * case["R"] * 3 + t * case["R"] * 10}


# ---- the definitions in 64 bits ------------------------------------------------------


def _exact_glr(case, seed, s, f):
    op, D = case["op"], case["D"]
    if op == "glr_step":
        spans, lead = None, (1, case["N"])
    elif case["packed"]:
        cuts = _borders(case, seed)
        spans, lead = list(zip(cuts[:-1], cuts[1:])), (case["tokens"], 1)
    else:
        spans, lead = None, (case["tokens"] // case["seqs"], case["seqs"])
    # time first: [T, rows in step, D]
    x, g = (f[k].reshape(lead[1], lead[0], D).transpose(0, 1) for k in ("x", "g"))
    sg = torch.sigmoid(g)
    log = {"log": lambda: g, "sigmoid": lambda: torch.nn.functional.logsigmoid(g),
           "rate": lambda: f["rate"] * sg}[case["gate"]]()
    a = log.exp()
    w = {"none": lambda: torch.ones_like(a), "linear": lambda: -torch.expm1(log),
         "sqrt": lambda: (-torch.expm1(2 * log)).sqrt()}[case["norm"]]()
    h = torch.empty_like(a)
    before = torch.empty_like(a)
    b = w * x
    runs = [(i, lo, hi) for i, (lo, hi) in enumerate(spans)] if spans is not None else [(None, 0, lead[0])]
    pick = lambda t, i: t if i is None else t[i:i + 1]  # noqa: E731
    zero = x.new_zeros(lead[1], D)
    ends = []
    for i, lo, hi in runs:
        now = pick(f["h0"], i) if f["h0"] is not None else zero
        for t in range(lo, hi):
            before[t] = now
            now = torch.addcmul(b[t], a[t], now)
            h[t] = now
        ends.append(now)
    shape = s["x"].shape
    rows = lambda t: t.transpose(0, 1).reshape(shape)  # noqa: E731
    hT = torch.cat(ends)
    if op == "glr_step":
        return rows(h), hT
    if op == "glr":
        out = [rows(h), hT]
        if case["keep"]:
            kept = before[::CHUNK].transpose(0, 1).contiguous()
            if case["packed"]:  # across a border: what the row held before it
                at = torch.arange(0, case["tokens"], CHUNK, device=x.device)
                kept = torch.cat([torch.zeros_like(h[:1, 0]), h[:, 0]])[at][None]
            out.append(kept)
        return out
    dy = f["dy"].reshape(lead[1], lead[0], D).transpose(0, 1)
    lam = torch.empty_like(a)
    starts = []
    for i, lo, hi in runs:
        mu = pick(f["dhT"], i) if f["dhT"] is not None else zero
        for t in range(hi - 1, lo - 1, -1):
            lam[t] = dy[t] + mu
            mu = a[t] * lam[t]
        starts.append(mu)
    slope = a * before
    if case["norm"] == "linear":
        slope = slope - a * x
    elif case["norm"] == "sqrt":
        slope = slope - torch.where(w > 0, a.square() / w, torch.zeros_like(w)) * x
    dlog = lam * slope
    dg = dlog * {"log": 1.0, "sigmoid": torch.sigmoid(-g), "rate": (f["rate"] if f["rate"] is not None else 0.0)
                 * sg * torch.sigmoid(-g)}[case["gate"]]
    out = [rows(w * lam), rows(dg)]
    if case["gate"] == "rate":
        out.append((dlog * sg).sum((0, 1)))
    if case["state"]:
        out.append(torch.cat(starts))
    return out


def _exact_ln(case, f):
    x = f["x"]
    if case["op"] == "ln":
        if case["residual"]:
            x = x + f["residual"]
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) / (var + EPS).sqrt()
        if case["affine"]:
            y = torch.addcmul(f["bias"], y, f["weight"])
        return [y, x] if case["residual"] else [y]
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    sd = (var + EPS).sqrt()
    xh, u = (x - mean) / sd, f["dy"] * (f["weight"] if case["affine"] else 1.0)
    D = case["D"]
    dx = (u - u.sum(-1, keepdim=True) / D - xh * ((u * xh).sum(-1, keepdim=True) / D)) / sd
    if case["residual"]:
        dx = dx + f["residual"]
    return [dx, (f["dy"] * xh).sum(0), f["dy"].sum(0)] if case["affine"] else [dx]


def _exact_rotary(case, seed, s, f):
    R = case["R"]
    freq, magnitude = _frequencies(case, s["q"].device)
    if case["op"] == "rotary":
        cuts = _borders(case, seed)
        at = torch.cat([torch.arange(hi - lo, device=freq.device) + s["offsets"][i]
                        for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:]))])
    else:
        at = s["positions"]
    turn = torch.polar(torch.full_like(freq, magnitude).expand(at.numel(), -1), at.double()[:, None] * freq)
    turn = (turn.conj() if case["backward"] else turn)[:, None]
    out = []
    for x in (f["q"], f["k"]):
        if x is None:
            continue
        rot, rest = x.reshape(-1, *x.shape[-2:]).split([R, case["D"] - R], -1)
        pairs = rot.unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        z = pairs[..., 0] + 1j * pairs[..., 1] if case["interleaved"] else pairs[..., 0, :] + 1j * pairs[..., 1, :]
        z = z * turn
        z = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).flatten(-2)
        out.append(torch.cat([z, rest], -1).reshape(x.shape))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] in ("glr", "glr_bwd", "glr_step"):
        return _exact_glr(case, seed, s, f)
    if case["op"] in ("ln", "ln_bwd"):
        return _exact_ln(case, f)
    return _exact_rotary(case, seed, s, f)
