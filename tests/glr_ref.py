"""The gated linear recurrence, layer norm and rotary positions in 64 bits, with error bounds of the
fp32 arithmetic: plain restatements of the definitions, on any device.

Half a unit of rounding is U = 2^-24.  Bounds count the roundings on the magnitudes that they work on;
ex2.approx is off by at most 1.4e-7 (3 U), rcp.approx, sqrt.approx and rsqrt.approx by 2 U each.
"""
import torch

U = 2.0 ** -24


def gates(g, rate, gate, norm):
    """(L, a, error of a, s, error of s, sig, error of sig); the errors are relative."""
    sig = torch.sigmoid(g)
    e_exp = (3 + 2 * g.abs()) * U  # e^-g: two roundings of its argument, 2^x
    e_sig = (1 - sig) * e_exp + 3 * U
    if gate == "log":
        L, eL = g, torch.zeros_like(g)
    elif gate == "sigmoid":
        L, eL = torch.nn.functional.logsigmoid(g), torch.zeros_like(g)
    else:
        L, eL = rate * sig, e_sig + U
    a = torch.exp(L)
    ea = e_sig if gate == "sigmoid" else 3 * U + L.abs() * (eL + 2 * U)
    # 2^x below 2^-126 (1.18e-38) is flushed to zero: an error of all of it
    ea = torch.where(a < 1.2e-38, torch.ones_like(a), ea)
    if norm is None:
        return L, a, ea, torch.ones_like(a), torch.zeros_like(a), sig, e_sig
    left = -torch.expm1(L) if norm == "linear" else -torch.expm1(2 * L)
    if gate == "sigmoid":  # e^-g a, and (1 - a)(1 + a)
        es = a * e_exp + 4 * U + (2 * U if norm == "sqrt" else 0)
    else:
        # the series: 3 U and L's own error (u e^u / (e^u - 1) <= 1); the difference (at least 0.39)
        es = 4 * U + eL + 3 * (2 * a * ea + 2 * U) + (2 * U if norm == "sqrt" else 0)
    return L, a, ea, left if norm == "linear" else left.sqrt(), es, sig, e_sig


def forward(x, g, rate, h0, gate, norm, spans):
    """(y, error, hT, error, states before each token, error, magnitudes) for spans (row, from, to)."""
    x, g = x.double(), g.double()
    rate = rate.double() if rate is not None else None
    _, a, ea, s, es, _, _ = gates(g, rate, gate, norm)
    y, ey, hp, ep, mp = (torch.zeros_like(x) for _ in range(5))
    ends, eends = [], []
    for n, (row, lo, hi) in enumerate(spans):
        h = h0[n].double().clone() if h0 is not None else x.new_zeros(x.shape[-1])
        e, m = torch.zeros_like(h), h.abs()
        for t in range(lo, hi):
            hp[row, t], ep[row, t], mp[row, t] = h, 2 * e, m
            b = s[row, t] * x[row, t]
            e = a[row, t] * (e + m * ea[row, t]) + b.abs() * (es[row, t] + U)
            h = a[row, t] * h + b
            m = a[row, t] * m + b.abs()
            e = e + 2 * U * m
            y[row, t], ey[row, t] = h, 2 * e
        ends.append(h)
        # (twice: stretches of time are composed, a few more roundings for every 8 tokens)
        eends.append(2 * e)
    return y, ey, torch.stack(ends), torch.stack(eends), hp, ep, mp


def backward(dy, x, g, rate, h0, dhT, gate, norm, spans):
    """((dx, error), (dg, error), (drate, error) or None, (dh0, error)) by the formula."""
    _, _, _, _, hp, ep, mp = forward(x, g, rate, h0, gate, norm, spans)
    x, g, dy = x.double(), g.double(), dy.double()
    rate = rate.double() if rate is not None else None
    _, a, ea, s, es, sig, e_sig = gates(g, rate, gate, norm)
    lam, el, ml = (torch.zeros_like(x) for _ in range(3))
    dh0, edh0 = [], []
    for n, (row, lo, hi) in enumerate(spans):
        m = dhT[n].double().clone() if dhT is not None else x.new_zeros(x.shape[-1])
        e, mag = torch.zeros_like(m), m.abs()
        for t in range(hi - 1, lo - 1, -1):
            v = dy[row, t] + m
            mv = dy[row, t].abs() + mag
            e = e + U * mv
            lam[row, t], el[row, t], ml[row, t] = v, 2 * e, mv
            e = a[row, t] * (e + mv * (ea[row, t] + U))
            m, mag = a[row, t] * v, a[row, t] * mv
        dh0.append(m)
        edh0.append(2 * e)
    dx, edx = s * lam, s * el + (s * lam).abs() * (es + U)
    m, em = a * lam, a * el + a * ml * (ea + U)
    if norm is None:
        slope, esl = hp, ep
    elif norm == "linear":
        slope, esl = hp - x, ep + U * (mp + x.abs())
    else:
        r = torch.where(s > 0, a / s, torch.zeros_like(s))
        slope, esl = hp - r * x, ep + (r * x).abs() * (ea + es + 4 * U) + U * (mp + (r * x).abs())
    d = m * slope
    ed = em * slope.abs() + m.abs() * esl + em * esl + U * d.abs()
    drate = None
    if gate == "sigmoid":
        f, ef = torch.sigmoid(-g), (3 + 2 * g.abs()) * U * a + 4 * U + es
    elif gate == "rate":
        w, ew = d * sig, ed * sig + d.abs() * sig * (e_sig + U)
        some = torch.zeros_like(w)
        for row, lo, hi in spans:
            some[row, lo:hi] = 1
        w, ew = w * some, ew * some
        tokens = w.shape[0] * w.shape[1]
        # a thread adds at most every eighth token, then warps, blocks and rows follow
        drate = w.sum((0, 1)), ew.sum((0, 1)) + (tokens / 8 + 32) * U * w.abs().sum((0, 1))
        f, ef = rate * sig * torch.sigmoid(-g), e_sig + (3 + 2 * g.abs()) * U + e_sig + 5 * U
    else:
        f, ef = torch.ones_like(g), torch.zeros_like(g)
    dg, edg = d * f, (ed + d.abs() * ef) * f.abs()
    return (dx, edx), (dg, edg), drate, (torch.stack(dh0), torch.stack(edh0))


def ln_forward(x, w, b, residual, eps):
    """(y, error, r): the mean off by (D/8 / threads + 10) roundings of the sum's magnitude, as the sums are
    taken over 8 columns a thread and then in a tree; the squares' sum by the same relative number."""
    r = x.double() + (residual.double() if residual is not None else 0)
    D = r.shape[-1]
    k = 28  # 16 columns a thread in order, 5 + 4 steps of a tree, 4 blocks
    mean = r.mean(-1, keepdim=True)
    e_mean = k * U * r.abs().mean(-1, keepdim=True) + 2 * U * mean.abs()
    e_r = U * r.abs() if residual is not None else torch.zeros_like(r)
    c = r - mean
    e_c = e_r + e_mean + U * c.abs() + U * mean.abs()
    var = c.square().mean(-1, keepdim=True)
    e_var = (2 * c.abs() * e_c + e_c.square()).mean(-1, keepdim=True) + (k + 3) * U * var
    rstd = (var + eps).rsqrt()
    e_rstd = 0.5 * e_var / (var + eps) + 4 * U  # relative, first order
    e_rstd = e_rstd * (1 + 2 * e_rstd)
    y = c * rstd
    e_y = e_c * rstd + y.abs() * (e_rstd + U)
    if w is not None:
        y, e_y = y * w.double(), e_y * w.double().abs()
        e_y = e_y + U * y.abs()
    if b is not None:
        y = y + b.double()
    return y, e_y + U * y.abs(), r, (c, e_c, rstd, e_rstd, D)


def ln_backward(dy, x, w, dres, eps):
    """((dx, error), (dw, error), (db, error))."""
    _, _, _, (c, e_c, rstd, e_rstd, D) = ln_forward(x, None, None, None, eps)
    dy = dy.double()
    k = 28
    u = dy * w.double() if w is not None else dy
    xh, e_xh = c * rstd, e_c * rstd + (c * rstd).abs() * (e_rstd + U)
    c1 = u.mean(-1, keepdim=True)
    e1 = (k + 2) * U * u.abs().mean(-1, keepdim=True)
    c2 = (u * xh).mean(-1, keepdim=True)
    e2 = ((k + 4) * U * (u * xh).abs() + u.abs() * e_xh).mean(-1, keepdim=True) + 3 * U * c2.abs()
    v = u - c1 - xh * c2
    e_v = 2 * U * (u.abs() + c1.abs() + (xh * c2).abs()) + e1 + xh.abs() * e2 + e_xh * c2.abs() + e_xh * e2
    dx = rstd * v
    e_dx = rstd * e_v + dx.abs() * (e_rstd + U)
    if dres is not None:
        dx = dx + dres.double()
        e_dx = e_dx + U * dx.abs()
    rows = dy.reshape(-1, D).shape[0]
    t = (dy * xh).reshape(-1, D)
    n = rows + 32  # at most every row in order
    dw = t.sum(0), (dy.abs() * e_xh).reshape(-1, D).sum(0) + n * U * t.abs().sum(0)
    flat = dy.reshape(-1, D)
    return (dx, e_dx), dw, (flat.sum(0), n * U * flat.abs().sum(0))


def frequencies(R, base=10000.0, scaling=None, factor=1.0, original_length=0, fast=32.0, slow=1.0):
    """Radians a position of every pair in 64 bits, and the magnitude."""
    import math
    out, mag = [], 1.0
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2))
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            def index(turns):
                return R * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), R - 1)
            keep = 1 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * keep + f / factor * (1 - keep)
            mag = 0.1 * math.log(factor) + 1
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), mag


def rotate(x, position, freq, magnitude, interleaved, backward=False):
    """(y, error): an angle of [-pi, pi] is off by 2^-24 pi at most, cos and sin by 2 U more."""
    x = x.double()
    R = 2 * freq.numel()
    # the angle modulo a turn, without losing it at far positions
    turn = position.double()[..., None] * (freq.to(x.device) / (2 * torch.pi))
    turn = (turn - turn.round())[..., None, :] * 2 * torch.pi
    c, s = magnitude * torch.cos(turn), magnitude * torch.sin(turn) * (-1 if backward else 1)
    y = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    err = torch.zeros_like(y)
    # angle: 2^-25 half turns of rounding, the table's 2^-54 relative in position * freq, then 2 U
    off = magnitude * (a.abs() + b.abs()) * ((3.2 + 2 + 3) * U + 2.0 ** -52 * position.double().abs()[..., None, None])
    err[..., first] = err[..., second] = off
    return y, err
