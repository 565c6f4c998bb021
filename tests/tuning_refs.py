"""64-bit definitions of the adapters, token log probabilities and block norms,
with bounds on what fp32 arithmetic and one rounding may be off by.

H is half an fp32 step.  `half_step(v, dtype)` is half a step of the output's type
at v: at most eps / 2 of |v|, and half the smallest number of fp16 below that.
"""
import torch

H = 2.0 ** -24
INF = float("inf")
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(v, dtype):
    tiny = 2.0 ** -25 if dtype is torch.float16 else 1e-38
    return v.abs() * (torch.finfo(dtype).eps / 2) + tiny


# ---------------------------------------------------------------- log probabilities

def logprobs(logits, targets, top=0):
    """dict as token_logprobs gives it, in 64 bits, with p and the all-masked rows."""
    l = logits.double()
    n, V = l.shape
    m = l.max(1).values
    empty = m == -INF
    d = l - torch.where(empty, 0.0, m)[:, None]
    s = d.exp().sum(1)
    logsum = torch.where(empty, 0.0, torch.log(s))
    lp = torch.where(empty[:, None], -INF, d - logsum[:, None])
    p = torch.where(empty[:, None], 0.0, lp.exp())
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    ent = torch.where(torch.isnan(logsum), logsum, ent)
    res = dict(stats=torch.stack((m, logsum), 1), entropy=ent, lp=lp, p=p, empty=empty, d=d)
    if targets is not None:
        on = (targets >= 0) & (targets < V)
        at = torch.where(on, targets, 0).long()
        res.update(on=on, at=at, logp=torch.where(on, lp.gather(1, at[:, None])[:, 0], 0.0))
    if top:
        rank = torch.where(torch.isnan(l), -INF, l) + 0.0
        ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :top]
        res.update(top_ids=ids.to(torch.int32), top_logp=lp.gather(1, ids))
    return res


def logprob_bounds(ref, V):
    """Bounds of logsum, entropy and of a log probability lp.

    A term e^d: d one rounding, times log2 e (a rounded constant, one rounding), and
    the exponential's 2 units in the last place: (3 |d| + 4) H.  A thread adds V / 256
    of them, then at most 64 more additions; a new maximum scales its sums by such a
    factor, at most once in 4096 values, by no more than the range in all; 16 joins."""
    p, d = ref["p"], ref["d"].clamp(min=-150)
    w = torch.where(p > 0, d.abs(), 0.0)
    span = w.max(1).values
    rel = ((p * (3 * w + 4)).sum(1) + V / 256 + 64 + 8 * (V / 4096 + 16) + 3 * span) * H
    logsum = rel + 2 * H * ref["stats"][:, 1].abs()
    mean = (p * w).sum(1)
    ent = logsum + (p * w * (3 * w + 5)).sum(1) * H + 2 * rel * mean + 4 * H * (mean + 1)

    def lp(v, at):
        return 2 * H * (v.abs() + at.abs()) + logsum
    return logsum, ent, lp


def logprobs_grad(logits, targets, ref, dlogp, dent):
    """Gradient and its bound for fp32 arithmetic from stats rounded to fp32."""
    p, lp = ref["p"], torch.where(ref["p"] > 0, ref["lp"], 0.0)
    n, V = p.shape
    on = torch.zeros(n, dtype=torch.bool, device=p.device) if dlogp is None else ref["on"]
    gl = torch.where(on, dlogp, 0.0).double() if dlogp is not None else torch.zeros_like(p[:, 0])
    ge = torch.zeros_like(gl) if dent is None else dent.double()
    ge = torch.where(ref["empty"], 0.0, ge)
    gl = torch.where(ref["empty"], 0.0, gl)
    e = ref["entropy"]
    g = -p * (gl[:, None] + ge[:, None] * (lp + e[:, None]))
    xm = torch.where(p > 0, ref["d"], 0.0).abs()
    logsum = ref["stats"][:, 1].abs()[:, None]
    # the argument of the exponential, and its factor
    rel = (xm + 3 * lp.abs() + logsum + 4 + 4) * H
    size = p * (gl.abs()[:, None] + ge.abs()[:, None] * (lp.abs() + e.abs()[:, None]))
    err = size * rel + p * ge.abs()[:, None] * (xm + lp.abs() + logsum + 4 * e.abs()[:, None]) * H
    # log p + entropy also holds the rest of (m + logsum) log2 e behind its fp32 value: at
    # most H times it, rounded in four operations, H of it each
    m = torch.where(ref["empty"], 0.0, ref["stats"][:, 0]).abs()[:, None]
    err += p * ge.abs()[:, None] * 4 * 1.45 * (m + logsum) * H * H
    if dlogp is not None:
        row = torch.arange(n, device=p.device)[on]
        g[row, ref["at"][on]] += gl[on]
        err[row, ref["at"][on]] += 2 * H * gl[on].abs()
    return g, err + 1e-36


# ---------------------------------------------------------------- block norms

def residual_norm(resid, y, gain, gate, scale, next_gain, eps):
    """dict(out, xn, stats) in 64 bits, with bounds out_err and xn_err.

    A factor 1 / rms: a sum of squares in chains of 16 and at most 20 more additions,
    halved by the root, and 4 roundings: 24 H."""
    f = torch.float64
    y, r = y.to(f), resid.to(f)
    hid = y.shape[1]
    r1 = torch.ones_like(y[:, :1])
    if gain is not None:
        r1 = (y.square().sum(1, keepdim=True) / hid + eps).rsqrt()
    v = y * r1 * (1.0 if gain is None else gain.to(f)) * (1.0 if gate is None else gate.to(f))
    out = scale * r + v
    err = H * (3 * (scale * r).abs() + 30 * v.abs())
    r2 = torch.ones_like(r1)
    res = dict(out=out, out_err=err)
    if next_gain is not None:
        r2 = (out.square().sum(1, keepdim=True) / hid + eps).rsqrt()
        g = next_gain.to(f)
        shift = (out.abs() * err).sum(1, keepdim=True) / out.square().sum(1, keepdim=True).clamp(
            min=1e-300)
        res.update(xn=out * r2 * g,
                   xn_err=(g * r2).abs() * err + (out * r2 * g).abs() * (28 * H + shift))
        res["r2_err"] = r2 * (24 * H + shift)
    res["stats"] = torch.cat((r1, r2), 1)
    return res


def residual_norm_grad(dout, dxn, out, y, stats, gain, gate, scale, next_gain):
    """(gradients, bounds) from the given statistics and rounded out."""
    f = torch.float64
    y = y.to(f)
    n, hid = y.shape
    r1, r2 = stats[:, :1].to(f), stats[:, 1:].to(f)
    zero = torch.zeros_like(y)
    do = zero.clone() if dout is None else dout.to(f)
    err = 2 * H * do.abs()
    g, b = {}, {}
    sums = (256 + 48) * H       # a chain of 256, the compensated sum, 32 chains joined
    if dxn is not None:
        dx, hat = dxn.to(f), out.to(f) * r2
        dn = dx * next_gain.to(f)
        g["dnext_gain"] = (dx * hat).sum(0)
        b["dnext_gain"] = (sums + 4 * H) * (dx * hat).abs().sum(0) + 1e-38
        mean = (dn * hat).mean(1, keepdim=True)
        size = (dn * hat).abs().mean(1, keepdim=True)
        do = do + r2 * (dn - hat * mean)
        err = err + H * (8 * (r2 * dn).abs() + 48 * r2 * hat.abs() * size)
    g["dresid"], b["dresid"] = scale * do, abs(scale) * (err + 2 * H * do.abs())
    z = y * r1 if gain is not None else y
    gn = torch.ones(hid, dtype=f, device=y.device) if gain is None else gain.to(f)
    ga = torch.ones_like(gn) if gate is None else gate.to(f)
    q = do * ga * gn
    qe = (err + 8 * H * do.abs()) * (ga * gn).abs()
    if gate is not None and gate.dim() == 2:
        g["dgate"] = (do * gn * z).sum(1, keepdim=True)
        b["dgate"] = ((err + 48 * H * do.abs()) * (gn * z).abs()).sum(1, keepdim=True) + 1e-38
    elif gate is not None:
        g["dgate"] = (do * gn * z).sum(0)
        b["dgate"] = ((err + (sums + 6 * H) * do.abs()) * (gn * z).abs()).sum(0) + 1e-38
    if gain is None:
        g["dy"], b["dy"] = q, qe
        return g, b
    g["dgain"] = (do * ga * z).sum(0)
    b["dgain"] = ((err + (sums + 6 * H) * do.abs()) * (ga * z).abs()).sum(0) + 1e-38
    mean = (q * z).mean(1, keepdim=True)
    me = ((qe + 48 * H * q.abs()) * z.abs()).mean(1, keepdim=True)
    g["dy"] = r1 * (q - z * mean)
    b["dy"] = r1 * (qe + z.abs() * me + 8 * H * (q.abs() + (z * mean).abs()))
    return g, b


# ---------------------------------------------------------------- adapters

# A product's sums: fp32 chains in the matrix units and joins, at most a term's worth of
# rounding for each of `terms` terms, and the two-part h or u within 2^-16 (bf16) or
# 2^-22 (fp16) of itself, two roundings each (an absolute 2^-25 where fp16 runs out).
PAIR = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}


def _by_token(ids, count, n):
    on = (ids >= 0) & (ids < count)
    return on, torch.where(on, ids, 0).long()


def adapter(x, ids, A, B, scale, base):
    """(out, bound), (h, bound) in 64 bits; the bounds are those of fp32 sums."""
    f = torch.float64
    n, (count, rank, cols), rows = x.shape[0], A.shape, B.shape[1]
    h = torch.zeros((n, rank), dtype=f, device=x.device)
    he = torch.zeros_like(h)
    out = torch.zeros((n, rows), dtype=f, device=x.device) if base is None else base.to(f, copy=True)
    oe = 2 * H * out.abs()
    for a in range(count):
        t = (ids == a).nonzero()[:, 0]
        if not len(t):
            continue
        s = 1.0 if scale is None else scale[a].to(f)
        xa, Aa, Ba = x[t].to(f), A[a].to(f), B[a].to(f)
        ha = xa @ Aa.t()
        ea = cols * H * (xa.abs() @ Aa.abs().t())
        h[t], he[t] = ha, ea
        ea = ea + PAIR[x.dtype] * ha.abs() + TINY[x.dtype]
        out[t] += s * (ha @ Ba.t())
        oe[t] += abs(s) * (ea @ Ba.abs().t() + (2 * rank + 4) * H * (ha.abs() @ Ba.abs().t()))
    return (out, oe), (h, he)


def adapter_grad(dy, x, h, ids, A, B, scale, base):
    """dict of (gradient, bound)."""
    f = torch.float64
    n, (count, rank, cols), rows = x.shape[0], A.shape, B.shape[1]
    dx = torch.zeros((n, cols), dtype=f, device=x.device) if base is None else base.to(f, copy=True)
    xe = 2 * H * dx.abs()
    dA, dB = torch.zeros(A.shape, dtype=f, device=x.device), torch.zeros(B.shape, dtype=f,
                                                                         device=x.device)
    Ae, Be = torch.zeros_like(dA), torch.zeros_like(dB)
    for a in range(count):
        t = (ids == a).nonzero()[:, 0]
        if not len(t):
            continue
        s = 1.0 if scale is None else scale[a].to(f)
        xa, da, ha = x[t].to(f), dy[t].to(f), h[t].to(f)
        Aa, Ba = A[a].to(f), B[a].to(f)
        u = da @ Ba
        ue = rows * H * (da.abs() @ Ba.abs()) + PAIR[x.dtype] * u.abs() + TINY[x.dtype]
        dx[t] += s * (u @ Aa)
        xe[t] += abs(s) * (ue @ Aa.abs() + (2 * rank + 4) * H * (u.abs() @ Aa.abs()))
        sums = (2 * len(t) + 16) * H
        dA[a] = s * (u.t() @ xa)
        Ae[a] = abs(s) * (ue.t() @ xa.abs() + sums * (u.abs().t() @ xa.abs()))
        dB[a] = s * (da.t() @ ha)
        Be[a] = abs(s) * sums * (da.abs().t() @ ha.abs())
    return dict(dx=(dx, xe), dA=(dA, Ae), dB=(dB, Be))
