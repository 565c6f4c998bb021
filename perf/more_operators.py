"""Measured cases of adapters, token log probabilities and block norms.

What a frozen 4-bit model needs beside its products to be tuned and to serve
many tuned versions at once, each operator in a plain form (elementary torch
operations in 32 bits) and as the calls a user makes of
quantized_expert_ffn_warp_gb300.moe:

* adapter:      out[t] = base[t] + scale[a] B[a] (A[a] x[t]),  a = ids[t]
                (low-rank adapters of many requests beside one projection)
* adapter_grad: the gradients of x, A and B
* logprobs:     log probability of given tokens, entropy, the likeliest tokens
* logprobs_grad: the gradient of the first two in the logits
* norm:         out = c resid + gate * gain * y / rms(y),
                xn = next_gain * out / rms(out)
                (the norm behind a block, its gate, the scaled residual, and the
                norm in front of the next block)
* norm_grad:    its gradients in resid, y, the gains and the gate
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
NORM_SCALE = 0.875


def listed():
    return [
        # a decode batch: a token of each request, nearly every one with its own adapter
        dict(name="ad_n13_2048x2048_r16_fp16", op="adapter", n=13, K=2048, rows=2048, r=16, L=64,
             reqs=13, plain=True, base=True, dtype="fp16"),
        # prompts of a few requests through the widest projection
        dict(name="ad_n4001_4096x14336_r64_bf16", op="adapter", n=4001, K=4096, rows=14336, r=64,
             L=16, reqs=9, plain=True, base=True, dtype="bf16"),
        # a short tuning step of a few tenants, small rank
        dict(name="adg_n300_2048x1024_r8_fp16", op="adapter_grad", n=300, K=2048, rows=1024, r=8,
             L=3, reqs=4, plain=False, base=True, dtype="fp16"),
        # a packed tuning batch
        dict(name="adg_n8192_4096x4096_r32_bf16", op="adapter_grad", n=8192, K=4096, rows=4096, r=32,
             L=8, reqs=21, plain=True, base=True, dtype="bf16"),
        # a few requests' answers with their alternatives, a wide vocabulary
        dict(name="lp_n3_v131072_top20_fp32", op="logprobs", n=3, V=131072, top=20, dtype="fp32",
             pad=64, live=1.0),
        # scoring of prompts, an odd vocabulary
        dict(name="lp_n4096_v32003_top5_bf16", op="logprobs", n=4096, V=32003, top=5, dtype="bf16",
             pad=0, live=0.95),
        # the gradient of a handful of tokens
        dict(name="lpg_n16_v32003_bf16", op="logprobs_grad", n=16, V=32003, ent=False,
             dtype="bf16", pad=0, live=1.0),
        # a tuning batch over a wide vocabulary, with an entropy term
        dict(name="lpg_n4096_v131072_bf16", op="logprobs_grad", n=4096, V=131072, ent=True,
             dtype="bf16", pad=64, live=0.9),
        # one token between two blocks
        dict(name="nm_n1_h4096_fp16", op="norm", n=1, H=4096, gate="token", gain=True, dtype="fp16"),
        # a long prompt between two blocks
        dict(name="nm_n16001_h4096_bf16", op="norm", n=16001, H=4096, gate="token", gain=True,
             dtype="bf16"),
        # a short batch's gradients
        dict(name="nmg_n77_h2048_bf16", op="norm_grad", n=77, H=2048, gate="channel", gain=True,
             dtype="bf16"),
        # a packed batch's gradients
        dict(name="nmg_n16384_h4096_bf16", op="norm_grad", n=16384, H=4096, gate="token", gain=True,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adapter", "adapter_grad", "logprobs", "logprobs_grad", "norm", "norm_grad"))
    if op.startswith("adapter"):
        K = 8 * _log_int(rng, 32, 1024)
        rows = _log_int(rng, 256, 14336)
        if op == "adapter_grad" or rng.random() < 0.7:
            rows = (rows + 7) // 8 * 8
        r = 8 * rng.choice((1, 2, 2, 3, 4, 8, 8, 12, 16))
        L = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, 8192)
        # no more traffic than the largest listed case, and a plain form over all adapters
        n = min(n, 8192 * 8192 // (K + rows), int(1e12 / (L * r * (K + rows))))
        n = max(n, 1)
        return dict(op=op, n=n, K=K, rows=rows, r=r, L=L,
                    reqs=min(n, rng.choice((1, n, _log_int(rng, 1, 100)))),
                    plain=rng.random() < 0.5, base=rng.random() < 0.7,
                    dtype=rng.choice(("fp16", "bf16")))
    if op.startswith("logprobs"):
        V = _log_int(rng, 1000, 262144)
        dtype = rng.choice(("fp32", "bf16", "fp16"))
        most = 4096 * 32003 if op == "logprobs" else 4096 * 131072
        n = min(_log_int(rng, 1, 16384), max(1, most // (2 * V if dtype == "fp32" else V)))
        c = dict(op=op, n=n, V=V, dtype=dtype, pad=rng.choice((0, 64)),
                 live=rng.choice((1.0, 0.9, 0.5)))
        if op == "logprobs":
            c["top"] = rng.choice((0, 1, 5, 20, 32))
        else:
            c["ent"] = rng.random() < 0.5
        return c
    H = 8 * _log_int(rng, 32, 2048)
    n = min(_log_int(rng, 1, 16384), 16384 * 4096 // H)
    return dict(op=op, n=n, H=H, gate=rng.choice(("token", "channel", "none")),
                gain=rng.random() < 0.8, dtype=rng.choice(("fp16", "bf16")))


# ---------------------------------------------------------------- inputs

def _request_adapters(case):
    """Adapter of each request, -1 for a request of the plain model."""
    return [-1 if case["plain"] and i % 7 == 3 else i % case["L"] for i in range(case["reqs"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    dt = DTYPES[case["dtype"]]
    n = case["n"]
    st = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    def rand(*shape):
        return torch.rand(shape, device="cuda", generator=g)

    if case["op"].startswith("adapter"):
        K, rows, r, L, reqs = (case[k] for k in ("K", "rows", "r", "L", "reqs"))
        # one token for each request, the others spread unevenly
        share = torch.cumsum(rand(reqs) ** 2 + 1e-3, 0)
        cut = torch.floor(share / share[-1] * (n - reqs) + 0.5).long() + torch.arange(
            1, reqs + 1, device="cuda")
        req = torch.searchsorted(cut, torch.arange(n, device="cuda"), right=True).clamp(max=reqs - 1)
        name = torch.randperm(L, device="cuda", generator=g)
        of_req = torch.tensor(_request_adapters(case), device="cuda")
        of_req = torch.where(of_req < 0, -1, name[of_req.clamp(min=0)])
        st["ids"] = of_req[req].to(torch.int32).contiguous()
        st["A"] = (randn(L, r, K) / math.sqrt(K)).to(dt)
        st["B"] = (randn(L, rows, r) * 0.05).to(dt)
        st["scale"] = rand(L) * 1.5 + 0.5
        st["x"] = randn(n, K).to(dt)
        if case["op"] == "adapter":
            st["base"] = randn(n, rows).to(dt) if case["base"] else None
        else:
            st["dy"] = (randn(n, rows) * 0.02).to(dt)
            st["base"] = (randn(n, K) * 0.02).to(dt) if case["base"] else None
            h = _adapter_h(st["x"].float(), st).view(n, L, r).sum(1)
            st["h"] = h.to(dt)
    elif case["op"].startswith("logprobs"):
        V = case["V"]
        l = 2.5 * randn(n, V)
        # a row's likely tokens, and a padded vocabulary's unused columns
        l.scatter_add_(1, torch.randint(0, V, (n, 8), device="cuda", generator=g),
                       10.0 * rand(n, 8))
        if case["pad"]:
            l[:, V - case["pad"]:] = -math.inf
        st["logits"] = l.to(dt)
        t = torch.randint(0, V - case["pad"], (n,), device="cuda", generator=g)
        likely = l.argmax(1)
        t = torch.where(rand(n) < 0.6, likely, t)
        st["targets"] = torch.where(rand(n) < case["live"], t, -1).to(torch.int32)
        if case["op"] == "logprobs_grad":
            st["fwd"] = _logprobs(st["logits"].float(), st["targets"], 0)
            st["dlogp"] = -(rand(n) + 0.5) / n
            st["dent"] = randn(n) * 0.01 / n if case["ent"] else None
    else:
        H = case["H"]
        outlier = torch.where(rand(H) < 1 / 256, 20.0, 1.0)
        st["resid"] = (randn(n, H) * outlier).to(dt)
        st["y"] = (0.5 * randn(n, H)).to(dt)
        st["gain"] = (rand(H) + 0.5).to(dt) if case["gain"] else None
        st["next_gain"] = (rand(H) + 0.5).to(dt)
        gate = {"token": (n, 1), "channel": (H,), "none": None}[case["gate"]]
        st["gate"] = torch.sigmoid(randn(*gate)).to(dt) if gate else None
        if case["op"] == "norm_grad":
            fwd = _norm(st)
            st["out"], st["stats"] = fwd["out"].to(dt), fwd["stats"]
            st["dout"] = (randn(n, H) * 0.02).to(dt)
            st["dxn"] = (randn(n, H) * 0.02).to(dt)
    return st


# ---------------------------------------------------------------- one pass

def _hot(st):
    """[n, L]: 1 at a token's adapter."""
    L = st["A"].shape[0]
    return (st["ids"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32)).float()


def _adapter_h(x, st):
    """A x of every token in its adapter's columns of [n, L r], 0 in the others."""
    L, r, K = st["A"].shape
    h = (x @ st["A"].float().reshape(L * r, K).t()).view(-1, L, r)
    return (h * _hot(st)[:, :, None]).view(-1, L * r)


def _adapter(st):
    L, r, _ = st["A"].shape
    dt = st["x"].dtype
    h = _adapter_h(st["x"].float(), st)
    wide = st["B"].float().permute(0, 2, 1).reshape(L * r, -1)
    out = (h * st["scale"].repeat_interleave(r)) @ wide
    if st["base"] is not None:
        out = out + st["base"].float()
    return dict(out=out.to(dt), h=h.view(-1, L, r).sum(1).to(dt))


def _adapter_grad(st):
    L, r, K = st["A"].shape
    dt = st["x"].dtype
    hot = _hot(st)
    dy = st["dy"].float()
    wide = st["B"].float().permute(0, 2, 1).reshape(L * r, -1)
    u = ((dy @ wide.t()).view(-1, L, r) * (hot * st["scale"])[:, :, None]).view(-1, L * r)
    dx = u @ st["A"].float().reshape(L * r, K)
    if st["base"] is not None:
        dx = dx + st["base"].float()
    dA = u.t() @ st["x"].float()
    h = (st["h"].float()[:, None, :] * (hot * st["scale"])[:, :, None]).reshape(-1, L * r)
    dB = (h.t() @ dy).view(L, r, -1).permute(0, 2, 1)
    return dict(dx=dx.to(dt), dA=dA.view(L, r, K).to(dt), dB=dB.to(dt).contiguous())


def _order(l):
    """Whole numbers in the order of the fp32 values l (no NaN)."""
    b = (l + 0.0).view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _logprobs(l, targets, top):
    """l fp32 [n, V]."""
    n, V = l.shape
    m = l.amax(1)
    d = l - m[:, None]
    e = torch.exp(d)
    s = e.sum(1)
    logsum = torch.log(s)
    ent = logsum - torch.where(e > 0, e * d, 0.0).sum(1) / s
    ok = targets >= 0
    at = targets.clamp(min=0).long()[:, None]
    logp = torch.where(ok, d.gather(1, at)[:, 0] - logsum, 0.0)
    out = dict(logp=logp, entropy=ent, stats=torch.stack((m, logsum), 1))
    if top:
        # ties go to the lowest index
        key = _order(l) * V + (V - 1 - torch.arange(V, device="cuda"))
        ids = torch.topk(key, top, dim=1).indices
        out.update(top_ids=ids.to(torch.int32), top_logp=d.gather(1, ids) - logsum[:, None])
    return out


def _logprobs_grad(st):
    l, f = st["logits"].float(), st["fwd"]
    logp = l - f["stats"][:, :1] - f["stats"][:, 1:]
    p = torch.exp(logp)
    ok = st["targets"] >= 0
    gl = torch.where(ok, st["dlogp"], 0.0)[:, None]
    d = -gl * p
    if st["dent"] is not None:
        d = d - torch.where(p > 0, st["dent"][:, None] * p * (logp + f["entropy"][:, None]), 0.0)
    d = d.scatter_add(1, st["targets"].clamp(min=0).long()[:, None], gl)
    return d.to(st["logits"].dtype)


def _rms(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _norm(st):
    y = st["y"].float()
    r1 = _rms(y) if st["gain"] is not None else torch.ones_like(y[:, :1])
    v = y * r1
    if st["gain"] is not None:
        v = v * st["gain"].float()
    if st["gate"] is not None:
        v = v * st["gate"].float()
    out = NORM_SCALE * st["resid"].float() + v
    r2 = _rms(out)
    return dict(out=out, xn=out * r2 * st["next_gain"].float(), stats=torch.cat((r1, r2), 1))


def _norm_grad(st):
    dt = st["y"].dtype
    o, y = st["out"].float(), st["y"].float()
    r1, r2 = st["stats"][:, :1], st["stats"][:, 1:]
    hat, dxn = o * r2, st["dxn"].float()
    res = dict(dnext_gain=(dxn * hat).sum(0))
    dn = dxn * st["next_gain"].float()
    do = st["dout"].float() + r2 * (dn - hat * (dn * hat).mean(1, keepdim=True))
    res["dresid"] = (NORM_SCALE * do).to(dt)
    hat = y * r1
    v = hat if st["gain"] is None else hat * st["gain"].float()
    if st["gate"] is not None:
        res["dgate"] = (do * v).sum(0) if st["gate"].dim() == 1 else (do * v).sum(1, keepdim=True)
        do = do * st["gate"].float()
    if st["gain"] is None:
        res["dy"] = do.to(dt)
        return res
    res["dgain"] = (do * hat).sum(0)
    dn = do * st["gain"].float()
    res["dy"] = (r1 * (dn - hat * (dn * hat).mean(1, keepdim=True))).to(dt)
    return res


def run(st):
    op = st["case"]["op"]
    if own:
        from quantized_expert_ffn_warp_gb300 import moe
        if op == "adapter":
            out, h = moe.adapter(st["x"], st["ids"], st["A"], st["B"], st["scale"],
                                 base=st["base"])
            return dict(out=out, h=h)
        if op == "adapter_grad":
            return moe.adapter_grad(st["dy"], st["x"], st["h"], st["ids"], st["A"], st["B"],
                                    st["scale"], base=st["base"])
        if op == "logprobs":
            return moe.token_logprobs(st["logits"], st["targets"], top=st["case"]["top"])
        if op == "logprobs_grad":
            return moe.token_logprobs_grad(st["logits"], st["targets"], st["fwd"], st["dlogp"],
                                           st["dent"])
        if op == "norm":
            return moe.residual_norm(st["resid"], st["y"], gain=st["gain"], gate=st["gate"],
                                     scale=NORM_SCALE, next_gain=st["next_gain"], eps=EPS)
        return moe.residual_norm_grad(st["dout"], st["dxn"], st["out"], st["y"], st["stats"],
                                      gain=st["gain"], gate=st["gate"], scale=NORM_SCALE,
                                      next_gain=st["next_gain"])
    if op == "adapter":
        return _adapter(st)
    if op == "adapter_grad":
        return _adapter_grad(st)
    if op == "logprobs":
        return _logprobs(st["logits"].float(), st["targets"], st["case"]["top"])
    if op == "logprobs_grad":
        return _logprobs_grad(st)
    if op == "norm":
        res = _norm(st)
        dt = st["y"].dtype
        return dict(out=res["out"].to(dt), xn=res["xn"].to(dt), stats=res["stats"])
    return _norm_grad(st)


# ---------------------------------------------------------------- 64 bits

def _exact_adapter(st, grad):
    x, ids = st["x"].to(F64), st["ids"].tolist()
    n, (L, r, K), rows = x.shape[0], st["A"].shape, st["B"].shape[1]
    width = K if grad else rows
    res = torch.zeros((n, width), dtype=F64, device="cuda")
    if st["base"] is not None:
        res += st["base"].to(F64)
    h = torch.zeros((n, r), dtype=F64, device="cuda")
    dA, dB = (torch.zeros(s, dtype=F64, device="cuda") for s in ((L, r, K), (L, rows, r)))
    for a in range(L):
        t = torch.tensor([i for i in range(n) if ids[i] == a], dtype=torch.long, device="cuda")
        if not len(t):
            continue
        A, B, c = st["A"][a].to(F64), st["B"][a].to(F64), float(st["scale"][a])
        if grad:
            dy = st["dy"][t].to(F64)
            u = c * torch.einsum("tj,jr->tr", dy, B)
            res[t] += torch.einsum("tr,rk->tk", u, A)
            dA[a] = torch.einsum("tr,tk->rk", u, x[t])
            dB[a] = c * torch.einsum("tj,tr->jr", dy, st["h"][t].to(F64))
        else:
            h[t] = torch.einsum("tk,rk->tr", x[t], A)
            res[t] += c * torch.einsum("tr,jr->tj", h[t], B)
    return dict(dx=res, dA=dA, dB=dB) if grad else dict(out=res, h=h)


def _exact_logprobs(st, top, grad):
    n = st["logits"].shape[0]
    parts = []
    step = max(1, (1 << 27) // st["logits"].shape[1])
    for a in range(0, n, step):
        rows = slice(a, a + step)
        l = st["logits"][rows].to(F64)
        tgt = st["targets"][rows].long()
        logp = torch.log_softmax(l, 1)
        p = logp.exp()
        ent = -torch.special.xlogy(p, p).sum(1)
        if grad:
            # columns of the softmax Jacobian: d logp_t / d l = onehot - p,
            # d entropy / d l = -p (log p + entropy)
            d = torch.zeros_like(l)
            if st["dent"] is not None:
                w = torch.special.xlogy(p, p) + p * ent[:, None]
                d -= st["dent"][rows].to(F64)[:, None] * w
            on = tgt >= 0
            gl = st["dlogp"][rows].to(F64) * on
            d -= gl[:, None] * p
            i = torch.arange(len(tgt), device="cuda")[on]
            d[i, tgt[on]] += gl[on]
            parts.append((d,))
            continue
        m = l.max(1).values
        got = torch.where(tgt >= 0, logp[torch.arange(len(tgt), device="cuda"), tgt], 0.0)
        stats = torch.stack((m, torch.logsumexp(l - m[:, None], 1)), 1)
        part = (got, ent, stats)
        if top:
            ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top]
            part += (ids.to(torch.int32), torch.take_along_dim(logp, ids, 1))
        parts.append(part)
    cat = [torch.cat(x) for x in zip(*parts)]
    return cat[0] if grad else dict(zip(("logp", "entropy", "stats", "top_ids", "top_logp"), cat))


def _exact_norm(st):
    y = st["y"].to(F64)
    r1 = torch.ones_like(y[:, 0])
    if st["gain"] is not None:
        r1 = ((y * y).sum(1) / y.shape[1] + EPS) ** -0.5
        y = torch.einsum("th,t,h->th", y, r1, st["gain"].to(F64))
    if st["gate"] is not None:
        y = st["gate"].to(F64) * y
    out = st["resid"].to(F64) * NORM_SCALE + y
    r2 = ((out * out).sum(1) / out.shape[1] + EPS) ** -0.5
    return dict(out=out, xn=torch.einsum("th,t,h->th", out, r2, st["next_gain"].to(F64)),
                stats=torch.stack((r1, r2), 1))


def _exact_norm_grad(st):
    """The statistics and the rounded output are inputs here."""
    H = st["y"].shape[1]
    r1, r2 = st["stats"][:, 0].to(F64), st["stats"][:, 1].to(F64)

    def back(dn, v, r):
        # of v r(v): r dn - r^3 / H v (v . dn)
        return r[:, None] * dn - v * (r ** 3 * torch.einsum("th,th->t", v, dn) / H)[:, None]

    o, y, dxn = st["out"].to(F64), st["y"].to(F64), st["dxn"].to(F64)
    do = st["dout"].to(F64) + back(dxn * st["next_gain"].to(F64), o, r2)
    res = dict(dnext_gain=torch.einsum("th,th,t->h", dxn, o, r2), dresid=do * NORM_SCALE)
    gain = torch.ones(H, dtype=F64, device="cuda") if st["gain"] is None else st["gain"].to(F64)
    gate = st["gate"]
    if gate is not None:
        if gate.dim() == 1:
            res["dgate"] = torch.einsum("th,th,t->h", do, y, r1) * gain
        else:
            res["dgate"] = torch.einsum("th,th,t,h->t", do, y, r1, gain)[:, None]
        do = do * gate.to(F64)
    if st["gain"] is None:
        res["dy"] = do
    else:
        res["dgain"] = torch.einsum("th,th,t->h", do, y, r1)
        res["dy"] = back(do * gain, y, r1)
    return res


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("adapter"):
        return _exact_adapter(st, op == "adapter_grad")
    if op.startswith("logprobs"):
        return _exact_logprobs(st, case.get("top", 0), op == "logprobs_grad")
    return _exact_norm(st) if op == "norm" else _exact_norm_grad(st)


# ---------------------------------------------------------------- floors

def work(case):
    n, op = case["n"], case["op"]
    if op.startswith("adapter"):
        K, rows, r, L = case["K"], case["rows"], case["r"], case["L"]
        used = len({a for a in _request_adapters(case) if a >= 0})
        weights = 2 * used * r * (K + rows)
        if op == "adapter":
            b = 2 * n * (K + rows * (1 + case["base"]) + r) + 4 * n + weights
            return {"bytes": b, "flops": 2 * n * r * (K + rows)}
        b = 2 * n * (rows + K * (2 + case["base"]) + r) + 4 * n + weights + 2 * L * r * (K + rows)
        return {"bytes": b, "flops": 4 * n * r * (K + rows)}
    if op.startswith("logprobs"):
        size = 4 if case["dtype"] == "fp32" else 2
        b = n * case["V"] * size
        if op == "logprobs":
            return {"bytes": b + n * (20 + 8 * case["top"]), "flops": 5 * n * case["V"]}
        return {"bytes": 2 * b + n * (20 + 4 * case["ent"]), "flops": 5 * n * case["V"]}
    H = case["H"]
    vectors = {"token": n, "channel": H, "none": 0}[case["gate"]] + H * (1 + case["gain"])
    if op == "norm":
        return {"bytes": 8 * n * H + 2 * vectors + 8 * n, "flops": 8 * n * H}
    return {"bytes": 12 * n * H + 6 * vectors + 8 * n, "flops": 20 * n * H}
