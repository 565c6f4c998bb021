"""Measured cases of the 4-bit linear products and the routing losses.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls a user makes of quantized_expert_ffn_warp_gb300.moe:

* linear:       y  = x W^T (+ bias) (+ residual),  W = (q - zero) * scale
* linear_grad:  dx = dy W, the gradient of the frozen 4-bit product's input
* balance:      per-expert counts, mean router probabilities, the load
                balance loss and the z loss of a routed batch
* balance_grad: their gradient in the router logits, with the gradient that
                arrives through the renormalised top-k weights

A weight matrix has the library's canonical layout: codes uint8 [rows, K/2]
(low nibble = even k), scales fp16 and zeros uint8 [rows, K/group].
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token through a square projection: latency
        dict(name="lin_n1_2048x2048_fp16", op="linear", n=1, rows=2048, K=2048, group=128,
             dtype="fp16", bias=False, residual=False, pad=0),
        # a decode batch through the widest projection, with the residual stream added
        dict(name="lin_n8_4096x14336_bf16", op="linear", n=8, rows=4096, K=14336, group=128,
             dtype="bf16", bias=False, residual=True, pad=0),
        # the vocabulary head (an odd row count) for a few sequences, rows of a wider buffer
        dict(name="lin_n3_32003x4096_fp16", op="linear", n=3, rows=32003, K=4096, group=128,
             dtype="fp16", bias=False, residual=False, pad=64),
        # a verified draft or a chunk of a prompt, finer groups, with a bias
        dict(name="lin_n33_6144x4096_bf16", op="linear", n=33, rows=6144, K=4096, group=64,
             dtype="bf16", bias=True, residual=False, pad=0),
        # a long prompt through the widest projection
        dict(name="lin_n4096_14336x4096_fp16", op="linear", n=4096, rows=14336, K=4096, group=128,
             dtype="fp16", bias=False, residual=False, pad=0),
        # the gradient of a handful of rows through an odd projection with fine groups
        dict(name="grad_n2_1027x2048_fp16", op="linear_grad", n=2, rows=1027, K=2048, group=32,
             dtype="fp16", pad=0),
        # the gradient of a decode-sized batch
        dict(name="grad_n8_14336x4096_bf16", op="linear_grad", n=8, rows=14336, K=4096, group=128,
             dtype="bf16", pad=0),
        # a training batch
        dict(name="grad_n2000_4096x4096_bf16", op="linear_grad", n=2000, rows=4096, K=4096,
             group=128, dtype="bf16", pad=0),
        # routing statistics of one decode batch
        dict(name="bal_n64_e64_k2_fp32", op="balance", n=64, E=64, k=2, segs=1, mask=False,
             dtype="fp32", dw=False),
        # a packed training batch of ragged sequences with padding tokens
        dict(name="bal_n32768_e256_k8_fp32", op="balance", n=32768, E=256, k=8, segs=37, mask=True,
             dtype="fp32", dw=False),
        # the gradient of one small batch, through the losses and the top-k weights
        dict(name="bgrad_n1000_e512_k4_fp32", op="balance_grad", n=1000, E=512, k=4, segs=1,
             mask=False, dtype="fp32", dw=True),
        # the gradient of a packed batch, logits in 16 bits
        dict(name="bgrad_n65521_e256_k8_bf16", op="balance_grad", n=65521, E=256, k=8, segs=61,
             mask=True, dtype="bf16", dw=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "linear_grad", "balance", "balance_grad"))
    if op in ("linear", "linear_grad"):
        group = rng.choice((32, 64, 128))
        rows = _log_int(rng, 128, 32768)
        K = max(1, _log_int(rng, 256, 14336) // group) * group
        # no more operations than the largest listed case, of plain arithmetic
        n = min(_log_int(rng, 1, 4096), max(1, int(4096 * 14336 * 4096 / (rows * K))))
        c = dict(op=op, n=n, rows=rows, K=K, group=group, dtype=rng.choice(("fp16", "bf16")),
                 pad=rng.choice((0, 0, 8, 200)))
        if op == "linear":
            c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        return c
    E = _log_int(rng, 8, 512)
    n = min(_log_int(rng, 1, 65536), 65536 * 256 // E)
    return dict(op=op, n=n, E=E, k=min(E, rng.choice((1, 2, 4, 6, 8))),
                segs=rng.choice((1, _log_int(rng, 1, 300))), mask=rng.random() < 0.5,
                dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), dw=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

def _rows_of(t, pad):
    """t as the leading columns of a buffer whose rows are `pad` elements longer."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    dt = DTYPES[case["dtype"]]
    n = case["n"]
    st = dict(case=case)
    if case["op"] in ("linear", "linear_grad"):
        rows, K, group = case["rows"], case["K"], case["group"]
        st["codes"] = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda",
                                    generator=g)
        st["scales"] = (torch.rand((rows, K // group), device="cuda", generator=g) * 0.015
                        + 0.005).half()
        st["zeros"] = torch.randint(6, 10, (rows, K // group), dtype=torch.uint8, device="cuda",
                                    generator=g)
        if case["op"] == "linear":
            st["x"] = _rows_of(torch.randn((n, K), device="cuda", generator=g).to(dt), case["pad"])
            st["bias"] = (torch.randn(rows, device="cuda", generator=g).to(dt)
                          if case["bias"] else None)
            st["residual"] = (torch.randn((n, rows), device="cuda", generator=g).to(dt)
                              if case["residual"] else None)
        else:
            st["dy"] = _rows_of((torch.randn((n, rows), device="cuda", generator=g) * 0.02).to(dt),
                                case["pad"])
        return st
    E, k, S = case["E"], case["k"], case["segs"]
    skew = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=F32))
    st["logits"] = (2.0 * torch.randn((n, E), device="cuda", generator=g) + skew).to(dt)
    top = torch.topk(st["logits"].float(), k, dim=1)
    st["idx"] = top.indices.to(torch.int32).contiguous()
    e = torch.exp(top.values - top.values[:, :1])
    st["w"] = (e / e.sum(1, keepdim=True)).contiguous()
    cuts = torch.sort(torch.randint(0, n + 1, (S - 1,), device="cuda", generator=g)).values
    ends = torch.tensor([0, n], device="cuda")
    st["seq"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32) if S > 1 else None
    st["mask"] = ((torch.rand(n, device="cuda", generator=g) < 0.94).to(torch.uint8)
                  if case["mask"] else None)
    if case["op"] == "balance_grad":
        st["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
        st["dw"] = (torch.randn((n, k), device="cuda", generator=g) * 1e-4 if case["dw"] else None)
        # what the forward pass left: counts and log-sum-exps of the batch
        seg = _segments(st["seq"], n)
        valid = _valid(st["mask"], n)
        st["lse"] = _lse(st["logits"].float(), valid)
        st["counts"], st["tokens"] = _counts(st["idx"], seg, valid, S, E)
    return st


def _segments(seq, n):
    """Segment of every token."""
    if seq is None:
        return torch.zeros(n, dtype=torch.int64, device="cuda")
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    return torch.searchsorted(seq[1:].contiguous(), t, right=True)


def _valid(mask, n):
    return torch.ones(n, dtype=torch.bool, device="cuda") if mask is None else mask != 0


def _lse(l, valid):
    m = l.max(1, keepdim=True).values
    return torch.where(valid, m[:, 0] + torch.log(torch.exp(l - m).sum(1)), 0.0)


def _counts(idx, seg, valid, S, E):
    flat = (seg[:, None] * E + idx.long())[valid].reshape(-1)
    counts = torch.zeros(S * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    tokens = torch.zeros(S, dtype=torch.int32, device="cuda")
    tokens.index_add_(0, seg, valid.to(torch.int32))
    return counts.view(S, E), tokens


# ---------------------------------------------------------------- one pass

def _dequant(st, group):
    """W fp32 [rows, K]."""
    q = st["codes"]
    q = torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1, group).float()
    return ((q - st["zeros"].float()[:, :, None]) * st["scales"].float()[:, :, None]).flatten(1)


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from quantized_expert_ffn_warp_gb300 import moe
        if op == "linear":
            return moe.linear(st["x"], st["codes"], st["scales"], st["zeros"], c["group"],
                              bias=st["bias"], residual=st["residual"])
        if op == "linear_grad":
            return moe.linear_input_grad(st["dy"], st["codes"], st["scales"], st["zeros"],
                                         c["group"])
        if op == "balance":
            return moe.balance_loss(st["logits"], st["idx"], seq_offsets=st["seq"],
                                    mask=st["mask"])
        fwd = dict(counts=st["counts"], tokens=st["tokens"], lse=st["lse"])
        return moe.balance_loss_grad(st["logits"], st["idx"], fwd, st["dloss"],
                                     topk_w=st["w"], dtopk_w=st["dw"], seq_offsets=st["seq"],
                                     mask=st["mask"])
    if op == "linear":
        y = st["x"].float() @ _dequant(st, c["group"]).t()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(st["x"].dtype)
    if op == "linear_grad":
        return (st["dy"].float() @ _dequant(st, c["group"])).to(st["dy"].dtype)

    n, E, k, S = c["n"], c["E"], c["k"], c["segs"]
    seg, valid = _segments(st["seq"], n), _valid(st["mask"], n)
    logits = st["logits"].float()
    if op == "balance":
        counts, tokens = _counts(st["idx"], seg, valid, S, E)
        lse = _lse(logits, valid)
        p = torch.where(valid[:, None], torch.exp(logits - lse[:, None]), 0.0)
        T = tokens.clamp(min=1).to(F64)
        # sums over long batches in 64 bits: the plain form adds in any order
        prob = torch.zeros((S, E), dtype=F64, device="cuda").index_add_(0, seg, p.to(F64))
        prob = prob / T[:, None]
        f = counts.to(F64) * E / (k * T[:, None])
        bal = (f * prob).sum() / (tokens > 0).sum().clamp(min=1)
        z = lse.to(F64).square().sum() / tokens.sum().clamp(min=1)
        return dict(loss=torch.stack((bal, z)).float(), counts=counts, tokens=tokens,
                    prob=prob.float(), lse=lse)
    p = torch.where(valid[:, None], torch.exp(logits - st["lse"][:, None]), 0.0)
    counts, tokens = st["counts"], st["tokens"]
    live = (tokens > 0).sum().clamp(min=1).float()
    T = tokens.clamp(min=1).float()
    f = (counts.float() * (E / (k * T[:, None])))[seg]
    d = p * (f - (f * p).sum(1, keepdim=True)) * (st["dloss"][0] / (live * T[seg]))[:, None]
    d = d + p * (2.0 * st["lse"] * st["dloss"][1] / tokens.sum().clamp(min=1))[:, None]
    if st["dw"] is not None:
        w, dw = st["w"], st["dw"]
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        dl = torch.where(valid[:, None], dl, 0.0)
        d = d.scatter_add(1, st["idx"].long(), dl)
    return d.to(st["logits"].dtype)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_grad"):
        rows, K, group = case["rows"], case["K"], case["group"]
        q = torch.empty((rows, K), dtype=F64, device="cuda")
        q[:, 0::2] = torch.remainder(st["codes"], 16).to(F64)
        q[:, 1::2] = torch.div(st["codes"], 16, rounding_mode="floor").to(F64)
        W = q.sub_(st["zeros"].to(F64).repeat_interleave(group, 1))
        W = W.mul_(st["scales"].to(F64).repeat_interleave(group, 1))
        if op == "linear_grad":
            return torch.einsum("tr,rk->tk", st["dy"].to(F64), W)
        y = torch.einsum("tk,rk->tr", st["x"].to(F64), W)
        for add in (st["bias"], st["residual"]):
            if add is not None:
                y += add.to(F64)
        return y
    n, E, k, S = case["n"], case["E"], case["k"], case["segs"]
    seq = [0, n] if st["seq"] is None else st["seq"].tolist()
    l = st["logits"].to(F64).requires_grad_(op == "balance_grad")
    live = torch.ones(n, dtype=F64, device="cuda") if st["mask"] is None else st["mask"].to(F64)
    logp = torch.log_softmax(l, 1)
    lse = (l - logp).mean(1) * live
    bal, parts, probs, T = 0.0, 0, [], []
    for s in range(S):
        a, b = seq[s], seq[s + 1]
        p = (logp[a:b].exp() * live[a:b, None]).sum(0)
        ids = st["idx"][a:b][live[a:b] > 0]
        cnt = torch.bincount(ids.reshape(-1).long(), minlength=E)
        t = float(live[a:b].sum())
        if t > 0:
            parts += 1
            bal = bal + E / (k * t * t) * (cnt.to(F64) * p).sum()
            p = p / t
        probs.append(p)
        T.append(t)
    bal = bal / max(parts, 1)
    z = (lse ** 2).sum() / max(sum(T), 1.0)
    if op == "balance":
        counts = torch.stack([torch.bincount(
            st["idx"][seq[s]:seq[s + 1]][live[seq[s]:seq[s + 1]] > 0].reshape(-1).long(),
            minlength=E) for s in range(S)]).to(torch.int32)
        return dict(loss=torch.stack((torch.as_tensor(bal, device="cuda", dtype=F64), z)),
                    counts=counts, tokens=torch.tensor(T, device="cuda").to(torch.int32),
                    prob=torch.stack(probs), lse=lse)
    total = st["dloss"][0].to(F64) * bal + st["dloss"][1].to(F64) * z
    if sum(T) == 0:
        return torch.zeros_like(l)
    grad = torch.autograd.grad(total, l)[0]
    if st["dw"] is not None:
        w, dw = st["w"].to(F64), st["dw"].to(F64)
        for j in range(k):    # column j of the softmax Jacobian diag(w) - w w^T, times dw
            jac = -w * w[:, j:j + 1]
            jac[:, j] += w[:, j]
            add = (jac * dw).sum(1) * live
            grad[torch.arange(n, device="cuda"), st["idx"][:, j].long()] += add
    return grad


# ---------------------------------------------------------------- floors

def work(case):
    n = case["n"]
    if case["op"] in ("linear", "linear_grad"):
        rows, K = case["rows"], case["K"]
        b = rows * K / 2 + 3 * rows * (K // case["group"]) + 2 * n * (rows + K)
        if case["op"] == "linear":
            b += 2 * rows * case["bias"] + 2 * n * rows * case["residual"]
        return {"bytes": b, "flops": 2 * n * rows * K}
    E, k, S = case["E"], case["k"], case["segs"]
    size = 4 if case["dtype"] == "fp32" else 2
    common = n * E * size + 4 * n + n * case["mask"] + 4 * (S + 1) + 4 * S * (E + 1)
    if case["op"] == "balance":
        return {"bytes": common + 4 * n * k + 4 * S * E + 8, "flops": 5 * n * E}
    return {"bytes": common + n * E * size + 12 * n * k * case["dw"] + 8, "flops": 8 * n * E}
