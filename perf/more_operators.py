"""What is measured of a layer of experts beside its 16- and 8-bit products: the router, the way
of the tokens' rows to the experts and back, and 4-bit blocks with a scale each.

Five operators:

* ``route``    scores of the experts, the best of them with their weights, each slot's row in the
               experts' order and where each expert's rows begin; with ``train`` also the logits'
               gradient
* ``rows``     the experts' outputs summed for each token by weight; with ``train`` the tokens'
               rows spread before that, and all gradients
* ``quantize`` rows to 4-bit floating point (1 sign, 2 exponent, 1 mantissa bit) in blocks of 32
               with a power of two each, and the values that they stand for
* ``gemm``     product of two such matrices
* ``grouped``  the same with the rows grouped by expert

`run` computes them in elementary torch operations (`own` false) or through this package's
entry points (`own` true); `exact` computes the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decoding step of 8 sequences: latency
        dict(name="route_decode", op="route", tokens=8, pad=0, experts=64, k=8, scoring="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, dtype="f32", train=False),
        # a prompt batch with padded tokens at its end: experts in groups on nodes of their own, a
        # bias that balances them
        dict(name="route_prompt", op="route", tokens=16384, pad=500, experts=256, k=8, scoring="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5, dtype="bf16", train=False),
        # a training batch of odd sizes, forward and backward
        dict(name="route_train", op="route", tokens=4001, pad=0, experts=60, k=6, scoring="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0, dtype="f32", train=True),
        # the experts' outputs of one decoding step
        dict(name="rows_decode", op="rows", tokens=8, pad=0, k=8, width=4096, dtype="bf16", train=False),
        # a training batch to the experts and back, with padded tokens, forward and backward
        dict(name="rows_train", op="rows", tokens=8192, pad=77, k=4, width=4096, dtype="bf16", train=True),
        # the activations of one decoding step before a 4-bit layer
        dict(name="quantize_decode", op="quantize", rows=8, cols=4096, dtype="bf16"),
        # the activations of a prompt batch, the widest layer input
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=14336, dtype="bf16"),
        # one token through the up projection of a 4-bit model: reads the weights once
        dict(name="gemm_token", op="gemm", m=1, n=14336, k=4096, out="bf16"),
        # a ragged batch and layer; scales in rows of 65 bytes
        dict(name="gemm_ragged", op="gemm", m=1000, n=1531, k=2080, out="f32"),
        # a prompt batch through the up projection
        dict(name="gemm_prompt", op="gemm", m=8192, n=14336, k=4096, out="bf16"),
        # decoding with 4-bit experts: one token's 8 experts of 64
        dict(name="grouped_decode", op="grouped", groups=64, active=8, rows=8, pad=0, n=4096, k=2048, out="bf16"),
        # a prompt batch through 4-bit experts, ragged groups, one of them empty
        dict(name="grouped_prompt", op="grouped", groups=16, active=15, rows=8192, pad=0, n=8192, k=4096, out="bf16"),
    ]


def draw(rng):
    """A case of the same ranges, no more work than the operator's largest listed one."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def size(lo, hi):
        v = spread(lo, hi)
        return v if rng.random() < 0.35 else min(hi, max(lo, (v + 8) // 16 * 16))

    op = rng.choice(["route", "rows", "quantize", "gemm", "gemm", "grouped", "grouped"])
    all_work = [work(c) for c in listed() if c["op"] == op]
    most = {x: max(w[x] for w in all_work) for x in ("bytes", "flops")}
    while True:
        if op == "route":
            tokens = spread(1, 16384)
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * spread(4, 256 // groups)
            top_groups = rng.randint(1, groups)
            group_top = rng.choice([1, 2])
            bias = rng.random() < 0.5
            c = dict(op=op, tokens=tokens, pad=rng.choice([0, 0, rng.randint(0, tokens - 1)]), experts=experts,
                     k=rng.randint(1, min(8, experts // groups * top_groups)),
                     scoring=rng.choice(["softmax", "sigmoid"]), bias=bias, groups=groups, top_groups=top_groups,
                     group_top=group_top, renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                     dtype=rng.choice(["bf16", "f16", "f32"]), train=rng.random() < 0.4)
        elif op == "rows":
            tokens = spread(1, 16384)
            c = dict(op=op, tokens=tokens, pad=rng.choice([0, 0, rng.randint(0, tokens - 1)]), k=rng.randint(1, 8),
                     width=size(16, 8192), dtype=rng.choice(["bf16", "f16", "f32"]), train=rng.random() < 0.5)
        elif op == "quantize":
            c = dict(op=op, rows=spread(1, 16384), cols=size(1, 16384), dtype=rng.choice(["bf16", "f16", "f32"]))
        elif op == "gemm":
            c = dict(op=op, m=spread(1, 8192), n=size(16, 16384), k=32 * spread(8, 512),
                     out=rng.choice(["bf16", "f16", "f32"]))
        else:
            groups = spread(1, 64)
            rows = spread(1, 16384)
            c = dict(op=op, groups=groups, active=rng.randint(1, min(groups, rows)), rows=rows,
                     pad=rng.choice([0, 0, rng.randint(1, 100)]), n=size(16, 14336), k=32 * spread(8, 256),
                     out=rng.choice(["bf16", "f16", "f32"]))
            if c["groups"] * c["n"] * c["k"] > 16 * 8192 * 4096:
                continue
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]:
            return c


def _normal(shape, gen, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def group_rows(case, seed):
    """Rows of each group: `active` of the groups at random, at least one row each, the rest
    shared out unevenly, as a router does."""
    rng = random.Random(seed * 1000003 + 17)
    rows = [0] * case["groups"]
    chosen = rng.sample(range(case["groups"]), case["active"])
    weight = [rng.expovariate(1.0) + 0.3 for _ in chosen]
    left = case["rows"] - len(chosen)
    share = [int(left * w / sum(weight)) for w in weight]
    share[0] += left - sum(share)
    for g, s in zip(chosen, share):
        rows[g] = 1 + s
    return rows


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx4(x):
    """Codes (two to a byte, the even element low) and scales of a matrix' rows in blocks of 32; a
    last block is filled up with zeros."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    y = torch.zeros((rows, blocks, 32), dtype=torch.float64, device=x.device)
    y.view(rows, blocks * 32)[:, :cols] = x
    a = y.abs()
    top = a.amax(dim=2, keepdim=True)
    _, e = torch.frexp(top)                       # top = m 2^e, 1/2 <= m < 1
    e = torch.where(top > 0, e - 3, torch.full_like(e, -127)).clamp(-127, 127)
    a = a * _power(-e)
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    # borders between neighbours; the even code takes the border itself
    for i, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= border) if i % 2 else (a > border)
    code += torch.signbit(y).to(torch.uint8) * 8
    packed = code[:, :, 0::2] + code[:, :, 1::2] * 16
    return packed.view(rows, blocks * 16).contiguous(), (e[:, :, 0] + 127).to(torch.uint8)


VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx4_values(q, scale, dtype):
    """rows x 32 blocks of the values that the codes stand for."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=dtype, device=q.device)
    codes = torch.stack((q & 15, q >> 4), dim=2).view(q.shape[0], scale.shape[1], 32)
    power = _power(scale.int() - 127).to(dtype)
    return (table[codes.int()] * power[:, :, None]).view(q.shape[0], -1)


def _random_mx4(rows, k, gen, scale):
    q = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, k // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 24) // k)
    for lo in range(0, rows, step):
        n = min(step, rows - lo)
        q[lo:lo + n], s[lo:lo + n] = _mx4(_normal((n, k), gen, scale))
    return q, s


def _slots(tokens, pad, k, seed):
    """A router's plan: the row of each token's slots, with no row for the padded tokens, and the
    number of rows."""
    rng = torch.Generator().manual_seed(seed + 5)
    live = (tokens - pad) * k
    rows = torch.full((tokens, k), -1, dtype=torch.int32)
    rows.view(-1)[:live] = torch.randperm(live, generator=rng).to(torch.int32)
    return rows.cuda(), live


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        # some experts are liked better than others
        logits = _normal((t, e), gen, 1.5) + _normal((1, e), gen, 0.5)
        if case["pad"]:
            logits[t - case["pad"]:] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["bias"] = _normal((e,), gen, 0.05) if case["bias"] else None
        s["dweights"] = _normal((t, k), gen, 0.1) if case["train"] else None
        return s
    if op == "rows":
        t, k, d = case["tokens"], case["k"], case["width"]
        dtype = DTYPES[case["dtype"]]
        s["rows"], _ = _slots(t, case["pad"], k, seed)
        s["y"] = _normal((t * k, d), gen, 1.0, dtype)
        s["weights"] = torch.softmax(_normal((t, k), gen), dim=1)
        if case["train"]:
            s["x"] = _normal((t, d), gen, 1.0, dtype)
            s["dout"] = _normal((t, d), gen, 0.1, dtype)
            s["dxs"] = _normal((t * k, d), gen, 0.1, dtype)
            # rows behind the last one keep what the user's buffers hold
            s["xs"] = torch.zeros((t * k, d), dtype=dtype, device="cuda")
            s["dy"] = torch.zeros((t * k, d), dtype=dtype, device="cuda")
        return s
    if op == "quantize":
        x = _normal((case["rows"], case["cols"]), gen, 1.0, DTYPES[case["dtype"]])
        x[:, ::97] *= 8  # a few channels much larger than the others, as activations have them
        s["x"] = x
        return s
    s["out"] = DTYPES[case["out"]]
    n, k = case["n"], case["k"]
    if op == "gemm":
        s["a"], s["sa"] = _random_mx4(case["m"], k, gen, 1.0)
        s["b"], s["sb"] = _random_mx4(n, k, gen, 1.0 / math.sqrt(k))
        return s
    offsets = [0]
    for r in group_rows(case, seed):
        offsets.append(offsets[-1] + r)
    total = case["rows"] + case["pad"]
    s["ranges"] = offsets
    s["offsets"] = torch.tensor(offsets, device="cuda")
    # with rows behind the last group the user hands in the buffer those rows keep their values in
    s["y"] = torch.zeros((total, n), dtype=s["out"], device="cuda") if case["pad"] else None
    s["a"], s["sa"] = _random_mx4(total, k, gen, 1.0)
    b, sb = _random_mx4(case["groups"] * n, k, gen, 1.0 / math.sqrt(k))
    s["b"], s["sb"] = b.view(case["groups"], n, k // 2), sb.view(case["groups"], n, k // 32)
    return s


# ------------------------------------------------------------------------ plain forms

def _plain_scores(logits, scoring, dtype):
    x = logits.to(dtype)
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(dim=1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _plain_route(s):
    c, logits = s["case"], s["logits"]
    t, n, k = c["tokens"], c["experts"], c["k"]
    # the choice in 64 bits: values next to the border have to fall on their side
    wide = _plain_scores(logits, c["scoring"], torch.float64)
    masked = logits == -math.inf
    choice = logits.double() if s["bias"] is None else wide + s["bias"].double()
    choice = choice.masked_fill(masked, -math.inf)
    if c["groups"] > 1:
        by_sum = choice if c["group_top"] == 1 or s["bias"] is not None else wide.masked_fill(masked, -math.inf)
        best = by_sum.view(t, c["groups"], -1).sort(dim=2, descending=True)[0][:, :, :c["group_top"]].sum(dim=2)
        kept = best.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros((t, c["groups"]), dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        choice = choice.masked_fill(~keep.repeat_interleave(n // c["groups"], dim=1), -math.inf)
    value, index = choice.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    none = value == -math.inf
    scores = _plain_scores(logits, c["scoring"], torch.float32)
    w = scores.gather(1, index).masked_fill(none, 0.0)
    total = w.sum(dim=1, keepdim=True) if c["renormalize"] else torch.ones_like(w[:, :1])
    weights = torch.where(total > 0, c["scale"] * w / total, torch.zeros_like(w))
    experts = index.masked_fill(none, n).view(-1)
    # slots in the order of the experts, each expert's by token; slots without an expert last
    order = experts.sort(stable=True)[1]
    rows = torch.empty_like(order)
    rows[order] = torch.arange(t * k, device=order.device)
    rows = rows.masked_fill(none.view(-1), -1).view(t, k)
    counts = (experts[:, None] == torch.arange(n, device=order.device)[None, :]).sum(dim=0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(dim=0)))
    out = [weights, index.masked_fill(none, -1).int(), rows.int(), offsets]
    if c["train"]:
        g = s["dweights"].masked_fill(none, 0.0) * c["scale"]
        if c["renormalize"]:
            share = torch.where(total > 0, w / total, torch.zeros_like(w))
            g = torch.where(total > 0, (g - (g * share).sum(dim=1, keepdim=True)) / total, torch.zeros_like(g))
        ds = torch.zeros_like(scores).scatter_add_(1, index, g.masked_fill(none, 0.0))
        if c["scoring"] == "sigmoid":
            d = scores * (1.0 - scores) * ds
        else:
            d = scores * (ds - (scores * ds).sum(dim=1, keepdim=True))
        out.append(d.to(logits.dtype))
    return tuple(out)


def _plain_combine(y, rows, weights, dtype):
    out = torch.zeros((rows.shape[0], y.shape[1]), dtype=torch.float32, device=y.device)
    for j in range(rows.shape[1]):
        at = rows[:, j].long()
        part = y[at.clamp(min=0)].float()
        w = (at >= 0).float() if weights is None else weights[:, j].masked_fill(at < 0, 0.0)
        out += part * w[:, None]
    return out.to(dtype)


def _plain_spread(x, rows, weights, total):
    out = torch.zeros((total + 1, x.shape[1]), dtype=x.dtype, device=x.device)  # the last: no row
    for j in range(rows.shape[1]):
        at = rows[:, j].long()
        out[torch.where(at < 0, total, at)] = x if weights is None else (x.float() * weights[:, j:j + 1]).to(x.dtype)
    return out[:total]


def _plain_rows(s):
    rows, y = s["rows"], s["y"]
    out = _plain_combine(y, rows, s["weights"], y.dtype)
    if not s["case"]["train"]:
        return out
    xs = _plain_spread(s["x"], rows, None, y.shape[0])
    dy = _plain_spread(s["dout"], rows, s["weights"], y.shape[0])
    dw = torch.zeros(rows.shape, dtype=torch.float32, device=y.device)
    for j in range(rows.shape[1]):
        at = rows[:, j].long()
        dw[:, j] = (y[at.clamp(min=0)].float() * s["dout"].float()).sum(dim=1).masked_fill(at < 0, 0.0)
    return xs, out, dy, dw, _plain_combine(s["dxs"], rows, None, y.dtype)


def _plain_quantize(s):
    q, scale = _mx4(s["x"])
    return _mx4_values(q, scale, torch.float32)[:, :s["x"].shape[1]].to(s["x"].dtype)


def _plain_gemm(a, sa, b, sb, out):
    return (_mx4_values(a, sa, torch.float32) @ _mx4_values(b, sb, torch.float32).t()).to(out)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "rows":
        return _plain_rows(s)
    if op == "quantize":
        return _plain_quantize(s)
    if op == "gemm":
        return _plain_gemm(s["a"], s["sa"], s["b"], s["sb"], s["out"])
    y = torch.zeros((s["a"].shape[0], s["b"].shape[1]), dtype=s["out"], device="cuda")
    for g in range(s["b"].shape[0]):
        lo, hi = s["ranges"][g], s["ranges"][g + 1]
        if hi > lo:
            y[lo:hi] = _plain_gemm(s["a"][lo:hi], s["sa"][lo:hi], s["b"][g], s["sb"][g], s["out"])
    return y


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import tiled_gemm_gemv_amd as mm
    c = s["case"]
    op = c["op"]
    if op == "route":
        weights, experts, rows, offsets = mm.route_topk(
            s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
            group_top=c["group_top"], renormalize=c["renormalize"], scale=c["scale"])
        if not c["train"]:
            return weights, experts, rows, offsets
        return weights, experts, rows, offsets, mm.route_topk_grad(
            s["logits"], experts, s["dweights"], scoring=c["scoring"], renormalize=c["renormalize"], scale=c["scale"])
    if op == "rows":
        if not c["train"]:
            return mm.combine_rows(s["y"], s["rows"], s["weights"], out_dtype=s["y"].dtype)
        xs = mm.spread_rows(s["x"], s["rows"], out=s["xs"])
        out = mm.combine_rows(s["y"], s["rows"], s["weights"], out_dtype=s["y"].dtype)
        dy, dw = mm.combine_rows_grad(s["dout"], s["y"], s["rows"], s["weights"], out=s["dy"])
        return xs, out, dy, dw, mm.combine_rows(s["dxs"], s["rows"], out_dtype=s["y"].dtype)
    if op == "quantize":
        q, scale = mm.quantize_mx4(s["x"])
        return mm.dequantize_mx4(q, scale, cols=c["cols"], out_dtype=s["x"].dtype)
    if op == "gemm":
        return mm.gemm_mx4(s["a"], s["b"], s["sa"], s["sb"], out_dtype=s["out"])
    return mm.gemm_mx4_grouped(s["a"], s["b"], s["offsets"], s["sa"], s["sb"], out=s["y"], out_dtype=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k, es = case["tokens"], case["experts"], case["k"], BYTES[case["dtype"]]
        moved = t * e * es + 12 * t * k + 8 * (e + 1) + (4 * e if case["bias"] else 0)
        flops = t * (5 * e + 2 * k)
        if case["train"]:
            moved += 4 * t * k + t * e * es
            flops += t * (5 * e + 4 * k)
        return {"bytes": moved, "flops": flops}
    if op == "rows":
        t, k, d, es = case["tokens"], case["k"], case["width"], BYTES[case["dtype"]]
        live = (t - case["pad"]) * k
        moved, flops = (live + t) * d * es + 8 * t * k, 2 * live * d
        if case["train"]:  # x and dout read, xs, dy written, dxs read, dx written, dw written
            moved += (2 * (t - case["pad"]) + 3 * live + t) * d * es + 4 * t * k
            flops += 4 * live * d
        return {"bytes": moved, "flops": flops}
    if op == "quantize":
        n, blocks = case["rows"] * case["cols"], case["rows"] * ((case["cols"] + 31) // 32)
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 17 * blocks, "flops": 3 * n}
    n, k, out = case["n"], case["k"], BYTES[case["out"]]
    row = k // 2 + k // 32
    if op == "gemm":
        m = case["m"]
        return {"bytes": (m + n) * row + m * n * out, "flops": 2 * m * n * k}
    rows = case["rows"]
    return {"bytes": (rows + case["active"] * n) * row + rows * n * out + 8 * (case["groups"] + 1),
            "flops": 2 * rows * n * k}


# -------------------------------------------------- the definitions, in 64 bits

def _exact_route(s):
    import numpy as np
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    t, n = x.shape
    k = c["k"]
    with np.errstate(over="ignore", invalid="ignore"):
        if c["scoring"] == "sigmoid":
            p = np.reciprocal(1 + np.exp(-x))
        else:
            m = x.max(axis=1)
            m[np.isneginf(m)] = 0
            p = np.exp(x - m[:, None])
            p /= np.maximum(p.sum(axis=1), 1e-300)[:, None]
    dead = np.isneginf(x)
    biased = s["bias"] is not None
    rank = p + s["bias"].double().cpu().numpy() if biased else x.copy()
    rank[dead] = -np.inf
    if c["groups"] > 1:
        per = n // c["groups"]
        basis = rank if biased or c["group_top"] == 1 else np.where(dead, -np.inf, p)
        parts = np.sort(basis.reshape(t, c["groups"], per), axis=2)[:, :, ::-1][:, :, :c["group_top"]].sum(axis=2)
        order = np.argsort(-parts, axis=1, kind="stable")[:, c["top_groups"]:]
        for column in order.T:
            for i in range(per):
                rank[np.arange(t), column * per + i] = -np.inf
    chosen = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    live = ~np.isneginf(np.take_along_axis(rank, chosen, axis=1))
    w = np.where(live, np.take_along_axis(p, chosen, axis=1), 0.0)
    total = w.sum(axis=1, keepdims=True) if c["renormalize"] else np.ones((t, 1))
    safe = np.where(total > 0, total, 1.0)
    weights = np.where(total > 0, c["scale"] * w / safe, 0.0)
    flat = np.where(live, chosen, n).reshape(-1)
    used = np.argsort(flat, kind="stable")[:int(live.sum())]
    rows = np.full(t * k, -1, dtype=np.int32)
    rows[used] = np.arange(used.size)
    offsets = np.searchsorted(flat[used], np.arange(n + 1), side="left")
    out = [weights, np.where(live, chosen, -1).astype(np.int32), rows.reshape(t, k), offsets.astype(np.int64)]
    if c["train"]:
        g = c["scale"] * np.where(live, s["dweights"].double().cpu().numpy(), 0.0)
        if c["renormalize"]:
            g = np.where(live & (total > 0), (g - (g * w).sum(axis=1, keepdims=True) / safe) / safe, 0.0)
        full = np.zeros((t, n))
        np.put_along_axis(full, chosen, g, axis=1)
        if c["scoring"] == "sigmoid":
            out.append(p * (1 - p) * full)
        else:
            out.append(p * full - p * (p * full).sum(axis=1, keepdims=True))
    return tuple(torch.from_numpy(v) for v in out)


def _exact_rows(s):
    d = torch.float64
    rows, y = s["rows"].long(), s["y"]
    t, k = rows.shape
    live = rows >= 0
    token, slot = live.nonzero(as_tuple=True)
    at = rows[token, slot]
    w = s["weights"].to(d)

    def summed(source, weights):
        out = torch.zeros((t, source.shape[1]), dtype=d, device="cuda")
        for j in range(k):
            of = slot == j
            part = source[at[of]].to(d)
            out[token[of]] += part if weights is None else part.mul_(weights[token[of], j].unsqueeze(1))
        return out

    out = summed(y, s["weights"].to(d))
    if not s["case"]["train"]:
        return out
    xs = torch.zeros(y.shape, dtype=d, device="cuda")
    dy = torch.zeros(y.shape, dtype=d, device="cuda")
    dw = torch.zeros((t, k), dtype=d, device="cuda")
    dout = s["dout"].to(d)
    for j in range(k):
        of = slot == j
        i, r = token[of], at[of]
        xs[r] = s["x"].to(d)[i]
        dy[r] = dout[i] * w[i, j].unsqueeze(1)
        dw[i, j] = torch.linalg.vecdot(y[r].to(d), dout[i])
    return xs, out, dy, dw, summed(s["dxs"], None)


def _exact_quantize(x):
    d = x.to(torch.float64)
    rows, cols = d.shape
    out = torch.empty_like(d)
    grid = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), dtype=torch.float64, device=x.device)
    steps = torch.tensor([2.0 ** (i - 160) for i in range(290)], dtype=torch.float64, device=x.device)
    for lo in range(0, cols, 32):
        block = d[:, lo:lo + 32]
        top = block.abs().max(dim=1, keepdim=True).values
        step = steps[torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))).long() - 2 + 160]
        a = (block.abs() / step).clamp(max=6.0)
        # the two neighbours on the grid, and the nearer one; halfway the one with an even number
        above = torch.searchsorted(grid, a.contiguous())
        below = (above - 1).clamp(min=0)
        up, down = grid[above] - a, a - grid[below]
        pick = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
        out[:, lo:lo + 32] = grid[pick] * step * torch.sign(block)
    return out


def _exact_values(q, scale):
    d = torch.float64
    both = torch.empty((q.shape[0], q.shape[1], 2), dtype=d, device=q.device)
    for i, code in enumerate((torch.bitwise_and(q, 15), torch.bitwise_right_shift(q, 4))):
        exponent, half, sign = (code // 2) % 4, (code % 2).to(d), 1.0 - 2.0 * (code // 8).to(d)
        normal = (2 + half) * torch.bitwise_left_shift(torch.ones_like(exponent), exponent).to(d) / 4
        both[:, :, i] = sign * torch.where(exponent == 0, half / 2, normal)
    powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=d, device=q.device)
    return both.view(q.shape[0], -1) * powers[scale.long()].repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "rows":
        return _exact_rows(s)
    if op == "quantize":
        return _exact_quantize(s["x"])
    a = _exact_values(s["a"], s["sa"])
    if op == "gemm":
        return torch.mm(a, _exact_values(s["b"], s["sb"]).t().contiguous())
    y = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(zip(s["ranges"][:-1], s["ranges"][1:])):
        if hi > lo:
            y[lo:hi] = torch.mm(a[lo:hi], _exact_values(s["b"][i], s["sb"][i]).t().contiguous())
    return y
