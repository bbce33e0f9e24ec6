"""What is measured of the grouped and the 8-bit integer matrix products.

Five operators:

* ``quantize``      rows of a 16- or 32-bit matrix to 8-bit integers with one scale each
* ``gemm_i8``       8-bit integer product, a scale for each row of A (token) and each row of B
                    (output channel)
* ``grouped16``     bf16/fp16 product whose rows are grouped by expert, ragged groups
* ``grouped16_bwd`` both gradients of ``grouped16``
* ``grouped_i8``    the 8-bit product, grouped by expert

`run` computes them in elementary torch operations (`own` false) or through this package's
entry points (`own` true); `exact` computes the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1}


def listed():
    return [
        # the activations of one decoding step (8 sequences) before an 8-bit layer: latency
        dict(name="quantize_decode", op="quantize", rows=8, cols=4096, dtype="bf16"),
        # the activations of a whole prompt batch, the widest layer input
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=14336, dtype="bf16"),
        # one token through the up projection of an 8-bit model: reads the weights once
        dict(name="i8_token", op="gemm_i8", m=1, n=14336, k=4096, out="bf16"),
        # a ragged batch and layer, no size a multiple of 8
        dict(name="i8_ragged", op="gemm_i8", m=1000, n=1531, k=777, out="f32"),
        # a prompt batch through the up projection
        dict(name="i8_prompt", op="gemm_i8", m=8192, n=14336, k=4096, out="bf16"),
        # decoding, 8 sequences with 2 experts each of 32: reads the chosen experts' weights once
        dict(name="experts_decode", op="grouped16", dtype="bf16", groups=32, active=13, rows=16, pad=0,
             n=4096, k=2048, trans=False, out="bf16"),
        # ragged groups, two of them empty, odd sizes, a padded row batch, weights stored N x K
        dict(name="experts_ragged", op="grouped16", dtype="f16", groups=8, active=6, rows=937, pad=63,
             n=777, k=1531, trans=True, out="f32"),
        # a prompt batch through the experts' up projection
        dict(name="experts_prompt", op="grouped16", dtype="bf16", groups=8, active=8, rows=16384, pad=0,
             n=14336, k=4096, trans=False, out="bf16"),
        # a small training batch, weight gradients kept in 32 bits for accumulation
        dict(name="experts_train_small", op="grouped16_bwd", dtype="f16", groups=8, active=7, rows=1000,
             pad=24, n=1024, k=520, trans=False, out="f32"),
        # a training batch through 16 experts, gradients in the weights' type
        dict(name="experts_train", op="grouped16_bwd", dtype="bf16", groups=16, active=16, rows=16384,
             pad=0, n=8192, k=2048, trans=False, out="bf16"),
        # decoding with 8-bit experts: one token's 8 experts of 64
        dict(name="i8_experts_decode", op="grouped_i8", groups=64, active=8, rows=8, pad=0, n=4096,
             k=2048, out="bf16"),
        # a prompt batch through 8-bit experts
        dict(name="i8_experts_prompt", op="grouped_i8", groups=16, active=15, rows=8192, pad=0, n=8192,
             k=4096, out="bf16"),
    ]


def draw(rng):
    """A case of the same ranges, no more work than the operator's largest listed one."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def size(lo, hi):
        v = spread(lo, hi)
        return v if rng.random() < 0.35 else min(hi, max(lo, (v + 8) // 16 * 16))

    op = rng.choice(["quantize", "gemm_i8", "grouped16", "grouped16", "grouped16_bwd", "grouped_i8"])
    most = max((work(c) for c in listed() if c["op"] == op), key=lambda w: w["flops"] + w["bytes"])
    while True:
        if op == "quantize":
            c = dict(op=op, rows=spread(1, 16384), cols=size(1, 16384), dtype=rng.choice(["bf16", "f16", "f32"]))
        elif op == "gemm_i8":
            c = dict(op=op, m=spread(1, 8192), n=size(16, 16384), k=size(16, 16384),
                     out=rng.choice(["bf16", "f16", "f32"]))
        else:
            groups = spread(1, 64)
            rows = spread(1, 16384)
            c = dict(op=op, groups=groups, active=rng.randint(1, min(groups, rows)), rows=rows,
                     pad=rng.choice([0, 0, rng.randint(1, 100)]), n=size(16, 14336), k=size(16, 8192))
            if op == "grouped_i8":
                c["out"] = rng.choice(["bf16", "f16", "f32"])
            else:
                c["dtype"] = rng.choice(["bf16", "f16"])
                c["trans"] = rng.random() < 0.5
                c["out"] = rng.choice([c["dtype"], "f32"])
            if c["groups"] * c["n"] * c["k"] > 16 * 8192 * 4096:
                continue
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]:
            return c


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


def _normal(shape, gen, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _int8(shape, gen):
    """8-bit values as rows of a normal matrix have them: the largest of some thousands at 127."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - at)
        flat[at:at + n] = _normal((n,), gen, 34.0).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _weights16(shape, gen, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for g in range(shape[0]):
        out[g] = _normal(shape[1:], gen, 1.0 / math.sqrt(shape[1]), dtype)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        x = _normal((case["rows"], case["cols"]), gen, 1.0, DTYPES[case["dtype"]])
        # a few channels much larger than the others, as activations have them
        x[:, ::97] *= 8
        return dict(case=case, x=x)
    out = DTYPES[case["out"]]
    if op == "gemm_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(case=case, out=out, a=_int8((m, k), gen), b=_int8((n, k), gen),
                    sa=_normal((m,), gen).abs_().mul_(0.01).add_(0.01),
                    sb=_normal((n,), gen).abs_().mul_(1e-4).add_(1e-4))
    rows = group_rows(case, seed)
    offsets = [0]
    for r in rows:
        offsets.append(offsets[-1] + r)
    total = case["rows"] + case["pad"]
    n, k, groups = case["n"], case["k"], case["groups"]
    state = dict(case=case, out=out, ranges=offsets, offsets=torch.tensor(offsets, device="cuda"))
    # with rows behind the last group the user hands in the buffer those rows keep their values in
    state["y"] = torch.zeros((total, n), dtype=out, device="cuda") if case["pad"] else None
    if op == "grouped_i8":
        state.update(a=_int8((total, k), gen), b=_int8((groups, n, k), gen),
                     sa=_normal((total,), gen).abs_().mul_(0.01).add_(0.01),
                     sb=_normal((groups, n), gen).abs_().mul_(1e-4).add_(1e-4))
        return state
    dtype = DTYPES[case["dtype"]]
    state["a"] = _normal((total, k), gen, 1.0, dtype)
    state["b"] = _weights16((groups, n, k) if case["trans"] else (groups, k, n), gen, dtype)
    if op == "grouped16_bwd":
        state["g"] = _normal((total, n), gen, 0.1, dtype)
        state["da"] = torch.zeros((total, k), dtype=dtype, device="cuda") if case["pad"] else None
    return state


# ------------------------------------------------------------------------ plain forms

def _plain_quantize(s):
    # in 64 bits: a quotient next to a half has to fall on its side
    x = s["x"].double()
    amax = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(amax > 0, x * 127.0 / amax, torch.zeros_like(x)).round()
    return q.to(torch.int8), (amax[:, 0].float() / 127.0)


def _plain_i8(a, b, sa, sb, out):
    return ((a.float() @ b.float().t()) * sa[:, None] * sb[None, :]).to(out)


def _plain_grouped(s, a, b, trans, out_dtype):
    y = torch.zeros((a.shape[0], b.shape[1] if trans else b.shape[2]), dtype=out_dtype, device="cuda")
    for g in range(b.shape[0]):
        lo, hi = s["ranges"][g], s["ranges"][g + 1]
        if hi > lo:
            w = b[g].float()
            y[lo:hi] = (a[lo:hi].float() @ (w.t() if trans else w)).to(out_dtype)
    return y


def _plain_grad_b(s, a, g_out, trans, out_dtype):
    left, right = (g_out, a) if trans else (a, g_out)
    d = torch.zeros((len(s["ranges"]) - 1, left.shape[1], right.shape[1]), dtype=out_dtype, device="cuda")
    for g in range(d.shape[0]):
        lo, hi = s["ranges"][g], s["ranges"][g + 1]
        if hi > lo:
            d[g] = (left[lo:hi].float().t() @ right[lo:hi].float()).to(out_dtype)
    return d


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return _plain_quantize(s)
    if op == "gemm_i8":
        return _plain_i8(s["a"], s["b"], s["sa"], s["sb"], s["out"])
    if op == "grouped16":
        return _plain_grouped(s, s["a"], s["b"], c["trans"], s["out"])
    if op == "grouped16_bwd":
        return (_plain_grouped(s, s["g"], s["b"], not c["trans"], s["a"].dtype),
                _plain_grad_b(s, s["a"], s["g"], c["trans"], s["out"]))
    y = torch.zeros((s["a"].shape[0], s["b"].shape[1]), dtype=s["out"], device="cuda")
    for g in range(s["b"].shape[0]):
        lo, hi = s["ranges"][g], s["ranges"][g + 1]
        if hi > lo:
            y[lo:hi] = _plain_i8(s["a"][lo:hi], s["b"][g], s["sa"][lo:hi], s["sb"][g], s["out"])
    return y


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import tiled_gemm_gemv_amd as mm
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return mm.quantize_i8(s["x"])
    if op == "gemm_i8":
        return mm.gemm_i8(s["a"], s["b"], s["sa"], s["sb"], out_dtype=s["out"])
    if op == "grouped16":
        return mm.gemm16_grouped(s["a"], s["b"], s["offsets"], trans_b=c["trans"], out=s["y"],
                                 out_dtype=s["out"])
    if op == "grouped16_bwd":
        da = mm.gemm16_grouped(s["g"], s["b"], s["offsets"], trans_b=not c["trans"], out=s["da"],
                               out_dtype=s["a"].dtype)
        left, right = (s["g"], s["a"]) if c["trans"] else (s["a"], s["g"])
        return da, mm.gemm16_grouped_grad_b(left, right, s["offsets"], out_dtype=s["out"])
    return mm.gemm_i8_grouped(s["a"], s["b"], s["offsets"], s["sa"], s["sb"], out=s["y"], out_dtype=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * BYTES[case["dtype"]] + n + 4 * case["rows"], "flops": 2 * n}
    if op == "gemm_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    rows, n, k, active, groups = (case[x] for x in ("rows", "n", "k", "active", "groups"))
    out = BYTES[case["out"]]
    if op == "grouped_i8":
        return {"bytes": rows * k + active * n * (k + 4) + 4 * rows + rows * n * out + 8 * (groups + 1),
                "flops": 2 * rows * n * k}
    if op == "grouped16":
        return {"bytes": 2 * (rows * k + active * n * k) + rows * n * out + 8 * (groups + 1),
                "flops": 2 * rows * n * k}
    return {"bytes": 2 * (rows * (2 * k + n) + active * n * k) + groups * n * k * out + 8 * (groups + 1),
            "flops": 4 * rows * n * k}


# -------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].to(torch.float64)
        top = x.abs().max(dim=1).values
        safe = torch.where(top == 0, torch.ones_like(top), top)
        return torch.round(x.mul(127.0).div(safe.unsqueeze(1))).to(torch.int8), top / 127.0
    d = torch.float64
    if op == "gemm_i8":
        acc = torch.mm(s["a"].to(d), s["b"].to(d).t().contiguous())
        return acc.mul_(s["sa"].to(d).unsqueeze(1)).mul_(s["sb"].to(d).unsqueeze(0))
    bounds = list(zip(s["ranges"][:-1], s["ranges"][1:]))
    total = case["rows"] + case["pad"]
    n, k = case["n"], case["k"]

    def weights(i):  # K x N
        w = s["b"][i].to(d)
        return w.t().contiguous() if op == "grouped_i8" or case["trans"] else w

    if op != "grouped16_bwd":
        y = torch.zeros((total, n), dtype=d, device="cuda")
        for i, (lo, hi) in enumerate(bounds):
            if lo == hi:
                continue
            part = torch.mm(s["a"][lo:hi].to(d), weights(i))
            if op == "grouped_i8":
                part = part * s["sa"][lo:hi].to(d).unsqueeze(1) * s["sb"][i].to(d)
            y[lo:hi] = part
        return y
    da = torch.zeros((total, k), dtype=d, device="cuda")
    db = torch.zeros(tuple(s["b"].shape), dtype=d, device="cuda")
    for i, (lo, hi) in enumerate(bounds):
        if lo == hi:
            continue
        grad = s["g"][lo:hi].to(d)
        da[lo:hi] = torch.mm(grad, weights(i).t().contiguous())
        each = torch.mm(s["a"][lo:hi].to(d).t().contiguous(), grad)
        db[i] = each.t() if case["trans"] else each
    return da, db
