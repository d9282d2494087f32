"""Timing cases of the fine-tuning and gated feed-forward operators.

A binarised model's feed-forward block reads x once for two projections and gates one with the other,

    h = silu(W_gate x) * (W_up x),   W[r][j] = sum_k alpha[k][r][j / 128] * B_k[r][j],  B_k in {-1, +1},

(decode: `gemv_gated`; prompts and training: `gemm_gated`).  Fine-tuning its scales against a teacher needs
the gradient of the gate (`gated_backward`), of the linear layers that share an input (`gemm_backward`: the
input's gradient and the group scales' gradients) and the loss against the teacher's top logits with its
gradient (`distill_loss`, `distill_backward`).

`run` computes a case's operator in its plain form, or, with `own` set, through the package's calls.  `exact`
computes it from the definition in 64 bits.  Weights are held in storage format 1: packed bits
[octet][kernel][16-column unit][row in octet] as 16-bit halfwords (set = +1, bit b = column 16 * unit + b) and
fp16 scales [octet][group][kernel][row in octet]; the scales' gradients have the layout of the scales, with
zeros in the rows that pad the last octet.
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- the cases -------------------------------------------------------------------------------------------------

def listed():
    return [
        # One token of a small block: launch latency is all there is.
        dict(name="gated decode b1 256x512", op="gemv_gated", kg=1, ku=1, m=256, n=512, batch=1, x="f32", h="f32"),
        # One token through the 7B block, the serving case: weights stream once.
        dict(name="gated decode b1 7B", op="gemv_gated", kg=3, ku=3, m=11008, n=4096, batch=1, x="bf16", h="bf16"),
        # Seven sequences decoded together in the 13B block, each projection with its own number of kernels.
        dict(name="gated decode b7 13B", op="gemv_gated", kg=4, ku=2, m=13824, n=5120, batch=7, x="bf16", h="bf16"),
        # A short prompt through a block of odd sizes.
        dict(name="gated tokens 77 odd", op="gemm_gated", kg=2, ku=1, m=1001, n=640, tokens=77, keep=False),
        # A training step's forward pass of the 7B block: the two projections are kept for the backward pass.
        dict(name="gated tokens 2048 7B", op="gemm_gated", kg=3, ku=3, m=11008, n=4096, tokens=2048, keep=True),
        # The gate's gradient in a small ragged batch.
        dict(name="gate gradient 33x1001", op="gated_backward", m=1001, tokens=33, remake=False),
        # The gate's gradient of the 7B block, the block's output made again for the projection that follows.
        dict(name="gate gradient 2048 7B", op="gated_backward", m=11008, tokens=2048, remake=True),
        # Query, key and value of a small layer with grouped heads, odd rows and a ragged batch.
        dict(name="layer gradient qkv small", op="gemm_backward", k="2,1,3", m="200,77,77", n=640, tokens=130),
        # Gate and up of the 7B block in a training step.
        dict(name="layer gradient 7B", op="gemm_backward", k="3,3", m="11008,11008", n=4096, tokens=2048),
        # A few sequences' last tokens against a teacher's top 16: a small ragged batch, loss and gradient apart.
        dict(name="distill 9x32001 apart", op="distill", v=32001, tokens=9, top=16, logits="f32", temp=2.0, fused=False,
             masked=True),
        # A training step's tokens against a teacher's top 64, loss and gradient in one call.
        dict(name="distill 2048x32000", op="distill", v=32000, tokens=2048, top=64, logits="bf16", temp=1.0, fused=True,
             masked=False),
        # The same in 32 bits with prompt tokens masked out, the loss first and the gradient later.
        dict(name="distill 1024x32000 apart", op="distill", v=32000, tokens=1024, top=32, logits="f32", temp=2.0,
             fused=False, masked=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _cols(rng, high):
    return 128 * _log(rng, 1, high // 128)


def draw(rng):
    op = rng.choice(["gemv_gated", "gemv_gated", "gemm_gated", "gemm_gated", "gated_backward", "gemm_backward",
                     "gemm_backward", "distill", "distill"])
    if op == "gemv_gated":
        return dict(op=op, kg=rng.randint(1, 4), ku=rng.randint(1, 4), m=_log(rng, 64, 13824), n=_cols(rng, 5120),
                    batch=rng.choice([1, 1, 2, 3, 5, 8, 11, 16]), x=rng.choice(["f32", "bf16", "bf16"]),
                    h=rng.choice(["f32", "bf16"]))
    if op == "gemm_gated":
        return dict(op=op, kg=rng.randint(1, 4), ku=rng.randint(1, 4), m=_log(rng, 64, 11008), n=_cols(rng, 4096),
                    tokens=_log(rng, 17, 2048), keep=rng.random() < 0.5)
    if op == "gated_backward":
        return dict(op=op, m=_log(rng, 64, 11008), tokens=_log(rng, 1, 2048), remake=rng.random() < 0.5)
    if op == "gemm_backward":
        parts = rng.randint(1, 3)
        return dict(op=op, k=",".join(str(rng.randint(1, 4)) for _ in range(parts)),
                    m=",".join(str(_log(rng, 64, 11008 if parts < 3 else 5120)) for _ in range(parts)),
                    n=_cols(rng, 4096), tokens=_log(rng, 17, 2048))
    v = _log(rng, 1000, 128000)
    return dict(op=op, v=v, tokens=_log(rng, 1, min(2048, 32000 * 2048 // v)), top=_log(rng, 1, 128),
                logits=rng.choice(["f32", "bf16", "bf16"]), temp=rng.choice([1.0, 2.0, 3.5]), fused=rng.random() < 0.5,
                masked=rng.random() < 0.5)


def _ints(text):
    return [int(v) for v in text.split(",")]


def work(case):
    op = case["op"]
    if op in ("gemv_gated", "gemm_gated"):
        m, n = case["m"], case["n"]
        rows = case["batch"] if op == "gemv_gated" else case["tokens"]
        xb = 4 if case.get("x") == "f32" else 2
        hb = 4 if case.get("h") == "f32" else 2
        weights = (case["kg"] + case["ku"]) * (m * n // 8 + m * (n // GROUP) * 2)
        out = rows * m * hb * (3 if case.get("keep") else 1)
        return {"bytes": weights + rows * n * xb + out, "flops": 2 * 2 * rows * m * n}
    if op == "gated_backward":
        elems = case["m"] * case["tokens"]
        return {"bytes": 2 * elems * (6 if case["remake"] else 5), "flops": 12 * elems}
    if op == "gemm_backward":
        n, t = case["n"], case["tokens"]
        total = {"bytes": 2 * 2 * t * n, "flops": 0}
        for k, m in zip(_ints(case["k"]), _ints(case["m"])):
            total["bytes"] += k * (m * n // 8 + m * (n // GROUP) * (2 + 4)) + 2 * t * m
            total["flops"] += 2 * 2 * t * m * n
        return total
    size = case["tokens"] * case["v"] * (4 if case["logits"] == "f32" else 2)
    # fused: the logits in, their gradient out; apart, the second call reads the logits again
    return {"bytes": size * (2 if case["fused"] else 3) + case["tokens"] * (case["top"] * 8 + 16),
            "flops": case["tokens"] * case["v"] * 8}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _weights(g, k, m, n):
    """Random kernels and decaying scales in storage format 1."""
    octets = (m + 7) // 8
    packed = torch.randint(0, 256, (octets * k * n,), generator=g, device="cuda", dtype=torch.uint8).view(torch.int32)
    decay = 0.02 * 2.0 ** -torch.arange(k, device="cuda", dtype=torch.float32)
    a = (0.5 + torch.rand(octets, n // GROUP, k, 8, generator=g, device="cuda")) * decay[:, None]
    return packed, a.to(torch.float16).reshape(-1)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    bf16 = torch.bfloat16
    if op in ("gemv_gated", "gemm_gated"):
        m, n = case["m"], case["n"]
        s["gate"] = _weights(g, case["kg"], m, n)
        s["up"] = _weights(g, case["ku"], m, n)
        rows = case["batch"] if op == "gemv_gated" else case["tokens"]
        s["x"] = _normal(g, (rows, n), DTYPES[case.get("x", "bf16")])
        s["h"] = torch.empty(rows, m, device="cuda", dtype=DTYPES[case.get("h", "bf16")])
        if case.get("keep"):
            s["g"], s["u"] = (torch.empty(rows, m, device="cuda", dtype=bf16) for _ in range(2))
    elif op == "gated_backward":
        shape = (case["tokens"], case["m"])
        s["dh"] = _normal(g, shape, bf16, 1e-2)
        s["g"], s["u"] = _normal(g, shape, bf16, 1.3), _normal(g, shape, bf16, 1.3)
        s["out"] = [torch.empty(shape, device="cuda", dtype=bf16) for _ in range(3 if case["remake"] else 2)]
    elif op == "gemm_backward":
        n, t = case["n"], case["tokens"]
        s["k"], s["m"] = _ints(case["k"]), _ints(case["m"])
        s["w"] = [_weights(g, k, m, n) for k, m in zip(s["k"], s["m"])]
        s["x"] = _normal(g, (t, n), bf16)
        s["dy"] = [_normal(g, (t, m), bf16, 1e-2) for m in s["m"]]
        s["dx"] = torch.empty(t, n, device="cuda", dtype=bf16)
        s["da"] = [torch.empty(a.numel(), device="cuda", dtype=torch.float32) for _, a in s["w"]]
    else:
        t, v, top = case["tokens"], case["v"], case["top"]
        dt = DTYPES[case["logits"]]
        # one entry in each of `top` equal parts of the vocabulary; the student has learnt some of it already
        at = torch.arange(top, device="cuda") + torch.rand(t, top, generator=g, device="cuda")
        index = (at * (v / top)).to(torch.int32).clamp_(0, v - 1)
        teacher = 6.0 + 2.0 * torch.randn(t, top, generator=g, device="cuda")
        z = 2.0 * torch.randn(t, v, generator=g, device="cuda")
        z.scatter_(1, index.long(), teacher - 1.0 + torch.randn(t, top, generator=g, device="cuda"))
        weight = torch.rand(t, generator=g, device="cuda") + 0.5
        if case["masked"]:
            # prompt tokens have no weight, some lists are shorter, some are empty
            weight[torch.rand(t, generator=g, device="cuda") < 0.25] = 0.0
            short = torch.rand(t, 1, generator=g, device="cuda") * 1.3
            index = torch.where(torch.arange(top, device="cuda") < (short * top).ceil(), index, torch.full_like(index, -1))
            index[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
        s["z"], s["teacher"], s["index"], s["weight"] = z.to(dt), teacher, index.contiguous(), weight / t
        s["grad"] = torch.rand(t, generator=g, device="cuda") + 0.5
        s["loss"], s["lse"] = (torch.empty(t, device="cuda", dtype=torch.float32) for _ in range(2))
        s["dz"] = torch.empty(t, v, device="cuda", dtype=dt)
    return s


# ---- one pass --------------------------------------------------------------------------------------------------

def _signs(packed, k, m, n):
    """The K sign matrices [k][8 * octets][n] as fp32."""
    octets = (m + 7) // 8
    b = packed.view(torch.uint8).view(octets, k, n // 16, 8, 2)
    bits = (b.unsqueeze(-1) >> torch.arange(8, device=b.device, dtype=torch.uint8)) & 1     # [o][k][q][row][byte][bit]
    return (2.0 * bits.float() - 1.0).permute(1, 0, 3, 2, 4, 5).reshape(k, octets * 8, n)


def _dense(weights, k, m, n):
    """W [m][n] in fp32."""
    packed, alpha = weights
    octets = (m + 7) // 8
    a = alpha.float().view(octets, n // GROUP, k, 8).permute(2, 0, 3, 1).reshape(k, octets * 8, n // GROUP, 1)
    w = (a * _signs(packed, k, m, n).view(k, octets * 8, n // GROUP, GROUP)).sum(0)
    return w.view(octets * 8, n)[:m]


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    gate = x @ _dense(s["gate"], c["kg"], c["m"], c["n"]).T
    up = x @ _dense(s["up"], c["ku"], c["m"], c["n"]).T
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(s["h"].dtype)
    return (h, gate.to(torch.bfloat16), up.to(torch.bfloat16)) if c.get("keep") else h


def _plain_gated_backward(s):
    dh, g, u = s["dh"].float(), s["g"].float(), s["u"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    out = [dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig]
    if s["case"]["remake"]:
        out.append(g * sig * u)
    return [t.to(torch.bfloat16) for t in out]


def _plain_gemm_backward(s):
    n = s["case"]["n"]
    x = s["x"].float()
    dx, das = torch.zeros_like(x), []
    for weights, k, m, dy in zip(s["w"], s["k"], s["m"], s["dy"]):
        octets = (m + 7) // 8
        dx += dy.float() @ _dense(weights, k, m, n)
        dw = torch.zeros(octets * 8, n, device=x.device)
        dw[:m] = dy.float().T @ x
        da = (_signs(weights[0], k, m, n) * dw).view(k, octets, 8, n // GROUP, GROUP).sum(-1)   # [k][o][row][g]
        das.append(da.permute(1, 3, 0, 2).reshape(-1))
    return dx.to(torch.bfloat16), das


def _plain_distill(s):
    c = s["case"]
    temp = c["temp"]
    valid = s["index"] >= 0
    at = s["index"].clamp(min=0).long()
    weight = torch.where(valid.any(1), s["weight"], torch.zeros_like(s["weight"]))
    # the teacher's distribution over its valid entries
    tv = torch.where(valid, s["teacher"], torch.full_like(s["teacher"], -math.inf)) / temp
    top = tv.max(1, keepdim=True).values
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(tv - top)
    total = e.sum(1, keepdim=True).clamp(min=1e-30)
    p = e / total
    logp = tv - top - torch.log(total)
    # the student's over the whole vocabulary
    z = s["z"].float() / temp
    high = z.max(1, keepdim=True).values
    ez = torch.exp(z - high)
    zsum = ez.sum(1, keepdim=True)
    lse = high + torch.log(zsum)
    term = torch.where(p > 0, p * (logp - (z.gather(1, at) - lse)), torch.zeros_like(p)).sum(1)
    used = weight != 0
    loss = torch.where(used, weight * term, torch.zeros_like(term))
    scale = weight / temp if c["fused"] else weight * s["grad"] / temp
    dz = (ez / zsum).scatter_add_(1, at, -p) * scale[:, None]
    dz = torch.where(used[:, None], dz, torch.zeros_like(dz))
    return loss, torch.where(used, lse[:, 0], torch.zeros_like(loss)), dz.to(s["z"].dtype)


def _plain(s):
    op = s["case"]["op"]
    if op in ("gemv_gated", "gemm_gated"):
        return _plain_gated(s)
    if op == "gated_backward":
        return _plain_gated_backward(s)
    if op == "gemm_backward":
        return _plain_gemm_backward(s)
    return _plain_distill(s)


def _own(s):
    import boolean_weight_matmul_b200 as mb

    c = s["case"]
    op = c["op"]
    code = {"f32": mb.F32, "bf16": mb.BF16}
    if op == "gemv_gated":
        if "ws" not in s:
            s["ws"] = mb.empty_gated_workspace(c["kg"], c["ku"], c["m"], c["n"], c["batch"])
        mb.gemv_gated(*s["gate"], c["kg"], *s["up"], c["ku"], c["m"], c["n"], GROUP, s["x"], code[c["x"]], c["batch"],
                      s["h"], code[c["h"]], s["ws"])
        return s["h"]
    if op == "gemm_gated":
        if "ws" not in s:
            s["ws"] = mb.empty_gemm_gated_workspace(c["m"], c["n"], c["tokens"])
        mb.gemm_gated(*s["gate"], c["kg"], *s["up"], c["ku"], c["m"], c["n"], GROUP, s["x"], c["tokens"], s["h"],
                      s.get("g"), s.get("u"), s["ws"])
        return (s["h"], s["g"], s["u"]) if c["keep"] else s["h"]
    if op == "gated_backward":
        mb.gated_backward(s["dh"], s["g"], s["u"], c["tokens"], c["m"], *s["out"])
        return s["out"]
    if op == "gemm_backward":
        if "ws" not in s:
            s["ws"] = mb.empty_gemm_backward_workspace(s["k"], s["m"], c["n"], c["tokens"])
        mb.gemm_backward([w[0] for w in s["w"]], [w[1] for w in s["w"]], s["k"], s["m"], c["n"], GROUP, s["x"],
                         c["tokens"], s["dy"], s["dx"], s["da"], s["ws"])
        return s["dx"], s["da"]
    v = c["v"]
    mb.distill_loss(s["z"], code[c["logits"]], c["tokens"], v, v, s["teacher"], s["index"], c["top"], c["temp"],
                    s["weight"], s["loss"], s["lse"], s["dz"] if c["fused"] else None, v)
    if not c["fused"]:
        mb.distill_backward(s["z"], code[c["logits"]], c["tokens"], v, v, s["teacher"], s["index"], c["top"], c["temp"],
                            s["weight"], s["lse"], s["grad"], s["dz"], v)
    return s["loss"], s["lse"], s["dz"]


def run(state):
    return _own(state) if own else _plain(state)


# ---- from the definition, in 64 bits -----------------------------------------------------------------------------

def _exact_planes(packed, k, m, n):
    """+-1 planes [k][m][n] in int8, gathered bit by bit from the halfwords of each row."""
    words = packed.view(torch.int16).view(-1, k, n // 16, 8)            # [octet][kernel][unit][row]
    planes = torch.empty(k, words.shape[0], 8, n // 16, 16, dtype=torch.int8, device=packed.device)
    for b in range(16):
        planes[..., b] = (torch.bitwise_and(words, 1 << b if b < 15 else -32768) != 0).permute(1, 0, 3, 2).to(torch.int8)
    return (2 * planes - 1).reshape(k, -1, n)[:, :m]


def _exact_weight(weights, k, m, n):
    planes = _exact_planes(weights[0], k, m, n)
    scales = weights[1].double().view(-1, n // GROUP, k, 8)
    w = torch.zeros(m, n, dtype=torch.float64, device=planes.device)
    for i in range(k):
        per_row = scales[:, :, i].transpose(1, 2).reshape(-1, n // GROUP)[:m]
        w += per_row.repeat_interleave(GROUP, dim=1) * planes[i]
    return w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gemv_gated", "gemm_gated"):
        m, n = case["m"], case["n"]
        x = s["x"].double()
        a = torch.einsum("tn,mn->tm", x, _exact_weight(s["gate"], case["kg"], m, n))
        b = torch.einsum("tn,mn->tm", x, _exact_weight(s["up"], case["ku"], m, n))
        h = a * torch.special.expit(a) * b
        return (h, a, b) if case.get("keep") else h
    if op == "gated_backward":
        d, a, b = s["dh"].double(), s["g"].double(), s["u"].double()
        e = torch.special.expit(a)
        out = [d * b * (e + a * e * torch.special.expit(-a)), d * a * e]
        return out + [a * e * b] if case["remake"] else out
    if op == "gemm_backward":
        n, x = case["n"], s["x"].double()
        dx, das = torch.zeros_like(x), []
        for weights, k, m, dy in zip(s["w"], s["k"], s["m"], s["dy"]):
            d = dy.double()
            dx += torch.einsum("tm,mn->tn", d, _exact_weight(weights, k, m, n))
            full = torch.einsum("tm,tn->mn", d, x)
            planes = _exact_planes(weights[0], k, m, n)
            octets = (m + 7) // 8
            da = torch.zeros(octets, n // GROUP, k, 8, dtype=torch.float64, device=x.device)
            for i in range(k):
                sums = torch.zeros(octets * 8, n // GROUP, dtype=torch.float64, device=x.device)
                sums[:m] = (full * planes[i]).unflatten(1, (-1, GROUP)).sum(2)
                da[:, :, i] = sums.view(octets, 8, -1).transpose(1, 2)
            das.append(da.reshape(-1))
        return dx, das
    temp = case["temp"]
    z = s["z"].double() / temp
    lse = torch.logsumexp(z, 1)
    valid = s["index"] >= 0
    some = valid.any(1) & (s["weight"] != 0)
    tv = s["teacher"].double().div(temp).masked_fill(~valid, -math.inf)
    tv[~valid.any(1)] = 0.0
    logp = torch.log_softmax(tv, 1).masked_fill(~valid, -math.inf)
    p = logp.exp()
    at = s["index"].long().masked_fill(~valid, 0)
    gap = (logp - z.gather(1, at) + lse[:, None]).masked_fill(~valid, 0.0)
    w = s["weight"].double() * some
    loss = w * (p * gap).sum(1)
    dz = torch.exp(z - lse[:, None])
    dz.scatter_add_(1, at, -p)
    dz *= (w / temp * (1.0 if case["fused"] else s["grad"].double()))[:, None]
    return loss, lse * some, dz
