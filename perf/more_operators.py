"""Cases of the operators on microscaled 4-bit numbers (e2m1 elements, one e8m0
scale for each 32 of a row): quantisation and its inverse, products with
weights in that format, and a mixture-of-experts layer for a few tokens on
experts in it.

`run` computes an operator in plain torch (32-bit, rounded once at the end), or
through the package's entry points where `own` is true.
"""
import math

import torch

own = False

BLOCK = 32       # elements that share a scale
DEV = "cuda"


def listed():
    return [
        # one token's activations, there and back: latency
        dict(name="quant 1x7168", op="quant", rows=1, k=7168, pad=0),
        # columns of a wider projection's output, an odd number of blocks
        dict(name="quant 777x2080 of columns", op="quant", rows=777, k=2080, pad=72),
        # a calibration's round trip over a prefill's activations
        dict(name="quant 16384x7168", op="quant", rows=16384, k=7168, pad=0),
        # one token's projection, bf16 activations: latency
        dict(name="proj 1x7168x1536", op="proj", rows=1, k=7168, n=1536, pad=0),
        # a decode batch through a large projection
        dict(name="proj 16x7168x14336", op="proj", rows=16, k=7168, n=14336, pad=0),
        # the largest decode batch, columns of a wider matrix, an odd number of outputs
        dict(name="proj 61x2080x7171", op="proj", rows=61, k=2080, n=7171, pad=64),
        # a step's activations quantised in front of the product: few tokens
        dict(name="linear 16x7168x7168", op="linear", rows=16, k=7168, n=7168, pad=0),
        # a short prompt, odd sizes
        dict(name="linear 300x4128x2050", op="linear", rows=300, k=4128, n=2050, pad=32),
        # a prefill's projection
        dict(name="linear 8192x7168x7168", op="linear", rows=8192, k=7168, n=7168, pad=0),
        # one user's next token through a device's share of a large layer: latency
        dict(name="moe 1 of 256", op="moe", rows=1, pads=0, k=7168, inter=512, experts=256, top=8, shared=1,
             scoring="sigmoid", bias=True, renorm=True),
        # a captured step's padded batch, softmax scores, few experts, odd numbers of blocks
        dict(name="moe 21 of 40 softmax", op="moe", rows=21, pads=5, k=2080, inter=1056, experts=40, top=4,
             shared=0, scoring="softmax", bias=False, renorm=False),
        # the largest step: every expert is read
        dict(name="moe 64 of 256", op="moe", rows=64, pads=0, k=7168, inter=512, experts=256, top=8, shared=1,
             scoring="sigmoid", bias=True, renorm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "proj", "linear", "moe"])
    k = BLOCK * _log(rng, 8, 256)
    pad = rng.choice([0, 8 * rng.randrange(1, 32)])
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, min(16384, 117440512 // k)), k=k, pad=pad)
    if op == "proj":
        return dict(op=op, rows=_log(rng, 1, 64), k=k, n=_log(rng, 64, 12000), pad=pad)
    if op == "linear":
        n = _log(rng, 64, 12000)
        return dict(op=op, rows=_log(rng, 1, min(8192, 420000000000 // (k * n))), k=k, n=n, pad=pad)
    inter = BLOCK * _log(rng, 4, 64)
    experts = min(_log(rng, 4, 256), 940000000 // (k * inter))
    rows = _log(rng, 1, 64)
    return dict(op=op, rows=rows, pads=rng.choice([0, rng.randrange(rows)]), k=k, inter=inter, experts=experts,
                top=rng.randrange(1, min(8, experts) + 1), shared=rng.choice([0, 0, 1, 2]),
                scoring=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5, renorm=rng.random() < 0.5)


ROUTE_SCALE = 2.5


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def weights(rows, k):
        """Codes of every kind, and scales that make rows of about unit norm."""
        codes = torch.randint(0, 256, (*rows, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        mid = 127 - round(math.log2(3 * math.sqrt(k)))
        return codes, torch.randint(mid - 1, mid + 2, (*rows, k // BLOCK), generator=gen, device=DEV,
                                    dtype=torch.uint8)

    s = dict(case)
    m, k = case["rows"], case["k"]
    wide = k + (case.get("pad") or 0)
    # channels of unequal size, as activations have them
    s["x"] = (rnd(m, wide) * (0.7 * rnd(wide)).exp()).to(torch.bfloat16)[:, wide - k:]
    if case["op"] in ("quant", "linear"):
        s["codes"] = torch.empty(m, k // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(m, k // BLOCK, dtype=torch.uint8, device=DEV)
    if case["op"] == "quant":
        s["values"] = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    elif case["op"] in ("proj", "linear"):
        s["w"], s["w_scale"] = weights((case["n"],), k)
        s["y"] = torch.empty(m, case["n"], dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "moe":
        e, i = case["experts"], case["inter"]
        every = e + case["shared"]
        s["x"] = rnd(m, k).to(torch.bfloat16)
        s["router"] = (rnd(e, k) / math.sqrt(k)).to(torch.bfloat16)
        s["router_bias"] = 0.05 * rnd(e) if case["bias"] else None
        s["w_up"], s["w_up_scale"] = weights((every, 2 * i), k)
        s["w_down"], s["w_down_scale"] = weights((every, k), i)
        s["out"] = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
        s["ids"] = torch.empty(m, case["top"], dtype=torch.int32, device=DEV)
        s["gates"] = torch.empty(m, case["top"], dtype=torch.float32, device=DEV)
        slots = torch.randperm(2 * m, generator=gen, device=DEV)[:m].to(torch.int32)
        if case["pads"]:
            slots[m - case["pads"]:] = -1
        s["slots"] = slots if case["pads"] else None
    return s


# ---- the plain forms -------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _plain_values(codes, scales):
    """What codes [..., K / 2] and scales [..., K / 32] stand for, fp32 [..., K]."""
    one = torch.tensor(_E2M1, device=DEV)
    pairs = torch.stack((one.repeat(16), one.repeat_interleave(16)), 1)  # low four bits first
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK))
    return (v * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _plain_quant(s):
    """Codes 0..15 and scales of x: the scale is the power of two that takes the largest into [4, 8)."""
    x = s["x"].float().unflatten(1, (-1, BLOCK))
    big = x.abs().amax(-1)
    code = torch.where(big > 0, torch.frexp(big).exponent.int() - 1 - 2 + 127, 0).clamp(0, 254)
    v = x.double() * torch.exp2((127 - code).double())[..., None]
    a = v.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (a / step).round() * step  # ties to the even code
    return torch.where(v < 0, -a, a).float(), code


def _plain_moe(s):
    e, k, i, top = s["experts"], s["k"], s["inter"], s["top"]
    live = slice(0, s["rows"] - s["pads"])
    x = s["x"][live]
    m = x.shape[0]
    # scores next to each other: 64 bits
    logits = x.double() @ s["router"].double().T
    if s["scoring"] == "sigmoid":
        score = 1 / (1 + (-logits).exp())
    else:
        score = (logits - logits.amax(1, keepdim=True)).exp()
        score = score / score.sum(1, keepdim=True)
    ranked = score if s["router_bias"] is None else score + s["router_bias"].double()
    ids = torch.sort(ranked, dim=1, descending=True, stable=True).indices[:, :top]
    gates = score.gather(1, ids)
    if s["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    gates = (gates * ROUTE_SCALE).float()
    every = e + s["shared"]
    al = torch.zeros(m, every, device=DEV).scatter(1, ids, gates)
    al[:, e:] = 1
    if m * top < e:  # the experts of each token
        which = torch.cat((ids, torch.arange(e, every, device=DEV).expand(m, -1)), 1)
        w = _plain_values(s["w_up"][which], s["w_up_scale"][which])
        h = (w * x.float()[:, None, None]).sum(-1)
        h = h[..., :i] / (1 + (-h[..., :i]).exp()) * h[..., i:]
        w = _plain_values(s["w_down"][which], s["w_down_scale"][which])
        y = ((w * h[:, :, None]).sum(-1) * al.gather(1, which)[..., None]).sum(1)
    else:  # every expert for every token
        w = _plain_values(s["w_up"].flatten(0, 1), s["w_up_scale"].flatten(0, 1))
        h = (x.float() @ w.T).unflatten(1, (every, 2 * i))
        h = h[..., :i] / (1 + (-h[..., :i]).exp()) * h[..., i:]
        h = (h * al[..., None]).transpose(0, 1)
        y = (h @ _plain_values(s["w_down"], s["w_down_scale"]).transpose(1, 2)).sum(0)
    s["out"][live] = y.to(torch.bfloat16)
    s["ids"].fill_(-1)[live] = ids.int()
    s["gates"].zero_()[live] = gates
    return {"out": s["out"], "ids": s["ids"], "gates": s["gates"]}


def _plain(s):
    if s["op"] == "moe":
        return _plain_moe(s)
    if s["op"] == "proj":
        s["y"].copy_(s["x"].float() @ _plain_values(s["w"], s["w_scale"]).T)
        return {"y": s["y"]}
    v, code = _plain_quant(s)
    v = (v * (code << 23).view(torch.float32)[..., None]).flatten(1)
    if s["op"] == "quant":
        s["values"].copy_(v)
        s["scales"].copy_(code)
        return {"values": s["values"], "scales": s["scales"].view(torch.float8_e8m0fnu)}
    s["y"].copy_(v @ _plain_values(s["w"], s["w_scale"]).T)
    return {"y": s["y"]}


def _own(s):
    import gated_delta_rule_tok_amd as kda
    op = s["op"]
    if op == "quant":
        kda.kda_mx4_quant(s["x"], s["codes"], s["scales"])
        kda.kda_mx4_dequant(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"].view(torch.float8_e8m0fnu)}
    if op == "proj":
        kda.kda_mx4_proj(s["x"], None, s["w"], s["w_scale"], s["y"])
        return {"y": s["y"]}
    if op == "linear":
        kda.kda_mx4_quant(s["x"], s["codes"], s["scales"])
        kda.kda_mx4_proj(s["codes"], s["scales"], s["w"], s["w_scale"], s["y"])
        return {"y": s["y"]}
    if "ws" not in s:  # kept for the calls that follow, as a server keeps it
        s["ws"] = torch.empty(kda.kda_mx4_moe_workspace_size(s["rows"], s["k"], s["inter"], s["experts"],
                                                             s["shared"], s["top"]),
                              dtype=torch.uint8, device=DEV)
    kda.kda_mx4_moe(s["x"], s["router"], s["router_bias"], s["w_up"], s["w_up_scale"], s["w_down"],
                    s["w_down_scale"], s["out"], s["ids"], s["gates"], s["ws"], scoring=s["scoring"],
                    renormalise=s["renorm"], route_scale=ROUTE_SCALE, state_indices=s["slots"])
    return {"out": s["out"], "ids": s["ids"], "gates": s["gates"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the work --------------------------------------------------------------

def work(case):
    op, m, k = case["op"], case["rows"], case["k"]
    if op == "quant":  # bf16 in, 4 bits and scales out, and back
        return {"bytes": 2 * (2 * m * k + m * k // 2 + m * k // BLOCK), "flops": 4 * m * k}
    if op in ("proj", "linear"):
        n = case["n"]
        return {"bytes": n * k // 2 + n * k // BLOCK + 2 * m * (k + n), "flops": 2 * m * n * k}
    e, i, top, shared = case["experts"], case["inter"], case["top"], case["shared"]
    m -= case["pads"]
    hit = e * (1 - (1 - top / e) ** m) + shared  # experts that at least one token takes, on average
    one = 3 * i * (k // 2 + k // BLOCK)
    return {"bytes": int(hit * one) + 2 * e * k + 4 * m * k + 8 * m * top,
            "flops": 2 * m * k * (e + 3 * i * (top + shared))}


# ---- 64 bits, from the definitions ------------------------------------------

def _decode(codes, scales):
    """[R, K / 2], [R, K / 32] -> fp64 [R, K], bit by bit."""
    c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.uint8, device=DEV)
    c[:, 0::2] = codes % 16
    c[:, 1::2] = codes // 16
    sign = 1.0 - 2.0 * (c // 8).double()
    power, half = (c % 8 // 2).double(), (c % 2).double() / 2
    size = torch.where(power > 0, (1 + half) * torch.exp2(power - 1), half)
    at = torch.arange(c.shape[1], device=DEV) // BLOCK
    return sign * size * torch.exp2(scales.double() - 127)[:, at]


def _nearest(x):
    """x as microscaled 4-bit numbers and its scales, fp64."""
    m, k = x.shape
    x = x.double().reshape(m, k // BLOCK, BLOCK)
    big = x.abs().amax(2)
    scale = torch.exp2((torch.floor(torch.log2(big)) - 2).clamp(-127, 127))
    t = x / scale[:, :, None]
    unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=1.0))) - 1)
    return ((t / unit).round() * unit).clamp(-6, 6).mul(scale[:, :, None]).reshape(m, k), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        v, scale = _nearest(s["x"])
        return {"values": v, "scales": scale}
    if op in ("proj", "linear"):
        x = s["x"].double() if op == "proj" else _nearest(s["x"])[0]
        return {"y": torch.matmul(x, _decode(s["w"], s["w_scale"]).T)}
    m, e, top, i = case["rows"] - case["pads"], case["experts"], case["top"], case["inter"]
    x = s["x"][:m].double()
    logits = torch.matmul(x, s["router"].double().T)
    score = torch.sigmoid(logits) if case["scoring"] == "sigmoid" else torch.softmax(logits, 1)
    ranked = score.clone() if s["router_bias"] is None else score + s["router_bias"].double()
    ids = torch.full((case["rows"], top), -1, dtype=torch.int32, device=DEV)
    gates = torch.zeros(case["rows"], top, dtype=torch.float64, device=DEV)
    row = torch.arange(m, device=DEV)
    for j in range(top):  # the largest that is left, the first of equals
        best = torch.where(ranked == ranked.amax(1, keepdim=True), torch.arange(e, device=DEV), e).amin(1)
        ids[:m, j] = best.int()
        gates[:m, j] = score[row, best]
        ranked[row, best] = -math.inf
    if case["renorm"]:
        gates[:m] /= gates[:m].sum(1, keepdim=True)
    gates[:m] *= ROUTE_SCALE
    out = s["out"].double()
    for j in range(e + case["shared"]):
        hit = ids[:m] == j
        at = hit.any(1).nonzero()[:, 0] if j < e else row
        if not len(at):
            continue
        gate = (gates[:m] * hit)[at].sum(1) if j < e else torch.ones(m, dtype=torch.float64, device=DEV)
        both = torch.matmul(x[at], _decode(s["w_up"][j], s["w_up_scale"][j]).T)
        h = both[:, :i] * torch.sigmoid(both[:, :i]) * both[:, i:]
        out[at] += gate[:, None] * torch.matmul(h, _decode(s["w_down"][j], s["w_down_scale"][j]).T)
    return {"out": out, "ids": ids, "gates": gates}
