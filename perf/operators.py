"""Cases of the operators around the gated delta rule: its chunked prefill and
its single-token step with one decay per head, the residual's addition with the
RMS norm, and products with 4-bit weights.

`run` computes an operator in plain torch (32-bit, rounded once at the end), or
through the package's entry points where `own` is true.
"""
import math

import torch

own = False

D = 128          # head_dim of the delta rule
CHUNK = 64       # tokens per chunk of the plain form
EPS = 1e-6
DEV = "cuda"
FP8_MAX = 448.0  # largest e4m3 value

_STATE = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the layer's headline batch: eight prompts of 2048 tokens, key heads shared by two value heads
        dict(name="prefill 8x2048", op="prefill", seqs=8, tokens=16384, ragged=False, hk=8, hv=16,
             state="fp32", initial=True, packed=False),
        # a serving step's ragged prompts, q, k, v, a and beta as columns of one projection's output
        dict(name="prefill ragged 32", op="prefill", seqs=32, tokens=30011, ragged=True, hk=16, hv=32,
             state="bf16", initial=True, packed=True),
        # one long document on a device's share of the heads, starting from nothing
        dict(name="prefill 1x8192", op="prefill", seqs=1, tokens=8192, ragged=False, hk=4, hv=8,
             state="bf16", initial=False, packed=True),
        # one user's next token: latency
        dict(name="decode 1", op="decode", seqs=1, slots=8, pad=0, hk=8, hv=16, state="fp32", packed=True),
        # a padded batch of a captured step, states kept in bf16
        dict(name="decode 37 of 48", op="decode", seqs=48, slots=77, pad=11, hk=16, hv=32, state="bf16",
             packed=True),
        # a full decode batch
        dict(name="decode 256", op="decode", seqs=256, slots=300, pad=0, hk=16, hv=16, state="fp32",
             packed=False),
        # the norm before one token's projections: latency
        dict(name="norm 1x7168", op="norm", rows=1, dim=7168, out="bf16", group=0, residual=True),
        # a prefill's rows into 8 bits with a scale for each 128 channels
        dict(name="norm 16384x7168 fp8 groups", op="norm", rows=16384, dim=7168, out="fp8", group=128,
             residual=True),
        # an odd width, a scale per row, no residual
        dict(name="norm 777x2050 fp8 rows", op="norm", rows=777, dim=2050, out="fp8", group=0,
             residual=False),
        # one token's projection
        dict(name="w4 1x7168x1536", op="w4", rows=1, k=7168, n=1536, group=128, zeros=False),
        # a decode batch through a large projection, asymmetric weights
        dict(name="w4 16x7168x14336", op="w4", rows=16, k=7168, n=14336, group=64, zeros=True),
        # the largest batch, fine groups, an odd number of outputs
        dict(name="w4 61x2048x7171", op="w4", rows=61, k=2048, n=7171, group=32, zeros=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "norm", "w4"])
    if op == "prefill":
        hk, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 2, 4])
        hv = min(32, hk * group)
        seqs = _log(rng, 1, 32)
        tokens = seqs * _log(rng, 1, 2048) + rng.randrange(64)
        tokens = min(tokens, 16384, 262144 // hv)
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=rng.random() < 0.7, hk=hk, hv=hv,
                    state=rng.choice(["fp32", "bf16"]), initial=rng.random() < 0.7,
                    packed=rng.random() < 0.5)
    if op == "decode":
        hk, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 2, 4])
        hv = min(32, hk * group)
        seqs = min(_log(rng, 1, 256), 4096 // hv)
        return dict(op=op, seqs=seqs, slots=seqs + rng.randrange(1, 40), pad=rng.randrange(0, seqs // 2 + 1),
                    hk=hk, hv=hv, state=rng.choice(["fp32", "bf16"]), packed=rng.random() < 0.5)
    if op == "norm":
        dim = rng.choice([_log(rng, 16, 16384), 8 * _log(rng, 16, 2048)])
        out, group = rng.choice([("bf16", 0), ("fp8", 0), ("fp8", 128)])
        return dict(op=op, rows=_log(rng, 1, max(1, min(16384, 117440512 // dim))), dim=dim, out=out,
                    group=group, residual=rng.random() < 0.7)
    group = rng.choice([32, 64, 128])
    return dict(op=op, rows=_log(rng, 1, 64), k=group * max(1, _log(rng, 256, 8192) // group),
                n=_log(rng, 64, 12000), group=group, zeros=rng.random() < 0.5)


def _lengths(case):
    """Sequence lengths that add up to the case's tokens; ragged ones span empty to several times the mean."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [t // n + (1 if i < t % n else 0) for i in range(n)]
    w = [((i * 7919 + 31) % 97 / 97.0) ** 2 for i in range(n)]
    total = sum(w) or 1.0
    ls = [int(t * x / total) for x in w]
    ls[-1] += t - sum(ls)
    return ls


def _heads(case, tokens, rnd):
    """q, k, v, a and beta logits: tensors of their own, or columns of one projection's output."""
    hk, hv = case["hk"], case["hv"]
    if case["packed"]:
        cols = (2 * hk + hv) * D + 2 * hv
        p = rnd(tokens, -(-cols // 8) * 8).to(torch.bfloat16)
        at = [0, hk * D, 2 * hk * D, (2 * hk + hv) * D]
        q = p[:, at[0]:at[1]].unflatten(1, (hk, D))
        k = p[:, at[1]:at[2]].unflatten(1, (hk, D))
        v = p[:, at[2]:at[3]].unflatten(1, (hv, D))
        return q, k, v, p[:, at[3]:at[3] + hv], p[:, at[3] + hv:at[3] + 2 * hv]
    return tuple(rnd(*s).to(torch.bfloat16)
                 for s in ((tokens, hk, D), (tokens, hk, D), (tokens, hv, D), (tokens, hv), (tokens, hv)))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uni(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    s = dict(case)
    if case["op"] in ("prefill", "decode"):
        hv = case["hv"]
        tokens = case["tokens"] if case["op"] == "prefill" else case["seqs"]
        s["q"], s["k"], s["v"], s["a"], s["beta"] = _heads(case, tokens, rnd)
        # decay rates 1..16 and time steps 0.001..0.1, as such layers are initialised
        s["A_log"] = (1 + 15 * uni(hv)).log()
        dt = (uni(hv) * math.log(100.0) + math.log(1e-3)).exp()
        s["dt_bias"] = dt + (-(-dt).expm1()).log()
        s["scale"] = D ** -0.5
        s["out"] = torch.zeros(tokens, hv, D, dtype=torch.bfloat16, device=DEV)
    if case["op"] == "prefill":
        n = case["seqs"]
        lens = _lengths(case)
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s["max_len"] = max(lens)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        dt = _STATE[case["state"]]
        s["s0"] = rnd(n, hv, D, D).mul_(0.3).to(dt) if case["initial"] else None
        s["sT"] = torch.empty(n, hv, D, D, dtype=dt, device=DEV)
    elif case["op"] == "decode":
        n = case["seqs"]
        s["pool"] = rnd(case["slots"], hv, D, D).mul_(0.3).to(_STATE[case["state"]])
        slots = torch.randperm(case["slots"], generator=gen, device=DEV)[:n].to(torch.int32)
        if case["pad"]:
            slots[n - case["pad"]:] = -1
        s["slots_of"] = slots
    elif case["op"] == "norm":
        m, dim = case["rows"], case["dim"]
        s["x"] = rnd(m, dim).to(torch.bfloat16)
        s["residual"] = rnd(m, dim).mul_(3).to(torch.bfloat16) if case["residual"] else None
        s["w"] = (1 + 0.1 * rnd(dim)).to(torch.bfloat16)
        fp8 = case["out"] == "fp8"
        s["out_t"] = torch.empty(m, dim, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device=DEV)
        groups = -(-dim // case["group"]) if case["group"] else 1
        s["out_scale"] = torch.empty(m, groups, dtype=torch.float32, device=DEV) if fp8 else None
    else:
        m, k, n, g = case["rows"], case["k"], case["n"], case["group"]
        s["x"] = rnd(m, k).to(torch.bfloat16)
        s["w"] = torch.randint(0, 256, (n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["scales"] = ((0.5 + uni(n, k // g)) * (0.25 / math.sqrt(k))).to(torch.bfloat16)
        s["zeros"] = torch.randint(4, 13, (n, k // g), generator=gen, device=DEV).to(torch.bfloat16) \
            if case["zeros"] else None
        s["y"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    return s


# ---- the plain forms -------------------------------------------------------

def _unit(x):
    x = x.float()
    return x / (x.square().sum(-1, keepdim=True) + EPS).sqrt()


def _gates(s):
    """log decay and beta, [T, Hv] in 32 bits."""
    x = s["a"].float() + s["dt_bias"]
    soft = x.clamp(min=0) + (-x.abs()).exp().log1p()
    return -s["A_log"].exp() * soft, 1 / (1 + (-s["beta"].float()).exp())


def _plain_prefill(s):
    """The chunked form: a triangular inverse of every chunk at once, then the states chunk after chunk."""
    hk, hv, n = s["hk"], s["hv"], s["seqs"]
    nc = -(-s["max_len"] // CHUNK)
    cu = s["cu"].long()
    pos = torch.arange(nc * CHUNK, device=DEV)
    row = cu[:-1, None] + pos
    valid = row < cu[1:, None]
    row = torch.where(valid, row, torch.zeros_like(row))

    def chunks(x):  # [T, H, ...] -> [N, Hv, nc, C, ...], zeros behind a sequence's end
        x = torch.where(valid.view(n, -1, *[1] * (x.dim() - 1)), x[row], torch.zeros((), device=DEV))
        if x.shape[2] != hv:
            x = x.repeat_interleave(hv // x.shape[2], 2)
        return x.transpose(1, 2).unflatten(2, (nc, CHUNK))

    log_a, beta = _gates(s)
    q, k, v = chunks(_unit(s["q"])) * s["scale"], chunks(_unit(s["k"])), chunks(s["v"].float())
    beta = chunks(beta)[..., None]
    g = chunks(log_a).double().cumsum(-1)
    t, j = torch.arange(CHUNK, device=DEV)[:, None], torch.arange(CHUNK, device=DEV)
    decay = torch.where(t >= j, (g[..., :, None] - g[..., None, :]).clamp(max=0).exp().float(), 0.0)
    a = torch.where(t > j, beta * decay * (k @ k.mT), 0.0)
    p = decay * (q @ k.mT)
    inv = torch.eye(CHUNK, device=DEV).expand_as(a).contiguous()
    for i in range(1, CHUNK):  # (I + A)^-1, a row at a time
        inv[..., i, :i] = -(a[..., i, :i, None] * inv[..., :i, :i]).sum(-2)
    grow = g.exp().float()[..., None]
    rest = (g[..., -1:] - g).exp().float()[..., None]
    state = s["s0"].float() if s["s0"] is not None else torch.zeros(n, hv, D, D, device=DEV)
    outs = []
    for c in range(nc):
        kc, qc = k[:, :, c], q[:, :, c]
        u = inv[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - grow[:, :, c] * (kc @ state)))
        outs.append(grow[:, :, c] * (qc @ state) + p[:, :, c] @ u)
        state = grow[:, :, c, -1:] * state + (rest[:, :, c] * kc).mT @ u
    out = torch.cat(outs, 2).transpose(1, 2)
    s["out"][row[valid]] = out[valid].to(torch.bfloat16)
    s["sT"].copy_(state)
    return {"out": s["out"], "state": s["sT"]}


def _plain_decode(s):
    group = s["hv"] // s["hk"]
    log_a, beta = _gates(s)
    q, k = (_unit(s[x]).repeat_interleave(group, 1) for x in ("q", "k"))
    live = s["slots_of"] >= 0
    slot = s["slots_of"].long()[live]
    state = s["pool"][slot].float() * log_a[live].exp()[..., None, None]
    q, k = q[live], k[live]
    u = beta[live][..., None] * (s["v"][live].float() - (k[..., None] * state).sum(-2))
    state = state + k[..., None] * u[..., None, :]
    s["out"][live] = (s["scale"] * (q[..., None] * state).sum(-2)).to(torch.bfloat16)
    s["pool"][slot] = state.to(s["pool"].dtype)
    return {"out": s["out"], "pool": s["pool"]}


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
        s["residual"].copy_(x)
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"].float()
    if s["out"] == "bf16":
        s["out_t"].copy_(y)
        return {"out": s["out_t"], "residual": s["residual"]}
    group = s["group"] or s["dim"]
    groups = -(-s["dim"] // group)
    y = torch.nn.functional.pad(y, (0, groups * group - s["dim"])).unflatten(1, (groups, group))
    c = y.abs().amax(-1) / FP8_MAX
    q = (y / torch.where(c > 0, c, 1.0)[..., None]).flatten(1)[:, :s["dim"]]
    s["out_t"].copy_(q.clamp(-FP8_MAX, FP8_MAX))
    s["out_scale"].copy_(c)
    return {"out": s["out_t"], "scale": s["out_scale"], "residual": s["residual"]}


def _plain_w4(s):
    w = torch.stack((s["w"] & 15, s["w"] >> 4), -1).flatten(1).float().unflatten(1, (-1, s["group"]))
    w = w - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])
    s["y"].copy_(s["x"].float() @ (w * s["scales"].float()[..., None]).flatten(1).T)
    return {"y": s["y"]}


def _own(s):
    import gated_delta_rule_tok_amd as kda
    op = s["op"]
    if op == "prefill":
        if "ws" not in s:  # kept for the calls that follow, as a server keeps it
            s["ws"] = torch.empty(kda.kda_gdr_get_workspace_size(s["tokens"], s["hk"], s["hv"], s["seqs"]),
                                  dtype=torch.uint8, device=DEV)
        kda.kda_gdr_prefill_fwd(s["q"], s["k"], s["v"], s["a"], s["beta"], s["A_log"], s["dt_bias"],
                                s["scale"], s["s0"], s["cu"], s["out"], s["sT"], s["ws"])
        return {"out": s["out"], "state": s["sT"]}
    if op == "decode":
        kda.kda_gdr_decode_step(s["q"], s["k"], s["v"], s["a"], s["beta"], s["A_log"], s["dt_bias"],
                                s["scale"], s["pool"], s["slots_of"], s["out"])
        return {"out": s["out"], "pool": s["pool"]}
    if op == "norm":
        kda.kda_add_rms_norm(s["x"], s["residual"], s["w"], EPS, s["out_t"], s["out_scale"], s["group"])
        if s["out"] == "bf16":
            return {"out": s["out_t"], "residual": s["residual"]}
        return {"out": s["out_t"], "scale": s["out_scale"], "residual": s["residual"]}
    kda.kda_w4_proj(s["x"], s["w"], s["scales"], s["zeros"], s["y"], s["group"])
    return {"y": s["y"]}


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "norm": _plain_norm,
            "w4": _plain_w4}[state["op"]](state)


# ---- the work --------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("prefill", "decode"):
        hk, hv = case["hk"], case["hv"]
        tokens = case["tokens"] if op == "prefill" else case["seqs"] - case["pad"]
        state = D * D * hv * (4 if case["state"] == "fp32" else 2)
        rows = tokens * ((2 * hk + 2 * hv) * D + 2 * hv) * 2
        n = case["seqs"] if op == "prefill" else tokens
        moves = 2 if op == "decode" or case["initial"] else 1
        # per token and value head: the decay, k S, the update and q S
        return {"bytes": rows + moves * n * state, "flops": 7 * D * D * tokens * hv}
    if op == "norm":
        m, dim = case["rows"], case["dim"]
        groups = -(-dim // case["group"]) if case["group"] else 1
        per = 2 + (4 if case["residual"] else 0) + (1 if case["out"] == "fp8" else 2)
        scales = 4 * m * groups if case["out"] == "fp8" else 0
        return {"bytes": m * dim * per + 2 * dim + scales, "flops": 6 * m * dim}
    m, k, n, g = case["rows"], case["k"], case["n"], case["group"]
    return {"bytes": n * k // 2 + n * (k // g) * (4 if case["zeros"] else 2) + 2 * m * (k + n),
            "flops": 2 * m * n * k}


# ---- 64 bits, from the definitions ------------------------------------------

def _serial(q, k, v, a, beta_logits, A_log, dt_bias, scale, state):
    """One token of the recurrence for a batch of sequences: [B, H, D] rows in fp64, state [B, Hv, D, D]."""
    group = v.shape[1] // q.shape[1]

    def norm(x):
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
        return x[:, :, None].expand(-1, -1, group, -1).reshape(v.shape[0], v.shape[1], D)

    q, k = norm(q), norm(k)
    decay = torch.exp(-torch.exp(A_log) * torch.logaddexp(a + dt_bias, torch.zeros_like(a)))
    beta = torch.sigmoid(beta_logits)
    state = state * decay[:, :, None, None]
    guess = torch.matmul(k[:, :, None, :], state)[:, :, 0]
    state = state + (beta[:, :, None] * k)[..., None] * (v - guess)[:, :, None, :]
    return scale * torch.matmul(q[:, :, None, :], state)[:, :, 0], state


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prefill", "decode"):
        rows = [s[x].double() for x in ("q", "k", "v", "a", "beta")]
        A_log, dt_bias = s["A_log"].double(), s["dt_bias"].double()
        out = s["out"].double()
        if op == "decode":
            pool = s["pool"].double()
            live = [i for i, x in enumerate(s["slots_of"].tolist()) if x >= 0]
            slot = s["slots_of"].long()[live]
            out[live], pool[slot] = _serial(*(x[live] for x in rows), A_log, dt_bias, s["scale"], pool[slot])
            return {"out": out, "pool": pool}
        cu = s["cu"].tolist()
        n, hv = case["seqs"], case["hv"]
        state = s["s0"].double() if case["initial"] else \
            torch.zeros(n, hv, D, D, dtype=torch.float64, device=DEV)
        # the longest sequences first, so that those still running are the first ones
        order = sorted(range(n), key=lambda i: cu[i] - cu[i + 1])
        state = state[order]
        lens = [cu[i + 1] - cu[i] for i in order]
        first = torch.tensor([cu[i] for i in order], device=DEV)
        left = n
        for t in range(s["max_len"]):
            while left and lens[left - 1] <= t:
                left -= 1
            at = first[:left] + t
            out[at], state[:left] = _serial(*(x[at] for x in rows), A_log, dt_bias, s["scale"], state[:left])
        back = torch.empty_like(state)
        back[order] = state
        return {"out": out, "state": back}
    if op == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * s["w"].double()
        res = None if s["residual"] is None else x
        if case["out"] == "bf16":
            return {"out": y, "residual": res}
        width = case["group"] or case["dim"]
        parts = y.split(width, 1)
        c = torch.stack([p.abs().max(1).values / FP8_MAX for p in parts], 1)
        z = torch.cat([p / c[:, i:i + 1].clamp(min=1e-300) for i, p in enumerate(parts)], 1)
        # the nearest e4m3 value, ties to the even one: 3 bits behind the leading one, 2^-9 the least step
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        return {"out": torch.round(z / step) * step, "scale": c, "residual": res}
    k, g = case["k"], case["group"]
    w = torch.empty(case["n"], k, dtype=torch.float64, device=DEV)
    w[:, 0::2] = (s["w"] % 16).double()
    w[:, 1::2] = (s["w"] // 16).double()
    at = torch.arange(k, device=DEV) // g
    w -= 8.0 if s["zeros"] is None else s["zeros"].double()[:, at]
    w *= s["scales"].double()[:, at]
    return {"y": torch.matmul(s["x"].double(), w.T)}
