"""GPU parity of the operators of include/kda_mx4.h against plain 64-bit forms
of their definitions.

Quantisation and its inverse are exact arithmetic: bits are compared.

Products (u = 2^-24, an fp32 rounding).  Products are exact and a sum of n terms
in fp32, in any order, is off by at most n u times the sum of their magnitudes;
bf16's rounding by half a step, 2^-8 of the value.  Roundings are independent, so
the relative root-mean-square error is far smaller: 2^-8 / sqrt(3) for values
spread over a step of the smallest relative size, 2.26e-3, and for sums that do
not cancel 2e-5 at most beside it.

The layer: G x and U x as above, with errors dG and dU; silu's slope is at most
1.1, so h = g silu(G) U is off by |g| (1.1 |U| dG + |silu| dU) + 2^-16 |h| (two
bf16 pieces hold 16 bits, and silu's few roundings 2^-20), and out by the sum over
inter and experts of |W_down| dh, the fp32 sum of those terms and bf16's half step.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RMS = 2.0 ** -8 / math.sqrt(3) + 2e-5


def _kda():
    import gated_delta_rule_tok_amd as kda
    return kda


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(codes, scales):
    """fp64 values, NaN where the scale is."""
    import torch
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                       device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
    return lut[c] * s.repeat_interleave(32, -1)


def _quant(x):
    """codes, scales of bf16 x by the definition, in fp64."""
    import torch
    b = x.double().unflatten(-1, (-1, 32))
    m = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    m = torch.where(bad, 1.0, m)
    # |x| = f 2^e with f in [1/2, 1): floor(log2 m) = e - 1
    s = torch.where(m > 0, torch.frexp(m).exponent - 1 - 2 + 127, 0).clamp(min=0)
    a = (b.abs() * torch.exp2(127.0 - s.double())[..., None]).clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (a / step).round() * step
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, v in enumerate([0, .5, 1, 1.5, 2, 3, 4, 6]):
        code[a == v] = i
    code += 8 * torch.signbit(b).to(torch.uint8)
    code[bad] = 0
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.where(bad, 255, s).to(torch.uint8)


def _run_quant(x, stream=None):
    import torch
    m, k = x.shape
    c = torch.full((m, k // 2), 0x5a, dtype=torch.uint8, device="cuda")
    s = torch.full((m, k // 32), 0x5a, dtype=torch.uint8, device="cuda")
    _kda().kda_mx4_quant(x, c, s, stream=stream)
    return c, s


def _weights(rows, k, seed, spread=1):
    """Codes of every kind with scales that give rows of about unit norm."""
    import torch
    g = _gen(seed)
    c = torch.randint(0, 256, (*rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    mid = 127 - round(math.log2(3 * math.sqrt(k)))
    s = torch.randint(mid - spread, mid + spread + 1, (*rows, k // 32), generator=g, device="cuda",
                      dtype=torch.uint8)
    return c, s


# ---- quantisation -----------------------------------------------------------

@pytest.mark.parametrize("m,k,pad", [(1, 32, 0), (1, 7168, 0), (3, 96, 0), (5, 160, 8), (777, 2080, 72),
                                     (1000, 64, 0), (37, 4128, 24), (2, 131072, 0)])
def test_quant(m, k, pad):
    import torch
    x = (torch.randn(m, k + pad, generator=_gen(m + k), device="cuda") *
         torch.randn(m, 1, generator=_gen(m), device="cuda").mul(8).exp()).bfloat16()[:, pad:]
    c, s = _run_quant(x)
    rc, rs = _quant(x)
    assert torch.equal(s, rs) and torch.equal(c, rc)
    v = torch.full((m, k + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_dequant(c, s, v[:, pad:])
    assert torch.equal(v[:, pad:].double(), _values(c, s)) and (v[:, :pad] == 7).all()


def test_quant_of_every_bf16():
    """Every value beside a zero, beside its likes and in mixed company."""
    import torch
    every = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    alone = torch.zeros(65536, 32, dtype=torch.bfloat16, device="cuda")
    alone[:, 5] = every
    perm = torch.randperm(65536, generator=_gen(1), device="cuda")
    near = every.view(-1, 32)
    finite = every[torch.isfinite(every)]
    order = finite.abs().float().sort().indices
    close = finite[order][:len(finite) // 512 * 512].view(-1, 512)  # 512 adjacent magnitudes, shuffled
    close = close[:, torch.randperm(512, generator=_gen(2), device="cuda")]
    for x in (alone, every[perm].view(-1, 64), near, close.reshape(-1, 32)):
        x = x.contiguous()
        c, s = _run_quant(x)
        rc, rs = _quant(x)
        assert torch.equal(s, rs) and torch.equal(c, rc)


def test_quant_of_what_is_not_finite():
    import torch
    x = torch.randn(4, 128, generator=_gen(3), device="cuda").bfloat16()
    clean = _run_quant(x)
    x[1, 40], x[2, 100], x[3, 3] = math.nan, math.inf, -math.inf
    c, s = _run_quant(x)
    hit = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[2, 3] = hit[3, 0] = True
    assert (s[hit] == 255).all() and (c.view(4, 4, 16)[hit] == 0).all()
    assert torch.equal(s[~hit], clean[1][~hit])
    assert torch.equal(c.view(4, 4, 16)[~hit], clean[0].view(4, 4, 16)[~hit])
    v = torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_dequant(c, s, v)
    assert torch.equal(v.view(4, 4, 32).isnan().all(-1), hit)


def test_dequant_of_every_code_and_scale():
    import torch
    s = torch.arange(256, device="cuda").to(torch.uint8)[:, None].contiguous()
    c = torch.arange(16, device="cuda").to(torch.uint8).repeat(256, 1)
    c = (c | (15 - c) << 4).contiguous()
    v = torch.empty(256, 32, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_dequant(c, s, v)
    ref = _values(c, s).float().bfloat16()  # 4 and 6 times 2^127: infinite in fp32 too
    assert torch.equal(v.view(torch.int16)[:255], ref.view(torch.int16)[:255]) and v[255].isnan().all()


# ---- products ---------------------------------------------------------------

def _check_product(x, w, ws, y, label):
    """x: fp64 values."""
    import torch
    wd = _values(w, ws)
    ref = x @ wd.T
    bound = 2.0 ** -8 * ref.abs() + x.shape[1] * U * (x.abs() @ wd.abs().T)
    err = (y.double() - ref).abs()
    rel = (err.norm() / ref.norm()).item() if ref.norm() else 0.0
    print(f"[parity] {label}: rms {rel:.3g}", flush=True)
    assert (err <= bound).all() and rel <= RMS, label


FEW = [(1, 32, 1), (1, 7168, 1536), (2, 96, 17), (3, 160, 33), (4, 2080, 100), (5, 544, 31), (15, 192, 100),
       (16, 448, 70), (17, 1024, 16), (31, 1152, 15), (33, 4128, 70), (64, 2048, 145), (64, 16384, 3),
       (50, 512, 4200), (16, 7168, 4300), (1, 131072, 5)]


@pytest.mark.parametrize("m,k,n", FEW)
def test_proj_of_bf16(m, k, n):
    import torch
    x = torch.randn(m, k, generator=_gen(m + n), device="cuda").bfloat16()
    w, ws = _weights((n,), k, n)
    y = torch.full((m, n), math.nan, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, None, w, ws, y)
    _check_product(x.double(), w, ws, y, f"bf16 {m}x{k}x{n}")
    y2 = torch.empty_like(y)
    _kda().kda_mx4_proj(x, None, w, ws, y2)
    assert torch.equal(y, y2)


MANY = [(65, 32, 1), (100, 96, 40), (128, 256, 128), (129, 288, 257), (200, 2080, 130), (256, 512, 256),
        (300, 4128, 2050), (513, 160, 700), (1000, 1024, 1030), (2049, 544, 64), (257, 7168, 3000), (3000, 64, 20)]


@pytest.mark.parametrize("m,k,n", FEW + MANY)
def test_proj_of_codes(m, k, n):
    import torch
    x, xs = _weights((m,), k, m + k, spread=3)
    w, ws = _weights((n,), k, n)
    y = torch.full((m, n), math.nan, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, xs, w, ws, y)
    _check_product(_values(x, xs), w, ws, y, f"codes {m}x{k}x{n}")
    y2 = torch.empty_like(y)
    _kda().kda_mx4_proj(x, xs, w, ws, y2)
    assert torch.equal(y, y2)


# tiles through LDS: one and several stages of 128, the last in part, scales of 512 in part,
# rows and columns of tiles in part, more tiles than compute units
TILES = [(1024, 32, 1030), (1100, 96, 1000), (1024, 128, 1024), (1025, 160, 1030), (2000, 256, 600), (1030, 416, 1024),
         (1024, 480, 1030), (1024, 512, 1024), (1030, 640, 1100), (129, 896, 8200), (8200, 1152, 130),
         (1024, 2080, 1100), (4500, 544, 4400), (4300, 1024, 4400), (70, 2048, 15000), (5000, 64, 5000),
         (33, 160, 8192), (50, 2048, 8300), (64, 544, 9000), (700, 4128, 800), (300, 512, 2050), (2000, 1056, 1000)]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("m,k,n", TILES)
def test_proj_in_tiles(m, k, n, shift):
    """shift: the scales begin at an odd address."""
    import torch
    x, xs = _weights((m,), k, m + k, spread=3)
    w, ws = _weights((n,), k, n)
    if shift:
        def moved(t):
            flat = torch.full((t.numel() + 1,), 0xAA, dtype=torch.uint8, device="cuda")
            flat[1:] = t.flatten()
            return flat[1:].view(t.shape)
        xs, ws = moved(xs), moved(ws)
    y = torch.full((m + 1, n + 3), 3.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, xs, w, ws, y[:m, :n])
    _check_product(_values(x, xs), w, ws, y[:m, :n], f"tiles {m}x{k}x{n}")
    assert (y[m:] == 3).all() and (y[:, n:] == 3).all()
    y2 = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, xs, w, ws, y2)
    assert torch.equal(y[:m, :n], y2)


@pytest.mark.parametrize("xshift,wshift", [(0, 1), (2, 3), (3, 0)])
@pytest.mark.parametrize("m,k,n", [(200, 928, 4100), (130, 960, 5000), (1000, 992, 1100), (2100, 992, 2060),
                                   (300, 1024, 2050), (90, 1056, 8200)])
def test_proj_in_tiles_between_nans(m, k, n, xshift, wshift):
    """Scales at any byte, with NaN scales right before and behind them."""
    import torch
    x, xs = _weights((m,), k, m + k, spread=3)
    w, ws = _weights((n,), k, n)

    def moved(t, shift):
        flat = torch.full((t.numel() + 32,), 0xFF, dtype=torch.uint8, device="cuda")
        flat[shift:shift + t.numel()] = t.flatten()
        return flat[shift:shift + t.numel()].view(t.shape)
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, moved(xs, xshift), w, moved(ws, wshift), y)
    _check_product(_values(x, xs), w, ws, y, f"tiles {m}x{k}x{n}, scales at {xshift}, {wshift}")


def test_proj_in_tiles_rows_do_not_mix():
    """NaN scales of one token and of one weight row stay in their row and column, also in
    the last blocks of k."""
    import torch
    m, k, n = 1100, 544, 1000
    x, xs = _weights((m,), k, 20)
    w, ws = _weights((n,), k, 21)
    y, z = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _kda().kda_mx4_proj(x, xs, w, ws, y)
    xs[1099, 16] = 255
    ws[500, 0] = 255
    _kda().kda_mx4_proj(x, xs, w, ws, z)
    hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    hit[1099] = hit[:, 500] = True
    assert z[hit].isnan().all() and torch.equal(z[~hit], y[~hit])


def test_operands_of_more_than_4_gib():
    """Rows whose offsets pass 32 bits."""
    import torch
    k, n = 65536, 140000
    w = torch.randint(0, 256, (n, k // 2), generator=_gen(22), device="cuda", dtype=torch.uint8)
    ws = torch.randint(100, 140, (n, k // 32), generator=_gen(23), device="cuda", dtype=torch.uint8)
    assert w.numel() > 1 << 32
    y = torch.full((3, n), math.nan, dtype=torch.bfloat16, device="cuda")
    x, xs = _weights((3,), k, 24)
    at = torch.cat((torch.arange(20), torch.arange(n - 40, n))).cuda()
    _kda().kda_mx4_proj(x, xs, w, ws, y)
    _check_product(_values(x, xs), w[at], ws[at], y[:, at], "codes, large w")
    b = torch.randn(3, k, generator=_gen(25), device="cuda").bfloat16()
    _kda().kda_mx4_proj(b, None, w, ws, y)
    _check_product(b.double(), w[at], ws[at], y[:, at], "bf16, large w")
    # as the rows of x in tiles, against few rows of w
    z = torch.full((n, 70), math.nan, dtype=torch.bfloat16, device="cuda")
    few, few_s = _weights((70,), k, 26)
    _kda().kda_mx4_proj(w, ws, few, few_s, z)
    _check_product(_values(w[at], ws[at]), few, few_s, z[at], "tiles, large x")
    del y, z
    v = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_dequant(w, ws, v)
    assert torch.equal(v[at].double(), _values(w[at], ws[at]))
    c, s = _run_quant(v)
    rc, rs = _quant(v[at])
    assert torch.equal(c[at], rc) and torch.equal(s[at], rs)


@pytest.mark.parametrize("m", [3, 20, 150])
def test_proj_of_strided_rows(m):
    import torch
    n = 50
    w, ws = _weights((n,), 256, 4)
    y = torch.full((m, 61), 3.0, dtype=torch.bfloat16, device="cuda")
    if m <= 64:
        x = torch.randn(m, 256 + 24, generator=_gen(5), device="cuda").bfloat16()[:, 24:]
        _kda().kda_mx4_proj(x, None, w, ws, y[:, 7:57])
        _check_product(x.double(), w, ws, y[:, 7:57], "strided")
        assert (y[:, :7] == 3.0).all() and (y[:, 57:] == 3.0).all()
    x, xs = _weights((m,), 256, 6)
    _kda().kda_mx4_proj(x, xs, w, ws, y[:, 3:53])
    _check_product(_values(x, xs), w, ws, y[:, 3:53], "strided codes")
    assert (y[:, :3] == 3.0).all() and (y[:, 57:] == 3.0).all()


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_proj_rows_do_not_mix(m):
    """A token's NaN stays in its row, a weight row's in its column, and a token's
    result does not depend on the values of the tokens beside it."""
    import torch
    kda, n, k = _kda(), 64, 512
    w, ws = _weights((n,), k, 7)
    x, xs = _weights((m,), k, 8)
    y, z = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i = m // 2
    others = [r for r in range(m) if r != i]
    kda.kda_mx4_proj(x, xs, w, ws, y)
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[i, 5] = 255
    ws2[9, 3] = 255
    kda.kda_mx4_proj(x, xs2, w, ws2, z)
    cols = [c for c in range(n) if c != 9]
    assert z[i].isnan().all() and z[:, 9].isnan().all() and torch.equal(z[others][:, cols], y[others][:, cols])
    x2, xs2 = _weights((m,), k, 9)
    x2[i], xs2[i] = x[i], xs[i]
    kda.kda_mx4_proj(x2, xs2, w, ws, z)
    assert torch.equal(z[i], y[i])
    if m > 64:
        return
    b = torch.randn(m, k, generator=_gen(10), device="cuda").bfloat16()
    kda.kda_mx4_proj(b, None, w, ws, y)
    b2 = torch.randn(m, k, generator=_gen(11), device="cuda").bfloat16()
    b2[i] = b[i]
    b2[others, 77] = math.nan
    kda.kda_mx4_proj(b2, None, w, ws2, z)
    assert torch.equal(z[i][cols], y[i][cols]) and z[others].isnan().all() and z[:, 9].isnan().all()


@pytest.mark.parametrize("m,k,n", [(1, 512, 100), (16, 160, 33), (130, 288, 140)])
@pytest.mark.parametrize("size", [-100, -60, 60, 100])
def test_proj_of_any_size(m, k, n, size):
    """Scales far from one on one side, undone on the other."""
    import torch
    x, xs = _weights((m,), k, 12)
    w, ws = _weights((n,), k, 13)
    y = torch.full((m, n), math.nan, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, (xs.int() + size).to(torch.uint8), w, (ws.int() - size).to(torch.uint8), y)
    _check_product(_values(x, xs), w, ws, y, f"2^{size}")
    if m <= 64:
        b = torch.randn(m, k, generator=_gen(14), device="cuda").bfloat16()
        _kda().kda_mx4_proj((b.double() * 2.0 ** size).bfloat16(), None, w, (ws.int() - size).to(torch.uint8), y)
        _check_product(b.double(), w, ws, y, f"bf16 2^{size}")


@pytest.mark.parametrize("m", [1, 16, 40])
def test_proj_of_the_least_weights(m):
    """Scales of 2^-127 and a little above, whose values bf16 holds as subnormals."""
    import torch
    k, n = 256, 48
    w, _ = _weights((n,), k, 16)
    ws = torch.randint(0, 4, (n, k // 32), generator=_gen(17), device="cuda", dtype=torch.uint8)
    x = torch.randn(m, k, generator=_gen(18), device="cuda").mul(2.0 ** 100).bfloat16()
    y = torch.full((m, n), math.nan, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, None, w, ws, y)
    _check_product(x.double(), w, ws, y, "least weights")
    c, s = _run_quant(x)
    _kda().kda_mx4_proj(c, s, w, ws, y)
    _check_product(_values(c, s), w, ws, y, "least weights, codes")


def test_proj_of_no_rows():
    import torch
    w, ws = _weights((5,), 64, 15)
    for x in (torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), None):
        y = torch.empty(0, 5, dtype=torch.bfloat16, device="cuda")
        if x is not None:
            _kda().kda_mx4_proj(x, None, w, ws, y)
        else:
            _kda().kda_mx4_proj(w[:0], ws[:0], w, ws, y)
    torch.cuda.synchronize()


# ---- the mixture-of-experts layer --------------------------------------------

class Moe:
    def __init__(self, m, k, inter, experts, top, shared=0, bias=False, seed=0, pad=0):
        import torch
        g = _gen(seed)

        def rnd(*s):
            return torch.randn(*s, generator=g, device="cuda")

        self.m, self.k, self.inter, self.experts, self.top, self.shared = m, k, inter, experts, top, shared
        self.x = rnd(m, k + pad).bfloat16()[:, pad:]
        self.router = (rnd(experts, k) / math.sqrt(k)).bfloat16()
        self.bias = rnd(experts) * 0.1 if bias else None
        self.w_up, self.s_up = _weights((experts + shared, 2 * inter), k, seed + 1)
        self.w_down, self.s_down = _weights((experts + shared, k), inter, seed + 2)
        self.out = torch.full((m, k + pad), 9.0, dtype=torch.bfloat16, device="cuda")[:, pad:]
        self.ids = torch.full((m, top), -7, dtype=torch.int32, device="cuda")
        self.gates = torch.full((m, top), math.nan, device="cuda")
        self.ws = torch.full((_kda().kda_mx4_moe_workspace_size(m, k, inter, experts, shared, top),), 0xFF,
                             dtype=torch.uint8, device="cuda")
        self.opts = dict(scoring="sigmoid", renormalise=True, route_scale=2.5)

    def run(self, **over):
        _kda().kda_mx4_moe(self.x, self.router, self.bias, self.w_up, self.s_up, self.w_down, self.s_down, self.out,
                           self.ids, self.gates, self.ws, **{**self.opts, **over})
        return self

    def choice(self):
        """ids, gates (fp64) by the formula."""
        import torch
        logits = self.x.double() @ self.router.double().T
        p = torch.sigmoid(logits) if self.opts["scoring"] == "sigmoid" else torch.softmax(logits, 1)
        key = p if self.bias is None else p + self.bias.double()
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :self.top]
        g = p.gather(1, ids)
        if self.opts["renormalise"]:
            g = g / g.sum(1, keepdim=True)
        return ids, g * self.opts["route_scale"]

    def check(self, label, live=None):
        import torch
        live = list(range(self.m)) if live is None else live
        ids, gates = self.choice()
        assert torch.equal(self.ids[live].long(), ids[live]), label
        assert ((self.gates[live].double() - gates[live]).abs() <= (U + 1e-12) * gates[live].abs()).all(), label
        ref = torch.zeros(self.m, self.k, dtype=torch.float64, device="cuda")
        off = torch.zeros_like(ref)
        hits = torch.zeros(self.m, self.experts + self.shared, dtype=torch.float64, device="cuda")
        hits.scatter_(1, ids, self.gates.double())
        hits[:, self.experts:] = 1
        n = self.inter * (self.top + self.shared)
        for e in range(self.experts + self.shared):
            at = [t for t in live if e >= self.experts or (ids[t] == e).any()]
            if not at:
                continue
            w, x = _values(self.w_up[e], self.s_up[e]), self.x[at].double()
            both, mag = x @ w.T, self.k * U * (x.abs() @ w.abs().T)
            a, u = both[:, :self.inter], both[:, self.inter:]
            silu = a * torch.sigmoid(a)
            g = hits[at, e][:, None]
            h = g * silu * u
            dh = g.abs() * (1.1 * u.abs() * mag[:, :self.inter] + silu.abs() * mag[:, self.inter:]) \
                + 2.0 ** -16 * h.abs()
            d = _values(self.w_down[e], self.s_down[e])
            ref[at] += h @ d.T
            off[at] += dh @ d.abs().T + n * U * (h.abs() @ d.abs().T)
        err = (self.out.double() - ref).abs()[live]
        rel = (err.norm() / ref[live].norm()).item()
        print(f"[parity] {label}: rms {rel:.3g}", flush=True)
        assert (err <= 2.0 ** -8 * ref.abs()[live] + off[live]).all() and rel <= RMS, label


MOE = [
    # m, k, inter, experts, top, shared, bias
    (1, 32, 32, 1, 1, 0, False), (1, 7168, 512, 64, 8, 1, True), (2, 96, 64, 5, 2, 0, True),
    (3, 160, 96, 17, 3, 2, False), (4, 2080, 160, 40, 4, 0, True), (7, 512, 544, 33, 6, 1, False),
    (16, 256, 128, 8, 2, 0, False), (17, 288, 64, 4, 4, 1, True), (33, 128, 96, 256, 8, 1, True),
    (64, 512, 256, 64, 8, 1, False), (64, 96, 32, 2, 1, 0, True), (64, 64, 64, 1000, 32, 16, False),
    (21, 2080, 1056, 40, 4, 0, False), (64, 1056, 352, 3, 2, 2, False), (1, 64, 64, 1024, 32, 0, True),
    (64, 288, 160, 300, 5, 1, True), (48, 4128, 32, 20, 3, 0, False), (5, 32, 2080, 9, 9, 0, True),
    (30, 96, 4096, 6, 1, 16, False), (64, 512, 64, 600, 9, 0, False),
]


@pytest.mark.parametrize("scoring,renorm", [("sigmoid", True), ("softmax", False)])
@pytest.mark.parametrize("m,k,inter,experts,top,shared,bias", MOE)
def test_moe(m, k, inter, experts, top, shared, bias, scoring, renorm):
    import torch
    p = Moe(m, k, inter, experts, top, shared, bias, seed=m + k)
    p.opts.update(scoring=scoring, renormalise=renorm)
    p.run().check(f"moe {m}x{k}x{inter} of {experts}")
    first = [t.clone() for t in (p.out, p.ids, p.gates)]
    p.ws.fill_(0x7f)
    p.run()
    assert all(torch.equal(a, b) for a, b in zip(first, (p.out, p.ids, p.gates)))


def test_moe_of_strided_rows_and_softmax_renormalised():
    p = Moe(9, 512, 128, 20, 3, 1, True, seed=30, pad=40)
    p.opts.update(scoring="softmax", renormalise=True, route_scale=1.0)
    base = p.out._base
    p.run().check("strided")
    assert (base[:, :40] == 9).all()


@pytest.mark.parametrize("m,pads", [(1, [0]), (6, [1, 4, 5]), (40, list(range(7, 40))), (64, list(range(0, 64, 2)))])
def test_moe_of_padding_rows(m, pads):
    import torch
    p = Moe(m, 256, 96, 30, 3, 1, True, seed=31)
    idx = torch.arange(m, dtype=torch.int32, device="cuda")
    idx[pads] = -1
    p.x[pads] = math.nan
    p.run(state_indices=idx)
    live = [i for i in range(m) if i not in pads]
    assert (p.out[pads] == 9).all() and (p.ids[pads] == -1).all() and (p.gates[pads] == 0).all()
    if live:
        p.check("padding", live)


def test_moe_of_one_expert_for_all():
    """Every token to the same experts; and to experts of its own."""
    import torch
    for m in (4, 17, 64):
        p = Moe(m, 128, 64, 64, 1, 0, False, seed=38)
        p.x[:] = p.x[0]
        p.run().check("all to one")
        p = Moe(m, 128, 64, 64, 1, 0, True, seed=39)
        p.router.zero_()
        p.router[:, :64] = torch.eye(64, device="cuda").bfloat16()
        p.x.zero_()
        p.x[torch.arange(m), torch.arange(m)] = 9
        p.x[:, 64:] = torch.randn(m, 64, generator=_gen(40), device="cuda").bfloat16()
        p.run().check("each its own")
        assert torch.equal(p.ids[:, 0].cpu(), torch.arange(m, dtype=torch.int32))


def test_moe_of_equal_scores():
    """Equal logits: the lowest indices; a bias decides, and does not enter the gates."""
    import torch
    p = Moe(3, 64, 32, 12, 4, 0, True, seed=32)
    p.router[:] = p.router[0]
    p.bias.zero_()
    p.run()
    assert torch.equal(p.ids, torch.arange(4, dtype=torch.int32, device="cuda").repeat(3, 1))
    p.bias[7] = 1e-6
    p.bias[3] = -1e-6
    p.run().check("equal scores")
    assert torch.equal(p.ids[0].cpu(), torch.tensor([7, 0, 1, 2], dtype=torch.int32))


def test_moe_of_saturated_scores():
    """Scores that are 1 to fp64's last bit are told apart by their logits where no bias is added."""
    import torch
    p = Moe(4, 64, 32, 16, 3, 0, False, seed=33)
    p.x[:] = p.x.abs()
    p.router[:] = (torch.arange(16, device="cuda")[:, None] + 40.0).bfloat16()
    p.run()
    assert torch.equal(p.ids[0].cpu(), torch.tensor([15, 14, 13], dtype=torch.int32))


def test_moe_of_what_is_not_finite():
    """A NaN in x, in a scale of an expert, in the router: in the rows that read it, and the ids stay valid."""
    import torch
    p = Moe(20, 256, 64, 16, 2, 0, False, seed=34)
    p.run()
    clean, ids = p.out.clone(), p.ids.clone()
    p.x[3, 17] = math.nan
    bad = int(ids[5, 0])
    p.s_up[bad, 3, 1] = 255
    p.run()
    hit = (ids == bad).any(1)
    hit[3] = True
    assert p.out[hit].isnan().all() and torch.equal(p.out[~hit], clean[~hit])
    assert torch.equal(p.ids[~hit], ids[~hit]) and ((p.ids >= 0) & (p.ids < 16)).all()
    p.router[4] = math.nan
    p.run()
    rest = ~hit & (ids != 4).all(1)
    assert (p.ids[~hit] != 4).all() and torch.equal(p.out[rest], clean[rest])


def test_moe_rows_do_not_depend_on_the_tokens_beside():
    import torch
    p = Moe(30, 1024, 128, 12, 3, 1, False, seed=35)
    p.run().check("first tokens")
    ids, gates = p.ids[11].clone(), p.gates[11].clone()
    x = p.x[11].clone()
    p.x[:] = torch.randn(30, 1024, generator=_gen(36), device="cuda").bfloat16()
    p.x[11] = x
    p.run().check("other tokens")
    # the choice and its gates to the bit (sums over experts may be in another order)
    assert torch.equal(p.ids[11], ids) and torch.equal(p.gates[11], gates)


def test_moe_of_no_tokens():
    import torch
    p = Moe(0, 64, 32, 4, 2, seed=37)
    ws = torch.empty(max(256, p.ws.numel()), dtype=torch.uint8, device="cuda")
    p.ws = ws
    p.run()
    torch.cuda.synchronize()


# ---- together ---------------------------------------------------------------

class Half:
    """The second half of a layer's step: residual + norm -> experts -> residual +
    norm -> quantised -> product with 4-bit weights (the next layer's projection)."""

    def __init__(self, m, k=512, n=200, seed=40):
        import torch
        self.moe = Moe(m, k, 128, 16, 4, 1, True, seed=seed)
        g = _gen(seed + 5)
        self.x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        self.r = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        self.nw = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).bfloat16()
        self.h = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
        self.c = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda")
        self.s = torch.zeros(m, k // 32, dtype=torch.uint8, device="cuda")
        self.w, self.ws = _weights((n,), k, seed + 6)
        self.y = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        self.z = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")

    def step(self):
        kda = _kda()
        kda.kda_add_rms_norm(self.x, self.r, self.nw, 1e-6, self.moe.x)
        self.moe.run()
        kda.kda_add_rms_norm(self.moe.out, self.r, self.nw, 1e-6, self.h)
        kda.kda_mx4_quant(self.h, self.c, self.s)
        kda.kda_mx4_proj(self.c, self.s, self.w, self.ws, self.y)
        kda.kda_mx4_proj(self.h, None, self.w, self.ws, self.z)

    def results(self):
        return [t.clone() for t in (self.r, self.moe.x, self.moe.out, self.moe.ids, self.moe.gates, self.h, self.c,
                                    self.s, self.y, self.z)]


@pytest.mark.parametrize("m", [1, 6, 40])
def test_a_layers_second_half(m):
    """Each operator on what the one before it wrote; then captured and replayed,
    each replay equal to the eager step."""
    import torch
    p = Half(m)
    r0 = p.r.clone()
    p.step()
    p.moe.check("experts")
    rc, rs = _quant(p.h)
    assert torch.equal(p.c, rc) and torch.equal(p.s, rs)
    _check_product(_values(p.c, p.s), p.w, p.ws, p.y, "quantised product")
    _check_product(p.h.double(), p.w, p.ws, p.z, "bf16 product")
    eager = p.results()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        p.step()
    torch.cuda.synchronize()
    other = Half(m, seed=60)
    for i in range(3):
        p.r.copy_(r0)
        for t in (p.moe.out, p.moe.ids, p.moe.gates, p.h, p.c, p.s, p.y, p.z):
            t.zero_()
        p.moe.ws.fill_(0xFF)
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        for a, b in zip(eager, p.results()):
            assert torch.equal(a, b), f"replay {i}"


def test_two_calls_at_once():
    """On two streams, with workspaces of their own."""
    import torch
    ps = [Moe(16, 1024, 256, 32, 4, 1, True, seed=70 + i) for i in range(2)]
    refs = [[t.clone() for t in (p.run().out, p.ids, p.gates)] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for p in ps:
            p.out.zero_()
            p.ids.zero_()
        torch.cuda.synchronize()
        for p, s in zip(ps, streams):
            p.run(stream=s)
        torch.cuda.synchronize()
        for p, ref in zip(ps, refs):
            assert all(torch.equal(a, b) for a, b in zip(ref, (p.out, p.ids, p.gates)))
