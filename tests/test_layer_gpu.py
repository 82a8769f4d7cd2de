"""GPU parity of the operators of include/kda_layer.h against plain 64-bit
forms of their definitions.

Bounds (u = 2^-24, an fp32 rounding; a bf16 rounding is off by at most half a
step, 2^-8 of the value, an e4m3 one by 2^-4 or half of the least step, 2^-10).

Delta rule.  Everything is fp32 sums of at most 128 + 64 terms, four of them
nested per chunk (k S, T R, P U and the update), with exact factors k and q and
factors S, R, U, T cut to two fp16 pieces (fp32 state: 2^-22 of the value) or
one (bf16 state: 2^-11).  A sum of n terms is off by at most n u times the sum
of the terms' magnitudes, which for the unit vectors k~, q~ is at most the norm
M of the other factor's column (Cauchy); a cut factor adds its cut, two per
product, eight in all.  The state's map is a contraction, so a chunk's error is
passed on undiminished at most:
    |dS| <= chunks * (4 * 192 u + 8 * cut) * M,
    |do| <= scale * (that + 3 * 2^-11 M)   (out takes one piece of S, U and P),
    M = largest column norm of S_t over the run, plus the largest |v|,
before the rounding of the stored value.  The decays are off by a few u each,
far inside the 192.  The serial form has no cut and one token per "chunk" with
sums of 128.  Roundings are independent of each other, so the relative
root-mean-square error is far smaller: for bf16 at most 2^-8 / sqrt(3) for the
stored value and sqrt(8) 2^-11 / sqrt(3) for the cuts, together 2.4e-3; for an
fp32 state sqrt(192) 4 u / sqrt(3) and sqrt(8) 2^-22 / sqrt(3), together 2.3e-6,
where the state is of the size of M.

Norm.  The sum of squares is off by dim u, its root by half of that, and y by
four roundings more; products with 4-bit weights: see _w4_check.
"""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

D = 128
U = 2.0 ** -24


def _kda():
    import gated_delta_rule_tok_amd as kda
    return kda


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


class Gdr:
    """Inputs of one call; packed: q, k, v, a, beta as columns of one matrix."""

    def __init__(self, T, hk, hv, seed, packed=False, correlated=False):
        import torch
        g = _gen(seed)

        def rnd(*s):
            return torch.randn(*s, generator=g, device="cuda")

        cols = (2 * hk + hv) * D + 2 * hv
        p = rnd(T, -(-cols // 8) * 8)
        if correlated:  # keys of a sequence close to one direction: a badly conditioned chunk
            p[:, hk * D:2 * hk * D] += 4 * rnd(1, hk * D)
        p = p.bfloat16()
        at = [0, hk * D, 2 * hk * D, (2 * hk + hv) * D, (2 * hk + hv) * D + hv]
        self.q = p[:, :at[1]].unflatten(1, (hk, D))
        self.k = p[:, at[1]:at[2]].unflatten(1, (hk, D))
        self.v = p[:, at[2]:at[3]].unflatten(1, (hv, D))
        self.a = p[:, at[3]:at[4]]
        self.beta = p[:, at[4]:at[4] + hv]
        if not packed:
            self.dense()
        self.T, self.hk, self.hv = T, hk, hv
        self.A_log = torch.rand(hv, generator=g, device="cuda").mul(2.7)
        self.dt_bias = rnd(hv) - 3
        self.scale = D ** -0.5

    def dense(self):
        for x in ("q", "k", "v", "a", "beta"):
            setattr(self, x, getattr(self, x).contiguous())

    def rows(self):
        return self.q, self.k, self.v, self.a, self.beta, self.A_log, self.dt_bias, self.scale


def _state(shape, dtype, seed):
    import torch
    return torch.randn(*shape, generator=_gen(seed), device="cuda").mul(0.5).to(dtype)


def _reference(x, spans, s0):
    """out rows and final states in fp64, token after token, all sequences in step; and M."""
    import torch
    n, grp = len(spans), x.hv // x.hk
    q, k, v, a, b = (t.double() for t in (x.q, x.k, x.v, x.a, x.beta))
    q = (q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(grp, 1)
    k = (k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(grp, 1)
    z = a + x.dt_bias.double()
    decay = (-x.A_log.double().exp() * torch.where(z > 30, z, z.clamp(max=30).exp().log1p())).exp()
    beta = torch.sigmoid(b)
    S = s0.double().clone() if s0 is not None else torch.zeros(n, x.hv, D, D, dtype=torch.float64, device="cuda")
    out = torch.zeros(x.T, x.hv, D, dtype=torch.float64, device="cuda")
    M = S.square().sum(2).sqrt().max().item()
    for i in range(max([t1 - t0 for t0, t1 in spans] + [0])):
        live = [j for j, (t0, t1) in enumerate(spans) if t0 + i < t1]
        at = [spans[j][0] + i for j in live]
        s = S[live] * decay[at][..., None, None]
        w = beta[at][..., None] * (v[at] - (k[at][..., None] * s).sum(2))
        s = s + k[at][..., None] * w[:, :, None, :]
        S[live] = s
        out[at] = x.scale * (q[at][..., None] * s).sum(2)
        M = max(M, s.square().sum(2).sqrt().max().item())
    return out, S, M + (v.abs().max().item() if x.T else 0.0)


def _spans(lens):
    at, spans = 0, []
    for n in lens:
        spans.append((at, at + n))
        at += n
    return spans


def _prefill(x, lens, dtype, s0=None, out=None, fin=None, ws=None, fill=0.0, stream=None):
    import torch
    kda = _kda()
    cu = torch.tensor([0] + [b for _, b in _spans(lens)], dtype=torch.int32, device="cuda")
    if out is None:
        out = torch.full((x.T, x.hv, D), fill, dtype=torch.bfloat16, device="cuda")
    if fin is None:
        fin = torch.full((len(lens), x.hv, D, D), float("nan"), dtype=dtype, device="cuda")
    if ws is None:
        ws = torch.full((kda.kda_gdr_get_workspace_size(x.T, x.hk, x.hv, len(lens)),), 0xFF,
                        dtype=torch.uint8, device="cuda")
    kda.kda_gdr_prefill_fwd(*x.rows(), s0, cu, out, fin, ws, stream=stream)
    return out, fin


def _check_gdr(x, spans, out, fin, ref, dtype, label, rows=None, rms=False):
    import torch
    o, S, M = ref
    longest = max(t1 - t0 for t0, t1 in spans)
    cut = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    tol = max(1, -(-longest // 64)) * (4 * 192 * U + 8 * cut) * M
    tol_o = x.scale * (tol + 3 * 2.0 ** -11 * M)
    do, ds = (out.double() - o).abs(), (fin.double() - S).abs()
    if rows is not None:
        do, o = do[rows], o[rows]
    worst_o = (do - 2.0 ** -8 * o.abs()).max().item() if do.numel() else 0.0
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    worst_s = (ds - half * S.abs()).max().item()
    rel_o, rel_s = ((d.norm() / y.norm().clamp(min=1e-300)).item() for d, y in ((do, o), (ds, S)))
    print(f"[parity] {label}: out {worst_o:.3g} of {tol_o:.3g}, rel {rel_o:.3g}, state {worst_s:.3g} of {tol:.3g}, "
          f"rel {rel_s:.3g}", flush=True)
    assert worst_o <= tol_o and worst_s <= tol, label
    if rms:
        assert rel_o <= 2.4e-3 and rel_s <= (2.4e-3 if dtype == torch.bfloat16 else 2.3e-6), label


CHUNKED = [
    ([100], 1, 1), ([64], 2, 4), ([65, 1, 0, 63, 130], 2, 2), ([200, 129], 1, 4), ([16, 17, 33, 48, 49], 3, 9),
    ([700], 5, 5), ([1, 300, 1, 0, 0, 128], 2, 6), ([9] * 20, 1, 2), ([257] * 40, 1, 2),
    # more sequences than a wave holds; more workgroups than run at once, longest sequences first
    ([10] * 100 + [70, 0, 200, 64, 1], 1, 2), ([i * 37 % 150 for i in range(33)], 4, 8),
]


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,hk,hv", CHUNKED, ids=lambda v: str(v)[:24])
def test_prefill(lens, hk, hv, state):
    """Both forms of the scan (few and many workgroups), ragged and empty
    sequences, shared key heads, with an initial state."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(sum(lens), hk, hv, seed=len(lens) + hv)
    s0 = _state((len(lens), hv, D, D), dtype, 3)
    out, fin = _prefill(x, lens, dtype, s0)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), dtype, f"{lens} {hk}/{hv} {state}",
               rms=True)


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,hk,hv,init", [([2500], 1, 2, True), ([5000], 4, 8, False), ([2048], 1, 1, True),
                                             ([9000, 0, 300, 1], 1, 2, True), ([4300, 4100], 8, 8, True)], ids=str)
def test_prefill_in_segments(lens, hk, hv, init, state):
    """Few states and long sequences: segments at once, joined by their maps;
    one in five tokens almost erases the state, the others keep nearly all of
    it.  Tokens behind the last sequence stay."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(sum(lens) + 5, hk, hv, seed=len(lens) + hv, packed=True)
    x.a = x.a - 6 + 14 * (torch.rand(x.a.shape, generator=_gen(1), device="cuda") < 0.2).bfloat16()
    s0 = _state((len(lens), hv, D, D), dtype, 3) if init else None
    out, fin = _prefill(x, lens, dtype, s0, fill=3.0)
    assert (out[-5:] == 3.0).all()
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), dtype, f"segments {lens} {state}",
               rows=slice(0, sum(lens)), rms=True)


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[1], [8], [3, 0, 8, 1, 20], [1] * 600], ids=lambda v: str(v)[:20])
def test_prefill_of_few_tokens(lens, state):
    """At most 8 tokens per sequence: the serial kernel."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(sum(lens), 2, 4, seed=len(lens), packed=True)
    s0 = _state((len(lens), 4, D, D), dtype, 5)
    out, fin = _prefill(x, lens, dtype, s0)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), dtype, f"{str(lens)[:20]} {state}", rms=True)


@pytest.mark.parametrize("lens", [[300, 70], [2, 5]], ids=str)
def test_prefill_from_nothing_in_place_and_strided(lens):
    """No initial state; the same from zeros, in place, and from strided views:
    the same bits each time, also on another workspace's rubbish."""
    import torch
    x = Gdr(sum(lens), 2, 4, seed=8, packed=True)
    out, fin = _prefill(x, lens, torch.float32)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), None), torch.float32, str(lens))
    s = torch.zeros_like(fin)
    out2, _ = _prefill(x, lens, torch.float32, s, fin=s)
    assert torch.equal(out, out2) and torch.equal(fin, s)
    x.dense()
    wide = torch.zeros(x.T, 4, 2 * D, dtype=torch.bfloat16, device="cuda")
    _, fin3 = _prefill(x, lens, torch.float32, out=wide[:, :, 64:64 + D])
    assert torch.equal(out, wide[:, :, 64:64 + D]) and torch.equal(fin, fin3)
    assert not wide[:, :, :64].any() and not wide[:, :, 64 + D:].any()


@pytest.mark.parametrize("lens", [[150, 30], [3, 4]], ids=str)
def test_rows_behind_the_last_sequence_stay(lens):
    import torch
    x = Gdr(sum(lens) + 70, 1, 2, seed=9)
    out, fin = _prefill(x, lens, torch.float32, fill=7.0)
    n = sum(lens)
    assert (out[n:] == 7.0).all()
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), None), torch.float32, str(lens),
               rows=slice(0, n))


def test_no_tokens():
    import torch
    x = Gdr(0, 1, 2, seed=10)
    s0 = _state((3, 2, D, D), torch.float32, 1)
    _, fin = _prefill(x, [0, 0, 0], torch.float32, s0)
    assert torch.equal(fin, s0)


@pytest.mark.parametrize("lens", [[400], [6]], ids=str)
def test_decays_of_every_size(lens):
    """Gates from almost 1 to e^-800 and below (infinite raw gates too), mixed
    in one chunk: tokens that erase the state between tokens that keep it."""
    import torch
    x = Gdr(lens[0], 1, 3, seed=11)
    raw = torch.tensor([-40.0, 0.0, 100.0, -40.0, -40.0, -3.0, float("inf"), -40.0, float("-inf")], device="cuda")
    x.a = raw[torch.randint(0, 9, (lens[0], 3), generator=_gen(2), device="cuda")].bfloat16()
    x.a[:, 1] = -30.0
    s0 = _state((1, 3, D, D), torch.float32, 4)
    out, fin = _prefill(x, lens, torch.float32, s0)
    y = Gdr(lens[0], 1, 3, seed=11)
    y.a = x.a.float().clamp(-1e4, 1e4).bfloat16()
    _check_gdr(x, _spans(lens), out, fin, _reference(y, _spans(lens), s0), torch.float32, f"decays {lens}")


@pytest.mark.parametrize("lens", [[150], [7]], ids=str)
def test_decay_rates_of_any_size(lens):
    """exp(A_log) beyond fp32 times a softplus below it: a finite decay."""
    import torch
    x = Gdr(lens[0], 1, 4, seed=23)
    x.A_log = torch.tensor([90.0, 120.0, 87.0, -120.0], device="cuda")
    x.dt_bias = torch.zeros(4, device="cuda")
    rate = torch.tensor([[-95.0, -127.0, -92.0, 100.0], [-112.0, -200.0, -100.0, 3e38]], device="cuda")
    x.a = rate[torch.arange(lens[0], device="cuda") % 2].bfloat16()
    s0 = _state((1, 4, D, D), torch.float32, 13)
    out, fin = _prefill(x, lens, torch.float32, s0)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), torch.float32, f"rates {lens}")


def test_keys_of_one_direction():
    """Nearly equal keys and hardly any decay: the triangle is far from the identity."""
    import torch
    x = Gdr(520, 2, 2, seed=12, correlated=True)
    x.dt_bias = x.dt_bias - 8
    out, fin = _prefill(x, [520], torch.float32)
    _check_gdr(x, [(0, 520)], out, fin, _reference(x, [(0, 520)], None), torch.float32, "correlated")


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e8, 1e30])
def test_values_and_states_of_any_size(size, state):
    """Each column carries its own power of two: the relative error does not
    depend on the size of the values, nor on that of the column beside."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(300, 1, 2, seed=16)
    x.v[:, 0, ::2] *= size
    s0 = _state((1, 2, D, D), dtype, 8)
    s0[:, 0, :, ::2] *= size
    out, fin = _prefill(x, [300], dtype, s0)
    o, S, _ = _reference(x, [(0, 300)], s0)
    for at in (slice(0, None, 2), slice(1, None, 2)):
        d, y = out.double()[:, 0, at] - o[:, 0, at], o[:, 0, at]
        assert d.norm() <= 2.4e-3 * y.norm()
        d, y = fin.double()[:, 0, :, at] - S[:, 0, :, at], S[:, 0, :, at]
        assert d.norm() <= (2.3e-6 if dtype == torch.float32 else 2.4e-3) * y.norm()


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[500], [2500], [8]], ids=str)
@pytest.mark.parametrize("size", [1e9, 1e30, 1e37])
def test_large_states_that_are_forgotten(lens, state, size):
    """A column far above one is erased, then values of zero in whole chunks:
    zeros, not 0 times infinity; values that follow are those of a new sequence."""
    import torch
    dtype = getattr(torch, state)
    n = lens[0]
    x = Gdr(n, 1, 2, seed=19)
    x.a[:] = 100.0
    keep = x.v.clone()
    x.v[:] = 0
    s0 = _state((1, 2, D, D), dtype, 10).clamp(-1, 1)
    s0[:, 0, :, ::2] *= size
    out, fin = _prefill(x, lens, dtype, s0)
    assert (out == 0).all() and (fin == 0).all()
    if n > 192:
        x.a[192:] = -1.0
        x.v[192:, :, 1:] = keep[192:, :, 1:]  # column 0 stays zero
        x.v[192:] *= 1e-9
        out, fin = _prefill(x, lens, dtype, s0)
        assert (out[:192] == 0).all() and (out[..., 0] == 0).all() and (fin[..., 0] == 0).all()
        y = Gdr(n - 192, 1, 2, seed=19)
        for f in ("q", "k", "v", "a", "beta"):
            setattr(y, f, getattr(x, f)[192:])
        y.A_log, y.dt_bias = x.A_log, x.dt_bias
        _check_gdr(y, [(0, y.T)], out[192:], fin, _reference(y, [(0, y.T)], None), dtype, f"forgotten {size} {state}")


@pytest.mark.parametrize("size", [1e-18, 1e15])
def test_keys_and_queries_of_any_size(size):
    import torch
    x = Gdr(200, 1, 1, seed=17)
    x.k *= size
    x.q /= size
    out, fin = _prefill(x, [200], torch.float32)
    _check_gdr(x, [(0, 200)], out, fin, _reference(x, [(0, 200)], None), torch.float32, f"keys times {size}")


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[200], [7], [2100]], ids=str)
@pytest.mark.parametrize("size", [1e-35, 1e10, 1e19, 1e37])
def test_rows_of_keys_and_queries_of_any_size(size, lens, state):
    """Rows whose squares fp32 does not hold, among ordinary ones and next to each other."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(lens[0], 1, 2, seed=21)
    x.k[1::3] *= size
    x.k[2::6] *= size
    x.q[2::5] *= size
    x.q[1] *= size
    s0 = _state((1, 2, D, D), dtype, 11)
    out, fin = _prefill(x, lens, dtype, s0)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), dtype, f"rows times {size}")


def test_zero_rows():
    """Keys and queries of zeros have norm 1e-3: no division by zero, and no update."""
    import torch
    x = Gdr(90, 1, 1, seed=13)
    x.k[10:40] = 0
    x.q[30:50] = 0
    out, fin = _prefill(x, [90], torch.float32)
    assert (out[30:50] == 0).all()
    _check_gdr(x, [(0, 90)], out, fin, _reference(x, [(0, 90)], None), torch.float32, "zero rows")


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[150], [6], [2300]], ids=str)
def test_zero_keys_that_nothing_forgets(lens, state):
    """Keys of zeros, and of less than a normal number, with values beside them
    and hardly any decay up to the chunk's end: no update, no overflow."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(lens[0], 1, 2, seed=18)
    x.dt_bias = x.dt_bias - 9
    x.k[lens[0] // 3:lens[0] // 2] = 0
    x.k[lens[0] - 3] = 1e-39
    s0 = _state((1, 2, D, D), dtype, 9)
    out, fin = _prefill(x, lens, dtype, s0)
    _check_gdr(x, _spans(lens), out, fin, _reference(x, _spans(lens), s0), dtype, f"zero keys {lens} {state}")


@pytest.mark.parametrize("lens", [[130, 100, 70], [2, 3, 4]], ids=str)
def test_what_is_not_finite_stays_in_its_sequence_and_head(lens):
    import torch
    x = Gdr(sum(lens), 2, 4, seed=14)
    out, fin = _prefill(x, lens, torch.float32)
    x.v[lens[0], 1] = float("nan")
    x.a[lens[0] + 1, 3] = float("nan")
    bad, bfin = _prefill(x, lens, torch.float32)
    keep = torch.ones(sum(lens), 4, dtype=torch.bool, device="cuda")
    keep[lens[0]:lens[0] + lens[1], 1::2] = False
    assert torch.equal(out[keep], bad[keep])
    keep = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    keep[1, 1::2] = False
    assert torch.equal(fin[keep], bfin[keep])
    assert bad[lens[0], 1].isnan().all() and bfin[1, 1].isnan().any() and bfin[1, 3].isnan().any()


def test_same_call_same_bits_on_any_stream():
    import torch
    lens = [333, 64, 500]
    x = Gdr(sum(lens), 2, 4, seed=15)
    first = _prefill(x, lens, torch.bfloat16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a = _prefill(x, lens, torch.bfloat16)
        b = _prefill(x, lens, torch.bfloat16, stream=s)
    s.synchronize()
    for y in (a, b):
        assert torch.equal(first[0], y[0]) and torch.equal(first[1], y[1])


@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,hk,hv", [(1, 1, 1), (5, 2, 6), (150, 2, 4), (129, 4, 4)])
def test_decode(n, hk, hv, state):
    """Random slots, padding rows (below zero and past the pool), strided rows;
    slots that no row names keep their bits."""
    import torch
    dtype = getattr(torch, state)
    x = Gdr(n, hk, hv, seed=20 + n, packed=True)
    pool = _state((n + 7, hv, D, D), dtype, 6)
    before = pool.clone()
    idx = torch.randperm(n + 7, generator=_gen(7), device="cuda")[:n].int()
    if n > 4:
        idx[1], idx[3] = -1, n + 7
    out = torch.full((n, hv, D), 5.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_gdr_decode_step(*x.rows(), pool, idx, out)
    live = (idx >= 0) & (idx < n + 7)
    y = Gdr(0, hk, hv, seed=20 + n)
    for f in ("q", "k", "v", "a", "beta"):
        setattr(y, f, getattr(x, f)[live])
    y.A_log, y.dt_bias, y.T = x.A_log, x.dt_bias, int(live.sum())
    slots = idx[live].long()
    spans = _spans([1] * y.T)
    _check_gdr(y, spans, out[live], pool[slots], _reference(y, spans, before[slots]), dtype, f"decode {n} {state}")
    assert (out[~live] == 5.0).all()
    rest = torch.ones(n + 7, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert torch.equal(pool[rest], before[rest])


def test_decode_of_large_keys_and_queries():
    import torch
    x = Gdr(9, 1, 2, seed=22)
    x.k[:3] *= 1e37
    x.q[2:5] *= 1e19
    x.k[6] *= 1e18
    x.q[6] *= 1e-20
    pool = _state((9, 2, D, D), torch.float32, 12)
    before = pool.clone()
    out = torch.zeros(9, 2, D, dtype=torch.bfloat16, device="cuda")
    _kda().kda_gdr_decode_step(*x.rows(), pool, torch.arange(9, dtype=torch.int32, device="cuda"), out)
    spans = _spans([1] * 9)
    _check_gdr(x, spans, out, pool, _reference(x, spans, before), torch.float32, "decode, large keys")


def test_prefill_then_decode_is_a_longer_prefill():
    import torch
    lens = [70, 129, 64]
    x = Gdr(sum(lens) + 3, 2, 4, seed=30)
    spans, at = [], 0
    for n in lens:
        spans.append((at, at + n + 1))
        at += n + 1
    ref = _reference(x, spans, None)
    head = torch.cat([torch.arange(t0, t1 - 1) for t0, t1 in spans]).cuda()
    last = torch.tensor([t1 - 1 for _, t1 in spans]).cuda()
    y, z = Gdr(0, 2, 4, seed=30), Gdr(0, 2, 4, seed=30)
    for f in ("q", "k", "v", "a", "beta"):
        setattr(y, f, getattr(x, f)[head])
        setattr(z, f, getattr(x, f)[last])
    y.T, z.T = len(head), 3
    for w in (y, z):
        w.A_log, w.dt_bias = x.A_log, x.dt_bias
    out = torch.zeros(x.T, 4, D, dtype=torch.bfloat16, device="cuda")
    out[head], pool = _prefill(y, lens, torch.float32)
    o = torch.zeros(3, 4, D, dtype=torch.bfloat16, device="cuda")
    _kda().kda_gdr_decode_step(*z.rows(), pool, torch.arange(3, dtype=torch.int32, device="cuda"), o)
    out[last] = o
    _check_gdr(x, spans, out, pool, ref, torch.float32, "prefill + decode")


# ---- the norm ---------------------------------------------------------------

def _norm_reference(x, r, w, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    return s, s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def _norm_inputs(m, dim, seed, pad=0, residual=True):
    import torch
    g = _gen(seed)
    x = torch.randn(m, dim + pad, generator=g, device="cuda").bfloat16()[:, :dim]
    r = torch.randn(m, dim + pad, generator=g, device="cuda").mul(3).bfloat16()[:, :dim] if residual else None
    w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).bfloat16()
    return x, r, w


def _check_norm(x, r, w, res_after, out, scale, group, label, eps=1e-6):
    import torch
    dim = x.shape[1]
    s, y = _norm_reference(x, r, w, eps)
    if r is not None:
        assert ((res_after.double() - s).abs() <= 2.0 ** -8 * s.abs() + 2 * U * s.abs()).all(), label
    rel = (dim / 2 + 8) * U
    if scale is None:
        d = (out.double() - y).abs()
        assert (d <= (2.0 ** -8 + 2 * rel) * y.abs() + 2.0 ** -134).all(), f"{label}: {d.max()}"
        return
    width = group or dim
    groups = -(-dim // width)
    yp = torch.nn.functional.pad(y, (0, groups * width - dim)).unflatten(1, (groups, width))
    c = yp.abs().amax(-1) / 448
    got = scale.double().view(-1, groups)
    assert ((got - c).abs() <= 2 * rel * c).all(), f"{label}: scales"
    per = got.repeat_interleave(width, 1)[:, :dim]
    d = (out.double() * per - y).abs()
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * per)
    assert (d <= bound * (1 + 1e-3) + 4 * rel * y.abs()).all(), f"{label}: codes"
    assert out.float().abs().amax() <= 448


DIMS = [1, 7, 8, 100, 127, 128, 129, 511, 512, 520, 2047, 2048, 2056, 4096, 4100, 7168, 8192, 8200, 16384, 16391,
        32768]


@pytest.mark.parametrize("out", ["bf16", "rows", "groups"])
@pytest.mark.parametrize("dim", DIMS)
def test_norm(dim, out):
    import torch
    for m, residual in ((1, True), (5, False), (3, True)):
        x, r, w = _norm_inputs(m, dim, dim + m, residual=residual)
        ra = r.clone() if residual else None
        fp8 = out != "bf16"
        o = torch.empty(m, dim, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
        group = 128 if out == "groups" else 0
        sc = torch.full((m, -(-dim // 128) if group else 1), -1.0, device="cuda") if fp8 else None
        _kda().kda_add_rms_norm(x, ra, w, 1e-6, o, sc, group)
        _check_norm(x, r, w, ra, o, sc, group, f"{m}x{dim} {out}")


@pytest.mark.parametrize("dim,pad", [(256, 8), (256, 3), (300, 1), (7168, 64)])
def test_norm_of_strided_rows_and_in_place(dim, pad):
    """Views of wider matrices, aligned and not; what lies between the rows stays; out = x."""
    import torch
    x, r, w = _norm_inputs(6, dim, 40, pad)
    whole = r._base.clone()
    ra = r._base[:, :dim]
    keep = r.clone()
    o = torch.full((6, dim + pad), 9.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_add_rms_norm(x, ra, w, 1e-6, o[:, :dim])
    _check_norm(x, keep, w, ra, o[:, :dim], None, 0, "strided")
    assert (o[:, dim:] == 9.0).all() and torch.equal(ra._base[:, dim:], whole[:, dim:])
    z = x.clone()
    _kda().kda_add_rms_norm(z, None, w, 1e-6, z)
    _check_norm(x, None, w, None, z, None, 0, "in place")
    q = torch.zeros(6, dim + pad, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(6, device="cuda")
    _kda().kda_add_rms_norm(x, None, w, 1e-6, q[:, :dim], sc)
    _check_norm(x, None, w, None, q[:, :dim], sc, 0, "strided codes")
    assert not q.view(torch.uint8)[:, dim:].any()


def test_norm_of_zeros_and_of_what_is_not_finite():
    import torch
    x, _, w = _norm_inputs(4, 300, 41, residual=False)
    x = x.contiguous()
    x[1] = 0
    x[2, :128] = 0
    x[3, 5] = float("nan")
    o = torch.empty(4, 300, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 3, device="cuda")
    _kda().kda_add_rms_norm(x, None, w, 1e-6, o, sc, 128)
    assert not sc[1].any() and not o[1].view(torch.uint8).any()
    assert sc[2, 0] == 0 and not o[2, :128].view(torch.uint8).any() and sc[2, 1] > 0
    assert sc[3].isnan().all()
    _check_norm(x[:3], None, w, None, o[:3], sc[:3], 128, "zeros")
    b = torch.empty(4, 300, dtype=torch.bfloat16, device="cuda")
    _kda().kda_add_rms_norm(x, None, w, 0.0, b)
    assert b[3].isnan().all()


@pytest.mark.parametrize("out", ["bf16", "rows", "groups"])
@pytest.mark.parametrize("dim", [100, 512, 2056, 16391])
@pytest.mark.parametrize("size,eps", [(1e20, 1e-6), (1e37, 0.0), (1e-20, 0.0), (1e-30, 0.0), (1e-15, 1e-30)])
def test_norm_of_rows_of_any_size(size, eps, dim, out):
    """Rows whose sum of squares fp32 does not hold, either way, and a row of zeros without eps."""
    import torch
    fp8 = out != "bf16"
    group = 128 if out == "groups" else 0
    for residual in (False, True):
        x, r, w = _norm_inputs(4, dim, dim + 9, residual=residual)
        x = x * size
        x[2] = 0
        if residual:
            r = r * size
            r[2] = 0
        ra = r.clone() if residual else None
        o = torch.empty(4, dim, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
        sc = torch.full((4, -(-dim // 128) if group else 1), -1.0, device="cuda") if fp8 else None
        _kda().kda_add_rms_norm(x, ra, w, eps, o, sc, group)
        rows = [0, 1, 3]
        _check_norm(x[rows], r[rows] if residual else None, w, ra[rows] if residual else None, o[rows],
                    sc[rows] if fp8 else None, group, f"{size} {dim} {out}", eps=eps)
        assert not o[2].float().any() and not (fp8 and sc[2].any())


@pytest.mark.parametrize("dim", [300, 2048, 2056])
def test_norm_of_infinities(dim):
    """What the formula gives: NaN in the place of an infinity, zeros beside it;
    in e4m3 a NaN scale for its group and scales and codes of zero for the others."""
    import torch
    x, _, w = _norm_inputs(3, dim, 43, residual=False)
    x = x.contiguous()
    x[0, 5] = float("inf")
    x[2, 5] = float("-inf")
    b = torch.empty(3, dim, dtype=torch.bfloat16, device="cuda")
    _kda().kda_add_rms_norm(x, None, w, 1e-6, b)
    o = torch.empty(3, dim, dtype=torch.float8_e4m3fn, device="cuda")
    sc, sr = torch.empty(3, -(-dim // 128), device="cuda"), torch.empty(3, 1, device="cuda")
    _kda().kda_add_rms_norm(x, None, w, 1e-6, o, sc, 128)
    for i in (0, 2):
        assert b[i, 5].isnan() and not b[i, :5].any() and not b[i, 6:].any()
        assert sc[i, 0].isnan() and not sc[i, 1:].any() and not o[i, 128:].float().any()
    _check_norm(x[1:2], None, w, None, o[1:2], sc[1:2], 128, "beside infinities")
    _kda().kda_add_rms_norm(x, None, w, 1e-6, o, sr)
    assert sr[0].isnan() and sr[2].isnan()
    _check_norm(x[1:2], None, w, None, o[1:2], sr[1:2], 0, "beside infinities")


def test_norm_of_many_rows():
    """More rows than one row of the grid holds (2^20)."""
    import torch
    m = (1 << 20) + 77
    x, r, w = _norm_inputs(m, 24, 42)
    ra = r.clone()
    o = torch.zeros(m, 24, dtype=torch.bfloat16, device="cuda")
    _kda().kda_add_rms_norm(x, ra, w, 1e-5, o)
    _check_norm(x, r, w, ra, o, None, 0, "many rows", eps=1e-5)


# ---- 4-bit products ---------------------------------------------------------

def _w4_inputs(m, k, n, group, zeros, seed, pad=0):
    import torch
    g = _gen(seed)
    x = torch.randn(m, k + pad, generator=g, device="cuda").bfloat16()[:, :k]
    w = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(n, k // group, generator=g, device="cuda") - 0.3).mul(0.1).bfloat16()
    z = torch.randint(0, 16, (n, k // group), generator=g, device="cuda").bfloat16() if zeros else None
    return x, w, s, z


def _w4_check(x, w, s, z, group, y, label):
    """A group's sum is formed as sum (128 + q) x - (128 + z) sum x: at most
    group terms of magnitude 143 |x| each, twice, in fp32 (group u each), a
    product with the scale, and the sum over the groups (at most K / group
    terms in order over 8 waves), plus bf16's half step."""
    import torch
    k = x.shape[1]
    q = torch.stack((w & 15, w >> 4), -1).flatten(1).double().unflatten(1, (-1, group))
    d = (q - (8.0 if z is None else z.double()[..., None])) * s.double()[..., None]
    xd = x.double()
    ref = xd @ d.flatten(1).T
    mag = xd.abs() @ s.double().abs().repeat_interleave(group, 1).T
    bound = 2.0 ** -8 * ref.abs() + (2 * (group + 4) + k / group + 8) * U * 143 * mag
    err = (y.double() - ref).abs()
    print(f"[parity] {label}: {(err - 2.0 ** -8 * ref.abs()).max().item():.3g}", flush=True)
    assert (err <= bound).all(), label


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,k,n,group", [
    (1, 32, 1, 32), (1, 7168, 1536, 128), (2, 96, 17, 32), (3, 160, 33, 32), (15, 192, 100, 64), (16, 448, 31, 64),
    (17, 1024, 16, 128), (31, 1152, 15, 128), (33, 4128, 70, 32), (64, 2048, 145, 64), (5, 1088, 144, 64),
    (1, 128, 5000, 128), (64, 16384, 3, 128), (50, 512, 4200, 64), (33, 256, 4111, 128), (20, 256, 5000, 32),
    (3, 256, 12400, 64), (16, 384, 4300, 128),
    # more groups than LDS holds scales of at a time
    (5, 9632, 40, 32), (16, 17408, 33, 64), (40, 4192, 4100, 32), (1, 33024, 17, 128),
])
def test_w4(m, k, n, group, zeros):
    import torch
    x, w, s, z = _w4_inputs(m, k, n, group, zeros, m + n)
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    _kda().kda_w4_proj(x, w, s, z, y, group)
    _w4_check(x, w, s, z, group, y, f"{m}x{k}x{n} g{group}")
    y2 = torch.empty_like(y)
    _kda().kda_w4_proj(x, w, s, z, y2, group)
    assert torch.equal(y, y2)


def test_w4_of_strided_rows():
    import torch
    x, w, s, z = _w4_inputs(9, 256, 50, 64, True, 50, pad=24)
    y = torch.full((9, 61), 3.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_w4_proj(x, w, s, z, y[:, 7:57], 64)
    _w4_check(x, w, s, z, 64, y[:, 7:57], "strided")
    assert (y[:, :7] == 3.0).all() and (y[:, 57:] == 3.0).all()


def test_w4_rows_do_not_mix():
    """A token's NaN stays in its row, and a row's result does not depend on the tokens beside it."""
    import torch
    x, w, s, z = _w4_inputs(16, 512, 64, 64, False, 51)
    y = torch.empty(16, 64, dtype=torch.bfloat16, device="cuda")
    _kda().kda_w4_proj(x, w, s, z, y, 64)
    one = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
    _kda().kda_w4_proj(x[4:5], w, s, z, one, 64)
    assert torch.equal(one[0], y[4])
    x2 = x.clone()
    x2[3, 100] = float("nan")
    y2 = torch.empty_like(y)
    _kda().kda_w4_proj(x2, w, s, z, y2, 64)
    assert y2[3].isnan().all() and torch.equal(y2[4:], y[4:]) and torch.equal(y2[:3], y[:3])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,k,n,group", [(1, 512, 100, 128), (16, 160, 33, 32), (40, 512, 4200, 64)])
@pytest.mark.parametrize("size", [1e-30, 1e30, 1e37, 3e38])
def test_w4_of_values_of_any_size(size, m, k, n, group, zeros):
    """Sums of 143 |x| beyond fp32 whose result is not."""
    import torch
    x, w, s, z = _w4_inputs(m, k, n, group, zeros, 53)
    x = (x.clamp(-1, 1) * size).bfloat16()
    s = s * 2.0 ** -12
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    _kda().kda_w4_proj(x, w, s, z, y, group)
    _w4_check(x, w, s, z, group, y, f"{size} {m}x{k}x{n}")


def test_w4_rows_do_not_depend_on_the_tokens_beside():
    """At one number of tokens, where each wave sums several blocks of k."""
    import torch
    for m in (3, 16, 40):
        x, w, s, z = _w4_inputs(m, 7168, 70, 64, True, 54)
        y = torch.empty(m, 70, dtype=torch.bfloat16, device="cuda")
        _kda().kda_w4_proj(x, w, s, z, y, 64)
        x2 = torch.randn(m, 7168, generator=_gen(55), device="cuda").bfloat16()
        x2[1] = x[1]
        y2 = torch.empty_like(y)
        _kda().kda_w4_proj(x2, w, s, z, y2, 64)
        assert torch.equal(y[1], y2[1])


# ---- together ---------------------------------------------------------------

class Layer:
    """A decode step of one layer: residual + norm -> 4-bit projection to q, k, v,
    a, beta -> delta rule on the pool -> 4-bit output projection -> residual +
    norm into e4m3."""

    def __init__(self, n, hidden, hk, hv, seed):
        import torch
        self.n, self.hidden, self.hk, self.hv = n, hidden, hk, hv
        cols = (2 * hk + hv) * D + 2 * hv
        self.cols = cols
        _, self.w_in, self.s_in, self.z_in = _w4_inputs(1, hidden, cols, 64, True, seed)
        _, self.w_out, self.s_out, _ = _w4_inputs(1, hv * D, hidden, 128, False, seed + 1)
        self.x, self.r, self.nw = _norm_inputs(n, hidden, seed + 2)
        g = Gdr(0, hk, hv, seed + 3)
        self.A_log, self.dt_bias, self.scale = g.A_log, g.dt_bias, g.scale
        self.pool = _state((n + 2, hv, D, D), torch.float32, seed + 4)
        self.idx = torch.arange(n + 1, 1, -1, dtype=torch.int32, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.h, self.p = torch.zeros(n, hidden, **bf), torch.zeros(n, -(-cols // 8) * 8, **bf)
        self.o, self.y = torch.zeros(n, hv, D, **bf), torch.zeros(n, hidden, **bf)
        self.q8 = torch.zeros(n, hidden, dtype=torch.float8_e4m3fn, device="cuda")
        self.c8 = torch.zeros(n, -(-hidden // 128), device="cuda")

    def views(self):
        at = [0, self.hk * D, 2 * self.hk * D, (2 * self.hk + self.hv) * D]
        p = self.p
        return (p[:, :at[1]].unflatten(1, (self.hk, D)), p[:, at[1]:at[2]].unflatten(1, (self.hk, D)),
                p[:, at[2]:at[3]].unflatten(1, (self.hv, D)), p[:, at[3]:at[3] + self.hv],
                p[:, at[3] + self.hv:at[3] + 2 * self.hv])

    def step(self):
        kda = _kda()
        kda.kda_add_rms_norm(self.x, self.r, self.nw, 1e-6, self.h)
        kda.kda_w4_proj(self.h, self.w_in, self.s_in, self.z_in, self.p[:, :self.cols], 64)
        kda.kda_gdr_decode_step(*self.views(), self.A_log, self.dt_bias, self.scale, self.pool, self.idx, self.o)
        kda.kda_w4_proj(self.o.view(self.n, -1), self.w_out, self.s_out, None, self.y, 128)
        kda.kda_add_rms_norm(self.y, self.r, self.nw, 1e-6, self.q8, self.c8, 128)

    def results(self):
        import torch
        return [t.clone() for t in (self.r, self.h, self.p, self.o, self.y, self.q8.view(torch.uint8), self.c8,
                                    self.pool)]


@pytest.mark.parametrize("n", [1, 6])
def test_a_layers_decode_step(n):
    """Each operator on what the one before it wrote, against the 64-bit forms;
    then the step captured in a graph and replayed, each replay equal to the
    eager step from the same pool and residual."""
    import torch
    m = Layer(n, 1024, 2, 4, 60)
    r0, pool0 = m.r.clone(), m.pool.clone()
    m.step()
    eager = m.results()
    r1 = (m.x.double() + r0.double()).bfloat16()
    _check_norm(m.x, r0, m.nw, r1, m.h, None, 0, "first norm")
    _w4_check(m.h, m.w_in, m.s_in, m.z_in, 64, m.p[:, :m.cols], "projection")
    g = Gdr(0, 2, 4, 63)
    g.q, g.k, g.v, g.a, g.beta = m.views()
    g.T, g.A_log, g.dt_bias = n, m.A_log, m.dt_bias
    slots, spans = m.idx.long(), _spans([1] * n)
    _check_gdr(g, spans, m.o, m.pool[slots], _reference(g, spans, pool0[slots]), torch.float32, "delta rule")
    _w4_check(m.o.view(n, -1), m.w_out, m.s_out, None, 128, m.y, "output projection")
    _check_norm(m.y, r1, m.nw, m.r, m.q8, m.c8, 128, "second norm")

    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        m.step()
    torch.cuda.synchronize()
    for i in range(3):
        m.r.copy_(r0)
        m.pool.copy_(pool0)
        for t in (m.h, m.p, m.o, m.y, m.c8):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, m.results()):
            assert torch.equal(a, b), f"replay {i}"


def test_prefill_in_a_graph():
    """Both launches of the chunked prefill captured and replayed between eager
    calls on another workspace."""
    import torch
    kda = _kda()
    lens = [200, 77]
    x = Gdr(sum(lens), 2, 4, seed=70)
    out, fin = _prefill(x, lens, torch.float32)
    ws = torch.empty(kda.kda_gdr_get_workspace_size(x.T, 2, 4, 2), dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 200, 277], dtype=torch.int32, device="cuda")
    o, f = torch.zeros_like(out), torch.zeros_like(fin)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        kda.kda_gdr_prefill_fwd(*x.rows(), None, cu, o, f, ws)
    for i in range(3):
        o.zero_()
        f.zero_()
        ws.fill_(0xFF)
        graph.replay()
        _prefill(Gdr(500, 2, 4, seed=71), [500], torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(f, fin), f"replay {i}"
