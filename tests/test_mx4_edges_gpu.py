"""The operators of include/kda_mx4.h where they can go wrong without any result looking
odd: the experts' layer on inputs whose exact answer is a small whole number or an
order and on weights beyond 4 GiB; tiles with rows of y in whole pieces that n does not
fill, and with scales and k that are read as they lie."""
from __future__ import annotations

import math

import pytest

from test_mx4_gpu import Moe, _check_product, _kda, _values, _weights

pytestmark = pytest.mark.gpu


def _codes(values, scale=127):
    """Codes and scales (all of them `scale`) of rows whose values are e2m1 numbers."""
    import torch
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    c = (values.abs()[..., None] == lut).int().argmax(-1).to(torch.uint8) + 8 * (values < 0).to(torch.uint8)
    s = torch.full((*values.shape[:-1], values.shape[-1] // 32), scale, dtype=torch.uint8, device="cuda")
    return c[..., 0::2] | c[..., 1::2] << 4, s


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("m,inter,experts", [(1, 32, 1), (1, 96, 3), (3, 160, 2), (4, 544, 1), (5, 64, 1), (17, 288, 2),
                                             (40, 32, 64), (64, 1056, 3), (64, 256, 200)])
def test_hidden_values_enter_down_in_24_bits(m, inter, experts, shared):
    """Every h is 2^e (2^23 + 2^12 + 1) or that without the 1, exactly (silu(a) = a for such
    a, gates are 1), and every out is the difference of two, times W_down's ones."""
    import torch
    k = 96
    p = Moe(m, k, inter, experts, 1, shared, seed=90)
    p.opts.update(route_scale=1.0)
    # (a device's power function need not be exact for powers of two)
    size = torch.tensor([1, 0.5, 0.25, 0.125, 0.0625], dtype=torch.float64, device="cuda")[torch.arange(m) % 5]
    p.x.zero_()
    p.x[:, 3] = (2.0 ** 23 * size).bfloat16()
    p.x[:, 40] = (2.0 ** 12 * size).bfloat16()
    p.x[:, 41] = size.bfloat16()
    p.x[:, 77] = 1
    p.router[:, :3] = 0  # (nothing of x that counts)
    p.router[:, 3:] = 0
    up = torch.zeros(experts + shared, 2 * inter, k, device="cuda")
    up[:, :inter, 3] = up[:, :inter, 40] = up[:, :inter:2, 41] = 1
    up[:, inter:, 77] = 1
    down = torch.zeros(experts + shared, k, inter, device="cuda")
    row = torch.arange(k, device="cuda")
    i = 2 * (row * 7 % (inter // 2))
    down[:, row, i], down[:, row, (i + 2) % inter + 1] = 1, -1
    (p.w_up, p.s_up), (p.w_down, p.s_down) = _codes(up), _codes(down)
    p.run()
    assert torch.equal(p.gates, torch.ones_like(p.gates))
    want = (size * (1 + shared))[:, None].expand(m, k)
    off = (p.out.double() != want).nonzero().tolist()
    assert not off, [(t, n, p.out[t, n].item(), want[t, n].item()) for t, n in off[:8]]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("m,experts,top", [(1, 16, 3), (6, 16, 5), (3, 200, 32)])
def test_no_bias_is_a_bias_of_zeros(m, experts, top, scoring):
    """Scores that fp64 holds as 1 or as 0 alike: the logits' order, which is that of the
    formula, with a bias of zeros, of any one number, and with none."""
    import torch
    p = Moe(m, 64, 32, experts, top, seed=91)
    p.opts.update(scoring=scoring, renormalise=False)
    p.x[:] = 1
    order = torch.randperm(experts, generator=torch.Generator().manual_seed(92))
    # logits 64 (16 + order): all scores of sigmoid are 1, all of softmax but the first 0
    # (by 64 a step: 745 and more below the largest after 12)
    p.router[:] = (16.0 + order)[:, None].cuda().bfloat16()
    want = order.argsort(descending=True)[:top].int().cuda().expand(m, -1)
    for bias in (None, torch.zeros(experts, device="cuda"), torch.full((experts,), 0.75, device="cuda")):
        p.bias = bias
        p.ids.fill_(-7)
        p.run()
        assert torch.equal(p.ids, want), bias


@pytest.mark.parametrize("m,experts", [(1, 12), (5, 12), (2, 100)])
def test_no_nan_is_taken_before_a_masked_expert(m, experts):
    """A score of NaN comes behind every number, minus infinity among them; those in the
    order of their indices."""
    import torch
    p = Moe(m, 64, 32, experts, 6, bias=True, seed=93)
    p.opts.update(renormalise=False)
    p.router[0] = p.router[2] = math.nan
    p.bias[3:] = -math.inf
    p.run()
    want = torch.tensor([1, 3, 4, 5, 6, 7], dtype=torch.int32, device="cuda").expand(m, -1)
    assert torch.equal(p.ids, want) and torch.isfinite(p.gates).all()
    # as many as are not NaN, and one that is
    q = Moe(m, 64, 32, 4, 3, bias=True, seed=94)
    q.router[0] = q.router[2] = math.nan
    q.bias[3] = -math.inf
    q.run()
    assert torch.equal(q.ids, torch.tensor([1, 3, 0], dtype=torch.int32, device="cuda").expand(m, -1))


@pytest.mark.parametrize("zeros", [False, True])
def test_no_nan_is_taken_before_a_score_of_zero(zeros):
    """A logit of minus infinity is a score of 0, and a number."""
    import torch
    p = Moe(3, 64, 32, 10, 4, seed=95)
    p.opts.update(renormalise=False)
    p.x[1] = p.x[1].abs()
    p.x[1, 9] = math.inf
    p.router[:, 9] = -1
    p.router[:5:2, 9] = 0  # infinity times 0
    p.bias = torch.zeros(10, device="cuda") if zeros else None
    p.run()
    assert torch.equal(p.ids[1].cpu(), torch.tensor([1, 3, 5, 6], dtype=torch.int32)) and (p.gates[1] == 0).all()
    live = [0, 2]
    assert torch.equal(p.ids[live].long(), p.choice()[0][live])


def test_infinite_biases():
    """Sums that are infinite are equal: the lowest index, whatever the logits."""
    import torch
    p = Moe(4, 64, 32, 70, 8, bias=True, seed=96)
    p.opts.update(renormalise=False)
    p.bias[5:] = -math.inf
    p.bias[[3, 1]] = math.inf
    p.run()
    assert torch.equal(p.ids[:, :2].cpu(), torch.tensor([1, 3], dtype=torch.int32).expand(4, -1))
    assert torch.equal(p.ids[:, 5:].cpu(), torch.tensor([5, 6, 7], dtype=torch.int32).expand(4, -1))
    p.check("infinite biases")


def test_experts_beyond_4_gib():
    """Rows of W_up and W_down whose offsets pass 32 bits: the experts behind them, and some in
    front."""
    import torch
    p = Moe(5, 4096, 4096, 620, 4, 2, True, seed=97)
    assert p.w_down.numel() > 1 << 32 and p.w_up.numel() > 1 << 33 and p.s_up.numel() > 1 << 29
    p.bias[:] = -1
    p.bias[[0, 250, 300, 515, 619]] = torch.tensor([1.0, 1.1, 1.2, 1.3, 1.4], device="cuda")
    p.run().check("large experts")
    assert (p.ids >= 512).any() and (p.ids < 512).any()
    q = Moe(40, 4096, 4096, 620, 4, 2, True, seed=97)
    q.bias[:] = -1
    q.bias[610:] = 0
    q.run().check("large experts, many tokens")
    assert (q.ids >= 610).all()


# (64 x 64, 128 x 128 and 256 x 256 tiles on 256 compute units, the scales as they lie and turned)
@pytest.mark.parametrize("m,k,n", [(300, 512, 2051), (300, 544, 2053), (300, 1024, 8195), (300, 1056, 8198),
                                   (1100, 256, 8197), (1100, 288, 8201), (70, 128, 16007)])
def test_rows_of_y_in_whole_pieces(m, k, n):
    """y_row a multiple of 8 and n none: 16-byte stores and single ones in a row; what is behind
    n, and behind the last row, stays."""
    import torch
    x, xs = _weights((m,), k, m + k, spread=3)
    w, ws = _weights((n,), k, n)
    row = (n + 15) // 8 * 8
    y = torch.full((m + 2, row), 3.0, dtype=torch.bfloat16, device="cuda")
    _kda().kda_mx4_proj(x, xs, w, ws, y[:m, :n])
    _check_product(_values(x, xs), w, ws, y[:m, :n], f"pieces {m}x{k}x{n}")
    assert (y[m:] == 3).all() and (y[:, n:] == 3).all()


@pytest.mark.parametrize("m,k,n", [(300, 512, 2100), (300, 1024, 8200), (1100, 512, 8200), (70, 128, 16000)])
def test_rows_of_whole_stages_do_not_mix(m, k, n):
    """A NaN scale of a token and of a weight row stay in their row and column where k is whole
    stages and scales lie at whole words: first, last and middle blocks."""
    import torch
    x, xs = _weights((m,), k, 60)
    w, ws = _weights((n,), k, 61)
    y, z = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _kda().kda_mx4_proj(x, xs, w, ws, y)
    for tokens, rows, block in ([0, m - 1], [5, n - 1], 0), ([63, 64], [64, n - 2], k // 32 - 1), ([17], [n // 2], k // 64):
        xn, wn = xs.clone(), ws.clone()
        xn[tokens, block] = wn[rows, block] = 255
        _kda().kda_mx4_proj(x, xn, w, wn, z)
        hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        hit[tokens] = hit[:, rows] = True
        assert z[hit].isnan().all() and torch.equal(z[~hit], y[~hit])
