"""The experts' layer (include/kda_mx4.h) where it can go wrong without any result
looking odd: inputs whose exact answer is a small whole number or an order."""
from __future__ import annotations

import math

import pytest

from test_mx4_gpu import Moe

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
