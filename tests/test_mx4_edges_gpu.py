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
