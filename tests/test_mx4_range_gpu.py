"""Products with microscaled 4-bit weights over the whole range of scales: what fp32
holds is exact, what passes it infinite, and what is below its least normal number
off by less than that."""
from __future__ import annotations

import math

import pytest

from test_mx4_gpu import _kda, _weights

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126


def _one(rows, k, at, code):
    """Codes of rows that hold one element `code` at `at`, zeros else."""
    import torch
    c = torch.zeros(rows, k // 2, dtype=torch.uint8, device="cuda")
    c[:, at // 2] = code << (4 * (at & 1))
    return c


def _power(e):
    """2^e, fp64 (from the bits: a device's power function need not be exact)."""
    import torch
    return ((e.long() + 1023) << 52).view(torch.float64)


def _check(y, want, label):
    import torch
    y = y.double()
    large, small = want.abs() >= 2.0 ** 128, want.abs() < LEAST
    assert torch.equal(y[large], torch.copysign(torch.full_like(y[large], math.inf), want[large])), label
    assert torch.equal(y[~large & ~small], want[~large & ~small]), label
    assert ((y - want).abs()[small] <= LEAST).all(), label
    return large.any() and small.any()


@pytest.mark.parametrize("code,value", [(2, 1.0), (7, 6.0), (1, 0.5), (10, -1.0)])
@pytest.mark.parametrize("k,at", [(32, 0), (96, 37), (128, 127), (544, 543)])
def test_every_pair_of_scales(k, at, code, value):
    """One product a sum, 255 scales of x by 255 of w: calls of few rows, and in tiles of all
    three sides."""
    import torch
    s = torch.arange(255, device="cuda")
    ws = s.to(torch.uint8)[:, None].repeat(1, k // 32)
    w = _one(255, k, at, code)
    for m, times in ((16, 1), (255, 1), (255, 33), (510, 33), (2040, 40)):
        x, xs = _one(m, k, at, 7), (torch.arange(m, device="cuda") % 255).to(torch.uint8)[:, None].repeat(1, k // 32)
        if m == 16:
            xs += 230
        y = torch.full((m, 255 * times), math.nan, dtype=torch.bfloat16, device="cuda")
        _kda().kda_mx4_proj(x, xs, w.repeat(times, 1), ws.repeat(times, 1), y)
        e = xs[:, :1].int() + s.repeat(times)[None] - 254
        both = _check(y, 6 * value * _power(e), f"{m} x {255 * times}")
        assert both or m == 16  # (few rows: scales from 230 on)


@pytest.mark.parametrize("m", [1, 4, 16, 64])
@pytest.mark.parametrize("k,at", [(32, 31), (544, 300)])
def test_bf16_rows_of_every_scale(k, at, m):
    import torch
    s = torch.arange(253, device="cuda")  # (bf16 holds these weights)
    w, ws = _one(253, k, at, 7), s.to(torch.uint8)[:, None].repeat(1, k // 32)
    for first in (-126, -60, 0, 64):
        e = first + torch.arange(m, device="cuda").clamp(max=63)
        x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
        x[:, at] = _power(e).bfloat16()
        y = torch.full((m, 253), math.nan, dtype=torch.bfloat16, device="cuda")
        _kda().kda_mx4_proj(x, None, w, ws, y)
        want = 6 * _power(e[:, None] + s[None] - 127)
        big = want >= 2.0 ** 128
        assert torch.isinf(y[big]).all() and torch.equal(y.double()[~big & (want >= LEAST)], want[~big & (want >= LEAST)])
        assert ((y.double() - want).abs()[want < LEAST] <= LEAST).all()


def test_what_is_lost_or_infinite_stays_in_its_row():
    import torch
    k, m, n = 544, 70, 9000
    x, xs = _weights((m,), k, 50)
    w, ws = _weights((n,), k, 51)
    y, z = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _kda().kda_mx4_proj(x, xs, w, ws, y)
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[3], ws2[17] = 254, 254
    xs2[5], ws2[20] = 0, 0
    _kda().kda_mx4_proj(x, xs2, w, ws2, z)
    rows = [r for r in range(m) if r not in (3, 5)]
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[17] = keep[20] = False
    assert torch.equal(z[rows][:, keep], y[rows][:, keep])
    assert not torch.isfinite(z[3, 17]) and abs(z[5, 20].item()) <= LEAST
