"""Host-side tests of include/kda_mx4.h (no GPU needed): every call fails its
argument checks before the library makes any HIP call.  Fake pointers are only
passed together with an argument that is invalid."""
from __future__ import annotations

import os
import re

import pytest

import gated_delta_rule_tok_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, WS_SMALL = 0, 1, 3
FAKE = 0x1000


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda_mx4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kda_[a-z_0-9]+)\s*\(", text))
    assert names == {"kda_mx4_quant", "kda_mx4_dequant", "kda_mx4_proj", "kda_mx4_moe_workspace_size", "kda_mx4_moe"}
    lib = kda.load_library()
    for n in names:
        assert hasattr(lib, n) and n in kda.__all__


def _rows(name, **over):
    first, last = ("x", "s") if name == "kda_mx4_quant" else ("c", "x")
    a = dict(x=FAKE, c=FAKE, s=FAKE) if first == "x" else dict(c=FAKE, s=FAKE, x=FAKE)
    a.update(stream=None, rows=4, k=96, row=96)
    a.update(over)
    return getattr(kda.load_library(), name)(*a.values())


@pytest.mark.parametrize("name", ["kda_mx4_quant", "kda_mx4_dequant"])
@pytest.mark.parametrize("over", [
    {"x": None}, {"c": None}, {"s": None}, {"x": FAKE + 8}, {"c": FAKE + 2}, {"rows": -1}, {"rows": 1 << 31},
    {"k": 0}, {"k": -32}, {"k": 48}, {"k": 1 << 21}, {"row": 88}, {"row": 100}, {"row": 1 << 31},
    {"rows": 1 << 30, "k": 1 << 20, "row": 1 << 20},
], ids=str)
def test_rows_refusals(name, over):
    assert _rows(name, **over) == INVALID


@pytest.mark.parametrize("name", ["kda_mx4_quant", "kda_mx4_dequant"])
def test_rows_of_nothing(name):
    assert _rows(name, rows=0, x=None, c=None, s=None) == OK


def _proj(**over):
    a = dict(x=FAKE, xs=None, w=FAKE, ws=FAKE, y=FAKE, stream=None, m=3, k=256, n=40, x_row=256, y_row=40)
    a.update(over)
    return kda.load_library().kda_mx4_proj(*a.values())


@pytest.mark.parametrize("over", [
    {"x": None}, {"w": None}, {"ws": None}, {"y": None}, {"x": FAKE + 8}, {"w": FAKE + 8}, {"y": FAKE + 1},
    {"m": -1}, {"m": 65}, {"m": 1 << 31, "xs": FAKE}, {"k": 0}, {"k": 40}, {"k": 1 << 21}, {"n": 0},
    {"n": (1 << 24) + 1}, {"x_row": 248}, {"x_row": 260}, {"x_row": 1 << 25}, {"y_row": 39}, {"y_row": 1 << 31},
    {"xs": FAKE, "x": FAKE + 4}, {"xs": FAKE, "m": (1 << 31) - 1, "n": 257, "y_row": 257},
], ids=str)
def test_proj_refusals(over):
    assert _proj(**over) == INVALID


def test_proj_of_nothing():
    assert _proj(m=0, x=None, y=None) == OK and _proj(m=0, xs=FAKE, x=None, y=None) == OK


def _moe(**over):
    a = dict(x=FAKE, router=FAKE, bias=None, w_up=FAKE, s_up=FAKE, w_down=FAKE, s_down=FAKE, idx=None, out=FAKE,
             ids=FAKE, gates=FAKE, ws=FAKE, stream=None, m=3, k=96, inter=64, experts=8, shared=1, top=2, x_row=96,
             out_row=96, scoring=0, renorm=1, scale=1.0, size=1 << 40)
    a.update(over)
    return kda.load_library().kda_mx4_moe(*a.values())


@pytest.mark.parametrize("over", [
    *[{x: None} for x in ("x", "router", "w_up", "s_up", "w_down", "s_down", "out", "ids", "gates", "ws")],
    *[{x: FAKE + 8} for x in ("x", "router", "w_up", "w_down", "out", "ws")],
    *[{x: FAKE + 2} for x in ("bias", "idx", "ids", "gates")],
    {"m": -1}, {"m": 65}, {"k": 0}, {"k": 80}, {"k": 1 << 17}, {"inter": 0}, {"inter": 48}, {"inter": 1 << 17},
    {"experts": 0}, {"experts": 1025}, {"shared": -1}, {"shared": 17}, {"top": 0}, {"top": 9},
    {"experts": 64, "top": 33}, {"x_row": 88}, {"x_row": 100}, {"x_row": 1 << 25}, {"out_row": 88}, {"out_row": 98},
    {"scoring": 2}, {"scoring": -1}, {"scale": float("nan")}, {"scale": float("inf")},
], ids=str)
def test_moe_refusals(over):
    assert _moe(**over) == INVALID


def test_moe_workspace():
    f = kda.kda_mx4_moe_workspace_size
    need = f(3, 96, 64, 8, 1, 2)
    assert need > 0 and need % 256 == 0 and _moe(size=need - 1) == WS_SMALL
    assert f(65, 96, 64, 8, 1, 2) == 0 and f(3, 90, 64, 8, 1, 2) == 0 and f(3, 96, 64, 8, 1, 9) == 0
    for m in range(64):
        assert f(m + 1, 96, 64, 8, 1, 2) >= f(m, 96, 64, 8, 1, 2)
    assert _moe(m=0, x=None, out=None, ids=None, gates=None, size=f(0, 96, 64, 8, 1, 2)) == OK


def test_binding_rejects_what_does_not_fit():
    import torch
    bf, u8 = torch.bfloat16, torch.uint8
    x, c, s = torch.zeros(2, 64, dtype=bf), torch.zeros(2, 32, dtype=u8), torch.zeros(2, 2, dtype=u8)
    with pytest.raises(ValueError):
        kda.kda_mx4_quant(x, c, s)
    with pytest.raises(ValueError):
        kda.kda_mx4_dequant(c, s, x)
    with pytest.raises(ValueError):
        kda.kda_mx4_proj(x, None, c, s, x)
    with pytest.raises(TypeError):
        kda.kda_mx4_proj(None, None, c, s, x)
    with pytest.raises(TypeError):
        kda.kda_mx4_moe(None, None, None, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        kda.kda_mx4_moe(x, x, None, c, s, c, s, x, s, s, s)
