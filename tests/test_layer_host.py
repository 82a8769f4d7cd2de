"""Host-side tests of include/kda_layer.h (no GPU needed): every call fails its
argument checks before the library makes any HIP call.  Fake pointers are only
passed together with an argument that is invalid."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import gated_delta_rule_tok_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, WS_SMALL = 0, 1, 3
FAKE = 0x1000
F = ctypes.c_float


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda_layer.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kda_[a-z_0-9]+)\s*\(", text))
    assert names == {"kda_gdr_get_workspace_size", "kda_gdr_prefill_fwd", "kda_gdr_decode_step",
                     "kda_add_rms_norm", "kda_w4_proj"}
    lib = kda.load_library()
    for n in names:
        assert hasattr(lib, n) and n in kda.__all__


def _prefill(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, a=FAKE, beta=FAKE, A_log=FAKE, dt_bias=FAKE, scale=0.1, s0=None,
             cu=FAKE, out=FAKE, sT=FAKE, ws=FAKE, stream=None, T=100, hk=2, hv=4, n=2, sdt=0,
             size=1 << 40, strides=None)
    a.update(over)
    return kda.load_library().kda_gdr_prefill_fwd(*a.values())


def _strides(**over):
    s = dict(q_token=256, q_head=128, k_token=256, k_head=128, v_token=512, v_head=128, a_token=4,
             a_head=1, beta_token=4, beta_head=1, out_token=512, out_head=128)
    s.update(over)
    return ctypes.byref(kda._GdrStrides(**s))


@pytest.mark.parametrize("over", [
    *[{x: None} for x in ("q", "k", "v", "a", "beta", "A_log", "dt_bias", "cu", "out", "sT", "ws")],
    *[{x: FAKE + 8} for x in ("q", "k", "v", "out", "s0", "sT", "ws")],
    *[{x: FAKE + 1} for x in ("a", "beta", "A_log", "dt_bias", "cu")],
    {"T": -1}, {"T": 1 << 31}, {"n": 0}, {"n": -3}, {"hk": 0}, {"hv": 0}, {"hk": 3}, {"hk": 8},
    {"hv": 65538}, {"sdt": 2}, {"sdt": -1}, {"scale": float("nan")}, {"scale": float("inf")},
    {"n": 1 << 19}, {"T": 1 << 30},
    *[{"strides": {x: v}} for x in ("q_token", "k_head", "v_token", "out_head") for v in (-8, 4, 1 << 31)],
    {"strides": {"a_token": -1}}, {"strides": {"beta_head": -1}}, {"strides": {"out_token": 0}},
    {"strides": {"out_head": 0}},
], ids=str)
def test_prefill_refusals(over):
    if "strides" in over:
        over = {"strides": _strides(**over["strides"])}
    assert _prefill(**over) == INVALID


def test_prefill_workspace():
    f = kda.kda_gdr_get_workspace_size
    need = f(100, 2, 4, 2)
    assert need > 0 and need % 256 == 0
    assert _prefill(size=need - 1) == WS_SMALL
    assert f(-1, 2, 4, 2) == 0 and f(100, 3, 4, 2) == 0 and f(100, 2, 4, 0) == 0 and f(100, 0, 0, 2) == 0
    for t in (0, 1, 63, 64, 65, 4096):
        assert f(t + 1, 2, 4, 2) >= f(t, 2, 4, 2)
    assert f(100, 2, 8, 2) >= need and f(100, 4, 4, 2) >= need and f(100, 2, 4, 3) >= need


def _decode(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, a=FAKE, beta=FAKE, A_log=FAKE, dt_bias=FAKE, scale=0.1, pool=FAKE,
             slots=9, idx=FAKE, out=FAKE, stream=None, n=3, hk=2, hv=4, sdt=0, strides=None)
    a.update(over)
    return kda.load_library().kda_gdr_decode_step(*a.values())


@pytest.mark.parametrize("over", [
    *[{x: None} for x in ("q", "k", "v", "a", "beta", "A_log", "dt_bias", "pool", "idx", "out")],
    *[{x: FAKE + 8} for x in ("q", "k", "v", "out", "pool")],
    {"idx": FAKE + 2}, {"n": -1}, {"slots": 0}, {"hk": 3}, {"sdt": 7}, {"scale": float("inf")},
    {"n": 1 << 20}, {"strides": {"q_token": 12}}, {"strides": {"out_token": 0}},
], ids=str)
def test_decode_refusals(over):
    if "strides" in over:
        over = {"strides": _strides(**over["strides"])}
    assert _decode(**over) == INVALID


def test_decode_of_nothing():
    assert _decode(n=0, q=None, k=None, v=None, a=None, beta=None, out=None, idx=None) == OK


def _norm(**over):
    a = dict(x=FAKE, res=FAKE, w=FAKE, eps=1e-6, out=FAKE, scale=None, stream=None, rows=4, dim=100,
             x_row=100, r_row=100, o_row=100, odt=0, group=0)
    a.update(over)
    return kda.load_library().kda_add_rms_norm(*a.values())


@pytest.mark.parametrize("over", [
    {"x": None}, {"w": None}, {"out": None}, {"x": FAKE + 1}, {"res": FAKE + 1}, {"w": FAKE + 1},
    {"out": FAKE + 1}, {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}, {"rows": -1},
    {"rows": 1 << 31}, {"dim": 0}, {"dim": 32769}, {"x_row": 99}, {"r_row": 99}, {"o_row": 99},
    {"x_row": 1 << 31}, {"odt": 2}, {"group": 128}, {"scale": FAKE}, {"odt": 1},
    {"odt": 1, "scale": FAKE, "group": 64}, {"odt": 1, "scale": FAKE + 2}, {"odt": 1, "scale": FAKE, "group": -1},
], ids=str)
def test_norm_refusals(over):
    assert _norm(**over) == INVALID


def test_norm_of_nothing():
    assert _norm(rows=0, x=None, res=None, out=None) == OK


def _w4(**over):
    a = dict(x=FAKE, w=FAKE, s=FAKE, z=None, y=FAKE, stream=None, m=3, k=256, n=40, group=64, x_row=256,
             y_row=40)
    a.update(over)
    return kda.load_library().kda_w4_proj(*a.values())


@pytest.mark.parametrize("over", [
    {"x": None}, {"w": None}, {"s": None}, {"y": None}, {"x": FAKE + 8}, {"w": FAKE + 8}, {"s": FAKE + 1},
    {"z": FAKE + 1}, {"y": FAKE + 1}, {"m": -1}, {"m": 65}, {"k": 0}, {"k": 96}, {"k": 1 << 21}, {"n": 0},
    {"n": (1 << 24) + 1}, {"group": 16}, {"group": 0}, {"group": 256}, {"x_row": 248}, {"x_row": 260},
    {"y_row": 39}, {"x_row": 1 << 31}, {"y_row": 1 << 31},
], ids=str)
def test_w4_refusals(over):
    assert _w4(**over) == INVALID


def test_w4_of_nothing():
    assert _w4(m=0, x=None, y=None) == OK


def test_binding_rejects_host_tensors():
    import torch
    bf = torch.bfloat16
    t, h = torch.zeros(4, 2, 128, dtype=bf), torch.zeros(4, 2, dtype=bf)
    p = torch.zeros(2)
    s = torch.zeros(1, 2, 128, 128)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_gdr_prefill_fwd(t, t, t, h, h, p, p, 1.0, None, cu, t, s, None)
    with pytest.raises(ValueError):
        kda.kda_gdr_decode_step(t, t, t, h, h, p, p, 1.0, s, cu, t)
    x = torch.zeros(2, 64, dtype=bf)
    with pytest.raises(ValueError):
        kda.kda_add_rms_norm(x, None, x[0], 1e-6, x)
    with pytest.raises(ValueError):
        kda.kda_w4_proj(x, torch.zeros(3, 32, dtype=torch.uint8), x, None, x, 32)
    with pytest.raises(TypeError):
        kda.kda_add_rms_norm(None, None, None, 1e-6, None)


def test_stream_and_device_queries():
    """The short forms where torch has them, the public calls where it does not."""
    from types import SimpleNamespace as N
    raw, device = kda._queries(N(_C=N(_cuda_getCurrentRawStream="r", _cuda_getDevice="d"), cuda=N()))
    assert raw == "r" and device == "d"
    cuda = N(current_stream=lambda i: N(cuda_stream=100 + i), current_device=lambda: 3)
    raw, device = kda._queries(N(_C=N(), cuda=cuda))
    assert raw(2) == 102 and device() == 3
