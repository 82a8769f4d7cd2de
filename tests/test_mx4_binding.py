"""What the Python binding of include/kda_mx4.h refuses before the library is called, on
the CPU: its tensors' own device takes the place of a GPU and a recorder that of the
call.  The library sees pointers only, so a shape that does not fit has to end here."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_tok_amd as kda

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


@pytest.fixture
def calls(monkeypatch):
    made = []
    kda._torch()
    monkeypatch.setattr(kda, "_gpu", lambda t, name: t.get_device())
    monkeypatch.setattr(kda, "_call", lambda name, fn, index, stream, before, after: made.append((name, before, after)))
    return made


def z(*shape, dtype=U8):
    return torch.zeros(*shape, dtype=dtype)


def _refused(calls, f, args, match, **more):
    with pytest.raises((ValueError, TypeError), match=match):
        f(*args.values(), **more)
    assert not calls


ROWS = {
    "few columns of codes": (dict(codes=z(3, 47)), "codes"), "codes of another row": (dict(codes=z(2, 48)), "codes"),
    "type of codes": (dict(codes=z(3, 48, dtype=torch.int8)), "codes"), "codes not dense": (dict(codes=z(3, 96)[:, :48]), "codes"),
    "few scales": (dict(scales=z(3, 2)), "scales"), "scales of fewer rows": (dict(scales=z(2, 3)), "scales"),
    "type of scales": (dict(scales=z(3, 3, dtype=F32)), "scales"), "no codes": (dict(codes=None), "codes"),
    "columns": (dict(x=z(3, 80, dtype=BF)), "32"), "no columns": (dict(x=z(3, 0, dtype=BF)), "32"),
    "type": (dict(x=z(3, 96, dtype=F32)), "x|out"), "dimensions": (dict(x=z(96, dtype=BF)), "x|out"),
    "columns apart": (dict(x=z(96, 3, dtype=BF).T), "x|out"),
}


@pytest.mark.parametrize("case", ROWS)
def test_quant_and_back(calls, case):
    over, match = ROWS[case]
    a = {**dict(x=z(3, 96, dtype=BF), codes=z(3, 48), scales=z(3, 3)), **over}
    _refused(calls, kda.kda_mx4_quant, a, match)
    _refused(calls, kda.kda_mx4_dequant, dict(codes=a["codes"], scales=a["scales"], out=a["x"]), match)


PROJ = {
    "codes' columns": (dict(x=z(4, 47), xs=z(4, 3)), "x|32"), "columns of x": (dict(x=z(4, 64, dtype=BF)), "w"),
    "odd columns of x": (dict(x=z(4, 90, dtype=BF)), "32"), "type of x": (dict(x=z(4, 96, dtype=torch.float16)), "x"),
    "bf16 as codes": (dict(xs=z(4, 3)), "x|w"), "rows of x's scales": (dict(x=z(4, 48), xs=z(3, 3)), "x_scales"),
    "columns of x's scales": (dict(x=z(4, 48), xs=z(4, 4)), "x_scales"), "columns of w": (dict(w=z(7, 64)), "w"),
    "type of w": (dict(w=z(7, 48, dtype=torch.int8)), "w"), "w not dense": (dict(w=z(7, 96)[:, ::2]), "w"),
    "rows of w's scales": (dict(ws=z(6, 3)), "w_scales"), "columns of w's scales": (dict(ws=z(7, 2)), "w_scales"),
    "rows of y": (dict(y=z(3, 7, dtype=BF)), "y"), "columns of y": (dict(y=z(4, 8, dtype=BF)), "y"),
    "type of y": (dict(y=z(4, 7, dtype=F32)), "y"), "columns of y apart": (dict(y=z(7, 4, dtype=BF).T), "y"),
    "no w": (dict(w=None), "w"), "no y": (dict(y=None), "y"),
}


@pytest.mark.parametrize("case", PROJ)
def test_proj(calls, case):
    over, match = PROJ[case]
    _refused(calls, kda.kda_mx4_proj,
             {**dict(x=z(4, 96, dtype=BF), xs=None, w=z(7, 48), ws=z(7, 3), y=z(4, 7, dtype=BF)), **over}, match)


def _moe():
    return dict(x=z(3, 96, dtype=BF), router=z(5, 96, dtype=BF), bias=z(5, dtype=F32), w_up=z(6, 128, 48),
                s_up=z(6, 128, 3), w_down=z(6, 96, 32), s_down=z(6, 96, 2), out=z(3, 96, dtype=BF),
                ids=z(3, 2, dtype=I32), gates=z(3, 2, dtype=F32), ws=z(1 << 20))


MOE = {
    "columns of x": (dict(x=z(3, 64, dtype=BF)), "router|out"), "odd columns of x": (dict(x=z(3, 100, dtype=BF)), "32"),
    "type of x": (dict(x=z(3, 96, dtype=F32)), "x"), "columns of the router": (dict(router=z(5, 64, dtype=BF)), "router"),
    "type of the router": (dict(router=z(5, 96, dtype=F32)), "router"),
    "more experts than weights": (dict(router=z(7, 96, dtype=BF), bias=None), "w_up"),
    "length of the bias": (dict(bias=z(6, dtype=F32)), "bias"), "type of the bias": (dict(bias=z(5, dtype=BF)), "bias"),
    "odd rows of w_up": (dict(w_up=z(6, 127, 48), s_up=z(6, 127, 3)), "w_up"),
    "inter of 48": (dict(w_up=z(6, 96, 48), s_up=z(6, 96, 3), w_down=z(6, 96, 24), s_down=z(6, 96, 1)), "w_up"),
    "columns of w_up": (dict(w_up=z(6, 128, 47)), "w_up"), "dimensions of w_up": (dict(w_up=z(6, 128 * 48)), "w_up"),
    "type of w_up": (dict(w_up=z(6, 128, 48, dtype=torch.int8)), "w_up"),
    "experts of w_up's scales": (dict(s_up=z(5, 128, 3)), "w_up_scales"),
    "columns of w_up's scales": (dict(s_up=z(6, 128, 2)), "w_up_scales"),
    "experts of w_down": (dict(w_down=z(5, 96, 32)), "w_down"), "rows of w_down": (dict(w_down=z(6, 95, 32)), "w_down"),
    "columns of w_down": (dict(w_down=z(6, 96, 31)), "w_down"),
    "w_down not dense": (dict(w_down=z(6, 96, 64)[..., :32]), "w_down"),
    "columns of w_down's scales": (dict(s_down=z(6, 96, 1)), "w_down_scales"),
    "rows of out": (dict(out=z(2, 96, dtype=BF)), "out"), "type of out": (dict(out=z(3, 96, dtype=F32)), "out"),
    "columns of out apart": (dict(out=z(96, 3, dtype=BF).T), "out"), "rows of the ids": (dict(ids=z(2, 2, dtype=I32)), "expert_ids"),
    "type of the ids": (dict(ids=z(3, 2, dtype=torch.int64)), "expert_ids"),
    "shape of the gates": (dict(gates=z(3, 3, dtype=F32)), "expert_gates"),
    "type of the gates": (dict(gates=z(3, 2, dtype=BF)), "expert_gates"),
    "type of the workspace": (dict(ws=z(1 << 18, dtype=F32)), "workspace"), "no workspace": (dict(ws=None), "workspace"),
    **{f"no {name}": ({name: None}, name) for name in ("router", "w_up")}, "no ids": (dict(ids=None), "expert_ids"),
    "no out": (dict(out=None), "out"), "no w_down": (dict(w_down=None), "w_down"),
}


@pytest.mark.parametrize("case", MOE)
def test_moe(calls, case):
    over, match = MOE[case]
    _refused(calls, kda.kda_mx4_moe, {**_moe(), **over}, match)


@pytest.mark.parametrize("more,match", [(dict(scoring="relu"), "scoring"), (dict(scoring=0), "scoring"),
                                        (dict(state_indices=z(2, dtype=I32)), "state_indices"),
                                        (dict(state_indices=z(3, dtype=torch.int64)), "state_indices")], ids=str)
def test_moe_options(calls, more, match):
    _refused(calls, kda.kda_mx4_moe, _moe(), match, **more)


def test_what_fits_is_passed_on(calls):
    """Each of the calls above without its fault reaches the library, with these numbers."""
    x, c, s = z(3, 96, dtype=BF), z(3, 48), z(3, 3)
    kda.kda_mx4_quant(z(3, 120, dtype=BF)[:, 24:], c, s)
    kda.kda_mx4_dequant(c, s, x)
    kda.kda_mx4_proj(z(4, 96, dtype=BF), None, z(7, 48), z(7, 3), z(4, 9, dtype=BF)[:, :7])
    kda.kda_mx4_proj(z(4, 48), z(4, 3), z(7, 48), z(7, 3), z(4, 7, dtype=BF))
    kda.kda_mx4_moe(*_moe().values(), scoring="softmax", renormalise=False, route_scale=2.5,
                    state_indices=z(3, dtype=I32))
    assert [(name, after) for name, _, after in calls] == [
        ("kda_mx4_quant", (3, 96, 120)), ("kda_mx4_dequant", (3, 96, 96)), ("kda_mx4_proj", (4, 96, 7, 96, 9)),
        ("kda_mx4_proj", (4, 96, 7, 0, 7)), ("kda_mx4_moe", (3, 96, 64, 5, 1, 2, 96, 96, 1, 0, 2.5, 1 << 20))]
