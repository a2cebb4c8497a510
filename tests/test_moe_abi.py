"""The routed expert layer's entry points refuse bad arguments before launching anything (no GPU needed)."""

import ctypes

import pytest
import torch

from expert_ffn_ragged_amd import rd

BIG = 1 << 31
OK, EINVAL, EUNSUPPORTED = rd.RD_OK, rd.RD_EINVAL, rd.RD_EUNSUPPORTED


def _call(name, ok, **kw):
    a = dict(ok)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(rd.library(), name)(*a.values(), None)


ROUTE = dict(logits=16, dtype=1, bias=None, limit=None, weights=16, ids=16, tokens=4, experts=8, top_k=2, score=0,
             groups=1, top_groups=1, renormalize=0, scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), EINVAL), (dict(weights=None), EINVAL), (dict(ids=None), EINVAL), (dict(logits=18), EINVAL),
    (dict(bias=18), EINVAL), (dict(limit=17), EINVAL), (dict(dtype=2), EINVAL), (dict(score=2), EINVAL),
    (dict(tokens=-1), EINVAL), (dict(top_k=0), EINVAL), (dict(top_k=9), EINVAL), (dict(experts=0, top_k=0), EINVAL),
    (dict(experts=2048), EUNSUPPORTED), (dict(experts=64, top_k=17), EUNSUPPORTED), (dict(tokens=BIG), EUNSUPPORTED),
    (dict(groups=3), EINVAL), (dict(groups=0), EINVAL), (dict(groups=4, top_groups=5), EINVAL),
    (dict(groups=4, top_groups=0), EINVAL), (dict(groups=4, top_groups=1, top_k=3), EINVAL),
    (dict(experts=64, groups=32, top_groups=4), EUNSUPPORTED),
    (dict(tokens=0, logits=None, weights=None, ids=None), OK)])
def test_route(kw, status):
    assert _call("rd_route", ROUTE, **kw) == status


BWD = dict(logits=16, dtype=0, ids=16, d_weights=16, d_logits=16, tokens=4, experts=8, top_k=2, score=1, renormalize=1,
           scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), EINVAL), (dict(ids=None), EINVAL), (dict(d_weights=None), EINVAL), (dict(d_logits=None), EINVAL),
    (dict(logits=17), EINVAL), (dict(dtype=1, d_logits=18), EINVAL), (dict(ids=18), EINVAL), (dict(score=-1), EINVAL),
    (dict(top_k=9), EINVAL), (dict(experts=1025), EUNSUPPORTED), (dict(tokens=0, logits=None), OK)])
def test_route_bwd(kw, status):
    assert _call("rd_route_bwd", BWD, **kw) == status


GROUP = dict(ids=16, n=8, experts=4, sizes=16, rows=16, slots=16, total=16, workspace=None, bytes=0)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), EINVAL), (dict(sizes=None), EINVAL), (dict(rows=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(total=None), EINVAL), (dict(n=-1), EINVAL), (dict(experts=0), EINVAL), (dict(experts=1025), EUNSUPPORTED),
    (dict(n=(1 << 30) + 1), EUNSUPPORTED), (dict(slots=18), EINVAL),
    (dict(n=1 << 20), EINVAL),                                   # needs a workspace
    (dict(n=1 << 20, workspace=16, bytes=64), EINVAL)])          # a larger one
def test_group_rows(kw, status):
    assert _call("rd_group_rows", GROUP, **kw) == status


def test_group_rows_workspace():
    assert rd.group_rows_workspace_size(512, 128) == 0
    need = rd.group_rows_workspace_size(225280, 256)
    assert 0 < need < 1 << 20 and need % 4 == 0
    assert rd.group_rows_workspace_size(-1, 4) == 0 and rd.group_rows_workspace_size(1 << 20, 2000) == 0


ROWS = dict(tokens=4, top_k=2, hidden=64, rows=8)
DISPATCH = dict(x=16, slots=16, xs=16, **ROWS)
COMBINE = dict(y=16, slots=16, weights=None, out=16, **ROWS)
COMBINE_BWD = dict(g=16, y=16, slots=16, weights=16, dy=16, dw=16, **ROWS)


@pytest.mark.parametrize("name,ok", [("rd_dispatch_rows", DISPATCH), ("rd_combine_rows", COMBINE),
                                     ("rd_combine_rows_bwd", COMBINE_BWD)])
def test_rows(name, ok):
    assert _call(name, ok, hidden=12) == EUNSUPPORTED
    assert _call(name, ok, hidden=0) == EINVAL
    assert _call(name, ok, top_k=0) == EINVAL
    assert _call(name, ok, top_k=17) == EUNSUPPORTED
    assert _call(name, ok, tokens=-1) == EINVAL
    assert _call(name, ok, rows=-1) == EINVAL
    assert _call(name, ok, rows=BIG) == EUNSUPPORTED
    assert _call(name, ok, tokens=1 << 30) == EUNSUPPORTED       # tokens * top_k past 2^31
    assert _call(name, ok, tokens=1 << 29, top_k=1, hidden=4096) == EUNSUPPORTED
    assert _call(name, ok, tokens=0) == OK
    for arg in ok:
        if arg not in ROWS and not (arg == "weights" and name == "rd_combine_rows"):
            assert _call(name, ok, **{arg: None}) == EINVAL, arg
            assert _call(name, ok, **{arg: 18}) == EINVAL, arg   # misaligned


QUANT = dict(x=16, dtype=0, limit=None, codes=16, scales=1, rows=4, cols=64, bits=4)
DEQUANT = dict(codes=16, scales=1, limit=None, out=16, dtype=0, rows=4, cols=64, bits=8)


@pytest.mark.parametrize("name,ok", [("rd_quantize_mx", QUANT), ("rd_dequantize_mx", DEQUANT)])
def test_quantisation(name, ok):
    assert _call(name, ok, cols=48) == EUNSUPPORTED
    assert _call(name, ok, cols=0) == EINVAL
    assert _call(name, ok, bits=6) == EINVAL
    assert _call(name, ok, dtype=3) == EINVAL
    assert _call(name, ok, rows=-1) == EINVAL
    assert _call(name, ok, rows=1 << 40, cols=1 << 30) == EUNSUPPORTED
    assert _call(name, ok, codes=24) == EINVAL
    assert _call(name, ok, limit=18) == EINVAL
    assert _call(name, ok, scales=None) == EINVAL
    assert _call(name, ok, rows=0, codes=None) == OK


MX = dict(x=16, xs=16, bits=4, w=16, ws=16, gs=16, G=4, off=None, gl=4, limit=None, out=16, dt=0, m=8, k=128, n=8)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), EINVAL), (dict(xs=None), EINVAL), (dict(w=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(gs=None), EINVAL), (dict(out=None), EINVAL), (dict(x=24), EINVAL), (dict(xs=18), EINVAL), (dict(w=24), EINVAL),
    (dict(ws=17), EINVAL), (dict(limit=18), EINVAL), (dict(bits=5), EINVAL), (dict(dt=4), EINVAL), (dict(k=64), EUNSUPPORTED),
    (dict(n=12), EUNSUPPORTED), (dict(n=1 << 20, k=4096), EUNSUPPORTED), (dict(k=1 << 24), EUNSUPPORTED), (dict(gl=3), EINVAL), (dict(gl=5, off=16), EINVAL),
    (dict(G=2000, gl=2000), EUNSUPPORTED), (dict(m=BIG), EUNSUPPORTED), (dict(m=0, x=None, out=None), OK)])
def test_product(kw, status):
    assert _call("rd_forward_mx", MX, **kw) == status


GLU_FWD = dict(fused=16, limit=None, act=16, codes=16, scales=1, rows=4, h=32)
GLU_BWD = dict(codes=16, scales=1, d_act=16, limit=None, weights=None, row_slots=None, d_fused=16, act=16, dot=16, rows=4,
               h=32, slots=4)


def test_glu():
    for name, ok in (("rd_glu_fwd_mx8", GLU_FWD), ("rd_glu_bwd_mx8", GLU_BWD)):
        assert _call(name, ok, h=48) == EUNSUPPORTED
        assert _call(name, ok, h=0) == EINVAL
        assert _call(name, ok, rows=BIG) == (EINVAL if name == "rd_glu_bwd_mx8" else EUNSUPPORTED)
        assert _call(name, ok, codes=None) == EINVAL
        assert _call(name, ok, act=24) == EINVAL
        assert _call(name, ok, limit=18) == EINVAL
        assert _call(name, ok, rows=0, codes=None, scales=None) == OK
    assert _call("rd_glu_bwd_mx8", GLU_BWD, slots=3) == EINVAL               # row r has slot r
    assert _call("rd_glu_bwd_mx8", GLU_BWD, slots=-1, row_slots=16) == EINVAL
    assert _call("rd_glu_bwd_mx8", GLU_BWD, dot=None) == EINVAL
    assert _call("rd_glu_bwd_mx8", GLU_BWD, weights=18) == EINVAL


def test_binding_refuses_what_it_can_see():
    """Types, devices and shapes are checked before the library is asked."""
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        rd.route(x, 2)                                # not on the GPU
    with pytest.raises(TypeError):
        rd.route(x.half(), 2)
    with pytest.raises(TypeError):
        rd.quantize_mx([1.0])
    with pytest.raises(TypeError):
        rd.dequantize_mx(x, x)
    with pytest.raises(ValueError):
        rd.dispatch_rows(x, x)                        # not on the GPU
    with pytest.raises(ValueError):
        rd._score("relu")
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_glu_rows_leave_room_for_the_grids_stride():
    for name, ok, extra in (("rd_glu_fwd_mx8", GLU_FWD, {}), ("rd_glu_bwd_mx8", GLU_BWD, dict(slots=BIG))):
        assert _call(name, ok, rows=BIG - 1, **extra) == EUNSUPPORTED
        assert _call(name, ok, rows=BIG - (1 << 20) + 1, **extra) == EUNSUPPORTED


@pytest.mark.parametrize("name,ok", [("rd_dispatch_rows", DISPATCH), ("rd_combine_rows", COMBINE),
                                     ("rd_combine_rows_bwd", COMBINE_BWD)])
def test_rows_refuses_counts_whose_products_pass_64_bits(name, ok):
    for tokens in (1 << 40, 1 << 60, 1 << 62, (1 << 63) - 1):
        for top_k in (1, 2, 4, 16):
            assert _call(name, ok, tokens=tokens, top_k=top_k, hidden=8) == EUNSUPPORTED
    assert _call(name, ok, tokens=BIG // 16, top_k=16) == EUNSUPPORTED
    assert _call(name, ok, hidden=(1 << 63) - 8) == EUNSUPPORTED
