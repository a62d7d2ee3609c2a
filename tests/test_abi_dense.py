"""Sizes and refusals of the norm, the int8 product, the gated block and the
pre-norm layer, on the host before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from group_limited_routed_moe_b200 import moe

L = moe.lib
BAD, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE, moe.MOE_OK
BF16, F16, F32 = 0, 1, 2
SAME, INT8, E4M3 = 0, 1, 2


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _norm(x=256, res=None, w=256, eps=1e-6, T=4, H=64, dt=BF16, s=None, fmt=SAME, group=0, out=256, sc=None):
    return L.moe_add_rmsnorm(_p(x), _p(res), _p(w), eps, T, H, dt, _p(s), fmt, group, _p(out), _p(sc), None)


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"T": (1 << 22) + 1}, {"H": 0}, {"H": -8}, {"H": 32769}, {"dt": F32}, {"dt": 7}, {"fmt": 3},
    {"fmt": -1}, {"group": 128}, {"fmt": INT8, "group": 64, "sc": 256}, {"eps": -1.0}, {"eps": float("nan")},
    {"eps": float("inf")}, {"x": None}, {"out": None}, {"res": 256}, {"fmt": INT8}, {"fmt": E4M3},
    {"x": 264}, {"w": 264}, {"out": 8}, {"res": 264, "s": 256}, {"res": 256, "s": 264},
    {"fmt": INT8, "sc": 264},
])
def test_norm_refusals(kw):
    assert _norm(**kw) == BAD
    assert moe.last_error()


def test_norm_no_tokens():
    assert _norm(T=0, x=None, out=None, w=None) == OK


def _norm_bwd(dy=256, s=256, w=256, eps=1e-6, T=4, H=64, dt=BF16, ds=None, dx=256, dw=256, ws=256, n=1 << 30):
    return L.moe_add_rmsnorm_backward(_p(dy), _p(s), _p(w), eps, T, H, dt, _p(ds), _p(dx), _p(dw), _p(ws), n, None)


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"H": 0}, {"H": 32769}, {"dt": F32}, {"eps": -1.0}, {"dy": None}, {"s": None}, {"dx": None},
    {"dy": 264}, {"s": 8}, {"w": 8}, {"ds": 8}, {"dx": 8}, {"dw": 8}, {"ws": 8},
])
def test_norm_backward_refusals(kw):
    assert _norm_bwd(**kw) == BAD


def test_norm_backward_workspace():
    need = L.moe_add_rmsnorm_backward_workspace_bytes
    assert need(4, 64) == 4 * 64 * 4
    assert need(0, 64) == 0 and need(-1, 64) == 0 and need(4, 0) == 0 and need(4, 32769) == 0
    assert need(1 << 22, 64) == need(1 << 20, 64) < 4096 * 64 * 4  # rows of partial sums: bounded
    assert _norm_bwd(n=need(4, 64) - 1) == WS
    assert _norm_bwd(ws=None) == WS
    assert _norm_bwd(T=0, dw=None, dy=None, s=None, dx=None, ws=None) == OK


def _int8(a=256, sa=256, b=256, sb=256, bias=None, T=4, N=64, K=64, dt=BF16, out=256):
    return L.moe_int8_matmul(_p(a), _p(sa), _p(b), _p(sb), _p(bias), T, N, K, dt, _p(out), None)


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"T": (1 << 22) + 1}, {"N": 0}, {"N": (1 << 20) + 1}, {"K": 0}, {"K": 8}, {"K": 24}, {"K": 131072},
    {"dt": 3}, {"a": None}, {"sa": None}, {"b": None}, {"sb": None}, {"out": None}, {"a": 8}, {"sa": 8}, {"b": 8},
    {"sb": 8}, {"bias": 8}, {"out": 8},
])
def test_int8_refusals(kw):
    assert _int8(**kw) == BAD


def test_int8_no_tokens():
    assert _int8(T=0, a=None, sa=None, out=None) == OK


def _ffn(x=256, wg=256, wu=256, wd=256, T=4, H=64, I=64, dt=BF16, res=None, h=256, saved=None, y=256):
    return L.moe_gated_ffn(_p(x), _p(wg), _p(wu), _p(wd), T, H, I, dt, _p(res), _p(h), _p(saved), _p(y), None)


SIZES = [{"T": -1}, {"T": (1 << 22) + 1}, {"H": 0}, {"H": 12}, {"H": 65544}, {"I": 0}, {"I": 4}, {"I": 65544},
         {"dt": F32}, {"dt": -1}]


@pytest.mark.parametrize("kw", SIZES + [
    {"x": None}, {"wg": None}, {"wu": None}, {"wd": None}, {"h": None}, {"y": None}, {"x": 8}, {"wg": 8}, {"wu": 8},
    {"wd": 8}, {"res": 8}, {"h": 8}, {"saved": 8}, {"y": 8},
])
def test_ffn_refusals(kw):
    assert _ffn(**kw) == BAD


def _ffn_bwd(dy=256, x=256, wg=256, wu=256, wd=256, h=256, saved=256, T=4, H=64, I=64, dt=BF16, dx=256, dwg=256,
             dwu=256, dwd=256, ws=256, n=1 << 30):
    return L.moe_gated_ffn_backward(_p(dy), _p(x), _p(wg), _p(wu), _p(wd), _p(h), _p(saved), T, H, I, dt, _p(dx),
                                    _p(dwg), _p(dwu), _p(dwd), _p(ws), n, None)


@pytest.mark.parametrize("kw", SIZES + [
    {"dy": None}, {"x": None}, {"wg": None}, {"wu": None}, {"wd": None}, {"h": None}, {"saved": None},
    {"dy": 8}, {"x": 8}, {"wg": 8}, {"wu": 8}, {"wd": 8}, {"h": 8}, {"saved": 8}, {"dx": 8}, {"dwg": 8}, {"dwu": 8},
    {"dwd": 8}, {"ws": 8},
    # what a wanted output needs
    {"dx": None, "dwg": None, "x": None}, {"dwg": None, "dwu": None, "wg": None}, {"dx": None, "saved": None},
    {"dx": None, "dwg": None, "dwu": None, "h": None},
])
def test_ffn_backward_refusals(kw):
    assert _ffn_bwd(**kw) == BAD


def test_ffn_sizes_and_workspace():
    assert L.moe_gated_ffn_saved_bytes(5, 72) == 32 * 96 * 6 and L.moe_gated_ffn_saved_bytes(64, 64) == 64 * 64 * 6
    assert L.moe_gated_ffn_backward_workspace_bytes(5, 64) == 5 * 64 * 4
    for f in (L.moe_gated_ffn_saved_bytes, L.moe_gated_ffn_backward_workspace_bytes):
        assert f(-1, 64) == 0 and f(5, -8) == 0 and f(5, 65544) == 0 and f((1 << 22) + 1, 64) == 0
        assert f(1 << 22, 65536) >= 1 << 40  # no 32-bit product
    assert _ffn_bwd(n=4 * 64 * 4 - 1) == WS
    assert _ffn_bwd(ws=None) == WS
    assert _ffn(T=0, x=None, h=None, y=None) == OK


def _layer(x=1024, res=None, w=1024, eps=1e-6, router=1024, bias=None, packed=1024, T=16, s=None, out=1024, ws=1024,
           n=1 << 40):
    return L.moe_layer_normed(_p(x), _p(res), _p(w), eps, _p(router), _p(bias), _p(packed), T, _p(s), _p(out), None,
                              None, _p(ws), n, None)


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"x": None}, {"router": None}, {"packed": None}, {"out": None}, {"ws": None}, {"res": 1024},
    {"ws": 1040}, {"packed": 1040}, {"router": 1040}, {"out": 1032}, {"x": 1032}, {"bias": 1032}, {"eps": -1.0},
])
def test_layer_normed_refusals(kw):
    assert _layer(**kw) == BAD


def test_layer_normed_workspace():
    need = moe.layer_normed_workspace_bytes(16)
    assert need >= moe.layer_workspace_bytes(16) + 16 * 1536 * 2 and need % 1024 == 0
    assert L.moe_layer_normed_workspace_bytes(-1) == 0
    assert _layer(n=need - 1) == WS
    assert _layer(T=0, x=None, out=None, ws=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    q, sc = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    for call in (lambda: moe.moe_add_rmsnorm(x), lambda: moe.moe_add_rmsnorm_backward(x, x),
                 lambda: moe.moe_int8_matmul(q, sc, q, sc), lambda: moe.moe_gated_ffn(x, w, w, w),
                 lambda: moe.moe_gated_ffn_backward(x, x, w, w, w, x),
                 lambda: moe.moe_layer_normed(x, None, None, 1e-6, w, None, w)):
        with pytest.raises(ValueError):
            call()
