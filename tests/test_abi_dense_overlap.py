"""Outputs that overlap inputs, the workspace or one another are refused by the
norm, the dense products, their backward passes and the pre-norm layer, before
any CUDA call.

The addresses are made up, so this runs only where a call that is not refused
cannot launch anything.
"""
import ctypes

import pytest
import torch

from group_limited_routed_moe_b200 import moe

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

L = moe.lib
T, H, I, N, K = 6, 64, 72, 40, 48
BF16, SAME, INT8 = 0, 0, 1


def _sizes(op):
    """Of an entry point's memory: bytes by name, in the order of its arguments."""
    row, up = T * H * 2, H * I * 2
    return {
        "norm": {"x": row, "residual": row, "weight": H * 2, "stream_out": row, "out": row},
        "norm8": {"x": row, "residual": row, "weight": H * 2, "stream_out": row, "out": T * H, "scales": T * 4},
        "norm_bwd": {"dy": row, "s": row, "weight": H * 2, "dstream": row, "dx": row, "dweight": H * 4,
                     "workspace": L.moe_add_rmsnorm_backward_workspace_bytes(T, H)},
        "int8": {"a": T * K, "a_scale": T * 4, "b": N * K, "b_scale": N * 4, "bias": N * 4, "out": T * N * 2},
        "ffn": {"x": row, "w_gate": up, "w_up": up, "w_down": up, "residual": row, "h": T * I * 2,
                "saved": L.moe_gated_ffn_saved_bytes(T, I), "y": row},
        "ffn_bwd": {"dy": row, "x": row, "w_gate": up, "w_up": up, "w_down": up, "h": T * I * 2,
                    "saved": L.moe_gated_ffn_saved_bytes(T, I), "dx": row, "dw_gate": up, "dw_up": up, "dw_down": up,
                    "workspace": L.moe_gated_ffn_backward_workspace_bytes(T, I)},
        "layer": {"x": T * moe.HIDDEN * 2, "residual": T * moe.HIDDEN * 2, "norm_weight": moe.HIDDEN * 2,
                  "router": L.moe_router_packed_bytes(), "bias": moe.N_EXPERTS * 4,
                  "packed": L.moe_packed_weight_bytes(), "stream_out": T * moe.HIDDEN * 2, "out": T * moe.HIDDEN * 2,
                  "topk_idx": T * moe.TOPK * 4, "topk_w": T * moe.TOPK * 4,
                  "workspace": L.moe_layer_normed_workspace_bytes(T)},
    }[op]


def _align(op, name):
    return {"router": 128, "packed": 128, "workspace": 1024}.get(name, 16) if op == "layer" else 16


OUTPUTS = {"norm": ["stream_out", "out"], "norm8": ["stream_out", "out", "scales"],
           "norm_bwd": ["dx", "dweight", "workspace"], "int8": ["out"], "ffn": ["h", "saved", "y"],
           "ffn_bwd": ["dx", "dw_gate", "dw_up", "dw_down", "workspace"],
           "layer": ["stream_out", "out", "topk_idx", "topk_w", "workspace"]}
# an output that may be this input itself (and not a part of it)
IN_PLACE = {("norm", "stream_out", "x"), ("norm", "stream_out", "residual"), ("norm", "out", "x"),
            ("norm", "out", "residual"), ("norm8", "stream_out", "x"), ("norm8", "stream_out", "residual"),
            ("ffn", "y", "x"), ("ffn", "y", "residual"), ("layer", "stream_out", "x"),
            ("layer", "stream_out", "residual"), ("layer", "out", "x"), ("layer", "out", "residual"),
            ("layer", "out", "stream_out"), ("layer", "stream_out", "out")}


def _call(op, at):
    p = {k: ctypes.c_void_p(v) for k, v in at.items()}
    size = _sizes(op)
    if op in ("norm", "norm8"):
        return L.moe_add_rmsnorm(p["x"], p["residual"], p["weight"], 1e-6, T, H, BF16, p["stream_out"],
                                 SAME if op == "norm" else INT8, 0, p["out"], p.get("scales"), None)
    if op == "norm_bwd":
        return L.moe_add_rmsnorm_backward(p["dy"], p["s"], p["weight"], 1e-6, T, H, BF16, p["dstream"], p["dx"],
                                          p["dweight"], p["workspace"], size["workspace"], None)
    if op == "int8":
        return L.moe_int8_matmul(p["a"], p["a_scale"], p["b"], p["b_scale"], p["bias"], T, N, K, BF16, p["out"], None)
    if op == "ffn":
        return L.moe_gated_ffn(p["x"], p["w_gate"], p["w_up"], p["w_down"], T, H, I, BF16, p["residual"], p["h"],
                               p["saved"], p["y"], None)
    if op == "layer":
        return L.moe_layer_normed(p["x"], p["residual"], p["norm_weight"], 1e-6, p["router"], p["bias"], p["packed"], T,
                                  p["stream_out"], p["out"], p["topk_idx"], p["topk_w"], p["workspace"],
                                  size["workspace"], None)
    return L.moe_gated_ffn_backward(p["dy"], p["x"], p["w_gate"], p["w_up"], p["w_down"], p["h"], p["saved"], T, H, I,
                                    BF16, p["dx"], p["dw_gate"], p["dw_up"], p["dw_down"], p["workspace"],
                                    size["workspace"], None)


def _apart(op):
    """Addresses one behind the other."""
    at, a = {}, 1 << 20
    for name, n in _sizes(op).items():
        a += -a % _align(op, name)
        at[name] = a
        a += -(-n // 16) * 16
    return at


PAIRS = [(op, o, other) for op in OUTPUTS for o in OUTPUTS[op] for other in _sizes(op) if other != o]


@pytest.mark.parametrize("op,out,other", PAIRS)
def test_overlaps_are_refused(op, out, other):
    size = _sizes(op)
    step = max(_align(op, out), 16)
    last = size[other] - 1 - (size[other] - 1) % step  # aligned, and still inside the other
    for move in ({last} if last else set()) | ({0} if (op, out, other) not in IN_PLACE else set()):
        # nothing else may be what is refused
        at = {name: (i + 1) << 32 for i, name in enumerate(size)}
        at[out] = at[other] + move
        assert _call(op, at) == moe.MOE_ERR_INVALID_ARG, f"{out} at {other} + {move}"
        assert "overlap" in moe.last_error()


@pytest.mark.parametrize("op", OUTPUTS)
def test_memory_side_by_side_and_in_place_is_not(op):
    """These calls go on to look for a device, of which there is none here."""
    assert _call(op, _apart(op)) not in (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG)
    for _, out, other in (c for c in IN_PLACE if c[0] == op):
        at = _apart(op)
        at[out] = at[other]
        assert _call(op, at) not in (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG), f"{out} = {other}"


def test_stream_and_output_in_the_same_place():
    at = _apart("norm")
    at["stream_out"] = at["out"] = at["x"]
    assert _call("norm", at) == moe.MOE_ERR_INVALID_ARG
