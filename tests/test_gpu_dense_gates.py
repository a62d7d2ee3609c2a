"""silu and its derivative in the gated block over gates from -100 to 100,
through the buffers that hold h, dg and du.

With rows that are one in their first element and zero elsewhere, a gate is the
weight itself, exactly, and so are u and dh.  What is left: the sigmoid's
relative error e(g) = 2^-21 + 1.25 |g| 2^-24 (approximate exponential and
reciprocal; the rounded exponent), at most four fp32 products (2^-22), the
rounding to 16 bits, sigmoids below 2^-126 flushed to zero, and in the backward
pass the gate cut at 2^-15 of itself, times the next derivative.
"""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe

pytestmark = pytest.mark.gpu

H, I = 8, 2048
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,kernel", [(5, "few"), (20, "few"), (100, "few"), (6000, "pairs")])
def test_gates(T, kernel, dtype):
    assert {moe.dense_plan(p, T, I, H)[0] for p in ("gate_up", "dh")} == {kernel}
    gate = torch.cat([torch.linspace(-100, 100, I - 600), torch.linspace(-4, 4, 600)]).to(dtype)
    first = torch.zeros(H, dtype=dtype)
    first[0] = 1
    x = first.repeat(T, 1).to(DEV)
    up = torch.where(torch.arange(I) % 3 > 0, 1.5, -3.0).to(dtype)
    wg, wu = (first[:, None] * v for v in (gate, up))
    wd = first.repeat(I, 1)
    wg, wu, wd = (t.contiguous().to(DEV) for t in (wg, wu, wd))
    h = torch.empty(T, I, dtype=dtype, device=DEV)
    moe.moe_gated_ffn(x, wg, wu, wd, h=h)
    _, saved = moe.moe_gated_ffn(x, wg, wu, wd, save=True)
    ws = torch.empty(moe.lib.moe_gated_ffn_backward_workspace_bytes(T, I) // 2, dtype=dtype, device=DEV)
    moe.moe_gated_ffn_backward(x, x, wg, wu, wd, saved, workspace=ws)
    dg, du = ws.view(2, T, I)
    g, u = gate.double(), up.double()
    s, half = torch.sigmoid(g), torch.finfo(dtype).eps / 2
    e, flush = 2.0 ** -21 + 1.25 * g.abs() * 2.0 ** -24, (s < 2.0 ** -125).double() * s

    def check(got, want, err, what):
        tol = err + half * (want.abs() + err) + 2.0 ** -22 * want.abs() + SMALLEST[dtype] / 2
        off = (got.double().cpu() - want).abs() - tol
        assert (off <= 0).all(), f"{what}: gate {gate[(off > 0).any(0)][:5].tolist()}"
    silu = g * s
    check(h, silu * u, (e * silu).abs() * u.abs() + flush * (g * u).abs(), "h")
    slope = s * (1 + g * (1 - s))
    cut = 2.0 ** -15 * g.abs() * 1.01
    check(du, silu, (e * silu).abs() + flush * g.abs() + cut * s * (1 + g.abs() * (1 - s)), "du")
    # 1 - s is off by what s is off by and its own rounding
    err = e * slope.abs() + s * g.abs() * (e * s + 2.0 ** -24) + flush * (1 + g.abs())
    check(dg, u * slope, u.abs() * (err + cut * s * (1 - s) * (2 + g.abs())) + 2.0 ** -15 * (u * slope).abs(), "dg")
