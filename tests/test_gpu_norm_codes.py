"""The norm's 8-bit codes next to ties: code = round(y / scale) of the fp32 y and
the scale that is stored.

Rows of ones with eps = 0 have a root mean square of exactly 1, so y is the
weight, exactly, and the expected codes follow from correctly rounded fp32
divisions on the host: no tolerance.
"""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe

pytestmark = pytest.mark.gpu

TOP = {"int8": 127.0, "e4m3": 448.0}


def _mantissas(dt):
    """The values of the type in [1, 2), at most 128 of them."""
    n = min(128, int(1 / torch.finfo(dt).eps))
    return 1 + torch.arange(n, dtype=torch.float32) / n


def _expected(y, amax, fmt):
    scale = amax / TOP[fmt]
    z = y / scale
    return scale, (torch.round(z).to(torch.int8) if fmt == "int8" else z.to(torch.float8_e4m3fn))


def _run(w, dt, fmt, group):
    x = torch.ones(3, w.numel(), dtype=dt, device=DEV)
    _, q, sc = moe.moe_add_rmsnorm(x, None, w.to(dt).to(DEV), 0.0, out_format=fmt, group=group)
    return q.cpu(), sc.cpu()


def _same(q, code):
    return torch.equal(q.view(torch.int8), code.view(torch.int8).expand_as(q))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scale_per_row(dtype, fmt):
    m = _mantissas(dtype)
    values = torch.cat([m * 2.0 ** e for e in range(-9, 1)])
    for amax in m[::3].tolist():
        for y in (values[values <= amax], values[values <= amax][:-1]):  # widths of both kinds among them
            y = torch.cat([torch.tensor([amax]), y, -y])
            scale, code = _expected(y, torch.tensor(amax), fmt)
            q, sc = _run(y, dtype, fmt, 0)
            assert (sc == scale).all()
            assert _same(q, code), f"largest value {amax}"


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scale_per_group(dtype, fmt, odd):
    """A group for every largest value: it, its half (a tie of int8 as it stands,
    63.5), and values over seven powers of two below it."""
    m = _mantissas(dtype)
    g = torch.Generator().manual_seed(3)
    rest = m[torch.randint(len(m), (len(m), 126), generator=g)] * 2.0 ** -torch.randint(
        1, 8, (len(m), 126), generator=g).float()
    y = torch.cat([m[:, None], m[:, None] / 2, rest], dim=1)
    scale, code = _expected(y, m[:, None], fmt)
    y, code, scale = y.flatten(), code.flatten(), scale.flatten()
    if odd:  # a last group of one column: the other kernel
        y, scale = torch.cat([y, torch.ones(1)]), torch.cat([scale, torch.tensor([1.0]) / TOP[fmt]])
        one = _expected(torch.ones(1), torch.ones(1), fmt)[1]
        code = torch.cat([code.view(torch.int8), one.view(torch.int8)])
    q, sc = _run(y, dtype, fmt, 128)
    assert torch.equal(sc, scale.expand_as(sc))
    assert _same(q, code)
