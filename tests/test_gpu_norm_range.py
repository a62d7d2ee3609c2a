"""The norm and its gradients of rows whose squares leave fp32's range, for eps
from 0 up, against 64 bits; ordinary rows between them stay what they are.

Tolerances as in test_gpu_norm.  The rows are scaled by a power of two before
they are summed again, which rounds nothing (an element more than 2^126 below
its row's largest one may vanish; none is here).
"""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe
from test_gpu_norm import TINY, _check_codes, _rel_y, _u

pytestmark = pytest.mark.gpu

DT = torch.bfloat16
SIZES = [4e-40, 1e-38, 1e-30, 1e-25, 1e-18, 1.0, 3e18, 1e19, 1e30]  # of a row's elements
HS = [1, 5, 64, 257, 1536, 4096, 8200, 16385]


def _rows(H, seed, reps=1):
    """Rows of every size, one after the other, `reps` times: unit noise times
    the size, no element below a quarter of it."""
    g = torch.Generator().manual_seed(seed)
    size = torch.tensor(SIZES, dtype=torch.float64).repeat(reps)[:, None]
    v = torch.randn(size.shape[0], H, generator=g).double()
    v = torch.where(v < 0, -1.0, 1.0) * v.abs().clamp(0.25, 4)
    return (v * size).to(DT), size, g


def _norm64(x, eps):
    x = x.double()
    eps = torch.tensor(eps, dtype=torch.float32).double()  # the value that is passed on
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    return rstd, x * rstd


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-12, 1e-6])
@pytest.mark.parametrize("H", HS)
def test_forward(H, eps):
    x, _, _ = _rows(H, H)
    _, y = _norm64(x, eps)
    got = moe.moe_add_rmsnorm(x.to(DEV), eps=eps)[1].cpu().double()
    # below 2^-126 a step of the type is 2^-133
    tol = y.abs() * (_u(DT) + _rel_y(H)) + 2.0 ** -133
    bad = ~((got - y).abs() <= tol)
    assert not bad.any(), f"rows of size {[SIZES[i] for i in bad.any(1).nonzero().flatten().tolist()]}"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", [5, 257, 1536])
def test_codes_without_eps(H, group, fmt):
    x, _, _ = _rows(H, H)
    _, y = _norm64(x, 0.0)
    _, q, sc = moe.moe_add_rmsnorm(x.to(DEV), eps=0.0, out_format=fmt, group=group)
    _check_codes(q.cpu(), sc.cpu(), y, group, fmt, H)


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-12, 1e-6])
@pytest.mark.parametrize("H", HS)
def test_backward(H, eps):
    """More rows than blocks, so that rows of both kinds follow one another in
    a block."""
    reps = 1000 if H <= 257 else 220 if H <= 4096 else 40
    x, size, g = _rows(H, H + 1, reps)
    T = x.shape[0]
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(DT)
    # gradients of a size that leaves dx inside the type's range
    dy = (torch.randn(T, H, generator=g).double() * size.clamp(1e-4, 1.0)).to(DT)
    rstd, n = _norm64(x, eps)
    d = dy.double()
    dn = d * w.double()
    m = (dn * n).mean(1, keepdim=True)
    want = rstd * (dn - n * m)
    dx, dw = moe.moe_add_rmsnorm_backward(*(t.to(DEV) for t in (dy, x, w)), eps=eps)
    rel = 2 * _rel_y(H) + 2.0 ** -21
    em = (rel + 2 * H * 2.0 ** -24) * (dn * n).abs().mean(1, keepdim=True)
    tol = (_u(DT) + 2.0 ** -22) * want.abs() + rstd * (rel * (dn.abs() + (n * m).abs()) + n.abs() * em) + 2.0 ** -133
    big = torch.finfo(DT).max
    got = dx.cpu().double()
    ok = ((got - want).abs() <= tol) | (got.isinf() & (want.abs() + tol >= big))
    assert ok.all(), f"rows of size {sorted(set(SIZES[i % len(SIZES)] for i in (~ok).any(1).nonzero().flatten().tolist()))}"
    wdw = (d * n).sum(0)
    tdw = (d * n).abs().sum(0) * (rel + (T + 8) * 2.0 ** -24) + 1e-30
    assert ((dw.cpu().double() - wdw).abs() <= tdw).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_zero_rows(dtype):
    """With eps they give zeros; without, the formula's 0 / 0 in their own rows,
    and in nobody else's."""
    x = torch.randn(40, 264, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[::3] = 0
    keep = [i for i in range(40) if i % 3]
    dy = torch.ones_like(x)
    for eps in (1e-44, 1e-6):
        y = moe.moe_add_rmsnorm(x.to(DEV), eps=eps)[1].cpu()
        dx, dw = moe.moe_add_rmsnorm_backward(dy.to(DEV), x.to(DEV), eps=eps)
        assert (y[::3] == 0).all() and torch.isfinite(y).all() and torch.isfinite(dw).all()
        assert torch.isfinite(dx[keep]).all() and not dx.isnan().any()
    y = moe.moe_add_rmsnorm(x.to(DEV), eps=0.0)[1].cpu()
    dx, _ = moe.moe_add_rmsnorm_backward(dy.to(DEV), x.to(DEV), eps=0.0, need_dweight=False)
    assert y[::3].isnan().all() and dx[::3].isnan().all()
    rstd, n = _norm64(x[keep], 0.0)
    assert ((y[keep].double() - n).abs() <= n.abs() * (_u(dtype) + _rel_y(264)) + TINY[dtype]).all()
    assert torch.isfinite(dx[keep]).all()
