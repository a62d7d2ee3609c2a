"""Offsets past 32 bits in the norm, the int8 product and the gated block:
sampled rows against 64 bits (the tolerances of test_gpu_norm and
test_gpu_dense)."""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe
from test_gpu_dense import Ref, _ok

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_norm():
    T, H = 70_000, 32_768  # 2.3e9 elements
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, H), generator=g, device=DEV, dtype=torch.bfloat16)
    rows = [0, 1, 65_535, 65_536, 65_537, T - 1]
    s, y, _ = moe.moe_add_rmsnorm(x, x)
    assert torch.equal(s[rows], x[rows] + x[rows])
    sd = s[rows].double()
    want = sd / torch.sqrt((sd * sd).mean(1, keepdim=True) + 1e-6)
    assert ((y[rows].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -9)).all()
    _, q, sc = moe.moe_add_rmsnorm(x, x, out_format="int8", group=128, stream_out=s)
    got = q[rows].double() * sc[rows].double().repeat_interleave(128, dim=1)
    assert ((got - want).abs() <= sc[rows].double().repeat_interleave(128, dim=1) * 0.51 + 2.0 ** -9 * want.abs()).all()
    del q, sc
    dx, _ = moe.moe_add_rmsnorm_backward(y, s)  # dy = y: dx = rstd (n - n mean(n^2)) is all but zero
    rstd = 1 / torch.sqrt((sd * sd).mean(1, keepdim=True) + 1e-6)
    yd = y[rows].double()
    n = sd * rstd
    wdx = rstd * (yd - n * (yd * n).mean(1, keepdim=True))
    assert ((dx[rows].double() - wdx).abs() <= 2.0 ** -8 * wdx.abs() + rstd * 2.0 ** -8 * yd.abs()).all()


def test_int8():
    T, N, K = 40_000, 65_540, 16  # 2.6e9 outputs
    g = torch.Generator(device=DEV).manual_seed(2)
    a, b = (torch.randint(-128, 128, (n, K), generator=g, device=DEV, dtype=torch.int8) for n in (T, N))
    sa, sb = (torch.rand(n, generator=g, device=DEV) for n in (T, N))
    y = moe.moe_int8_matmul(a, sa, b, sb)
    rows = [0, 255, 32_766, 32_767, 32_768, T - 1]
    want = (a[rows].double() @ b.double().t()) * sa[rows].double()[:, None] * sb.double()
    err = (y[rows].double() - want).abs()
    assert (err <= want.abs() * (2.0 ** -8 + 2.0 ** -20)).all()


def test_gated_block():
    """With dy zero but for a few rows, the weights' gradients are those of
    these rows, and dx is zero in all others."""
    T, H, I = 530_000, 8, 4104  # 2.2e9 elements of h, 13 GB of saved values
    rows = [0, 31, 32, 261_631, 523_263, 523_264, 523_265, T - 1]
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
    wg, wu = ((0.3 * torch.randn((H, I), generator=g, device=DEV)).bfloat16() for _ in range(2))
    wd = (0.02 * torch.randn((I, H), generator=g, device=DEV)).bfloat16()
    dy = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    dy[rows] = torch.randn((len(rows), H), generator=g, device=DEV).bfloat16()
    y, saved = moe.moe_gated_ffn(x, wg, wu, wd, save=True)
    ref = Ref(x[rows].cpu(), wg.cpu(), wu.cpu(), wd.cpu(), dy=dy[rows].cpu())
    _ok(y[rows], ref.y, ref.ty, "y")
    dx, *dws = moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved)
    _ok(dx[rows], ref.grads[0], ref.tgrads[0], "dx")
    dx[rows] = 0
    assert not dx.any()
    for d, v, e in zip(dws, ref.grads[1:], ref.tgrads[1:]):
        _ok(d, v, e)
