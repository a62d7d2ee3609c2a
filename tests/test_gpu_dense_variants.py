"""The gated block and the int8 product in every way they can run (kernel, tile,
sharing of tiles by k), element by element against 64 bits, with the bounds of
test_gpu_dense.  The formulas are computed in fp64 on the device."""
import pytest
import torch

import dense_shapes
from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe
from test_gpu_dense import TYPES, Ref, _ffn_inputs, _round_err

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()
    assert moe.get_device_status(0) == moe.MOE_OK


def _ok(got, want, tol, what):
    assert got.shape == want.shape
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"{what}: {float((err / (tol + 1e-300)).max()):.3g} times the bound"


def test_every_way_is_taken_on_this_device():
    assert not dense_shapes.uncovered(10_000, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,I", dense_shapes.FFN)
def test_gated_block(T, H, I, dtype):
    x, wg, wu, wd, r, dy = (t.to(DEV) for t in _ffn_inputs(T, H, I, TYPES[dtype], T + H + I, scale=1.2))
    y, saved = moe.moe_gated_ffn(x, wg, wu, wd, residual=r, save=True)
    grads = moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved)
    ref = Ref(x, wg, wu, wd, r, dy)
    _ok(y, ref.y, ref.ty, "y")
    for name, a, v, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, ref.grads, ref.tgrads):
        _ok(a, v, e, name)
    assert torch.equal(moe.moe_gated_ffn(x, wg, wu, wd, residual=r), y)
    again = moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,K", dense_shapes.INT8)
def test_int8(T, N, K, out):
    dt = TYPES[out]
    g = torch.Generator(device=DEV).manual_seed(T + N + K)
    a, b = (torch.randint(-128, 128, (n, K), generator=g, device=DEV, dtype=torch.int8) for n in (T, N))
    sa, sb = (0.01 * torch.exp(torch.randn(n, generator=g, device=DEV)) for n in (T, N))
    if out == "f16":
        sb = sb * 0.001  # inside fp16's range
    bias = torch.randn(N, generator=g, device=DEV)
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    tol = want.abs() * 2.0 ** -22  # the sum's conversion and two products
    _ok(moe.moe_int8_matmul(a, sa, b, sb, out_dtype=dt), want, tol + _round_err(want, dt), "without bias")
    want = want + bias.double()
    tol = tol + want.abs() * 2.0 ** -24
    got = moe.moe_int8_matmul(a, sa, b, sb, bias=bias, out_dtype=dt)
    _ok(got, want, tol + _round_err(want, dt), "with bias")
    assert torch.equal(moe.moe_int8_matmul(a, sa, b, sb, bias=bias, out_dtype=dt), got)
