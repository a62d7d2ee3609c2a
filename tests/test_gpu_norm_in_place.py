"""The norm written over its own inputs, where that is allowed: bit for bit what
it gives elsewhere; and refusals of the binding's calls that overlap."""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 1), (3, 31), (37, 264), (5, 1531), (9, 4096), (3, 8200), (2, 32767)])
def test_out_over_an_input(T, H):
    g = torch.Generator().manual_seed(T)
    x, r, w = (torch.randn(s, generator=g).bfloat16().to(DEV) for s in ((T, H), (T, H), (H,)))
    s, y, _ = moe.moe_add_rmsnorm(x, r, w)
    for over in ("x", "residual"):
        a = {"x": x.clone(), "residual": r.clone()}
        gs, gy, _ = moe.moe_add_rmsnorm(a["x"], a["residual"], w, out=a[over])
        assert gy is a[over] and torch.equal(gy, y) and torch.equal(gs, s)
        a = {"x": x.clone(), "residual": r.clone()}  # the stream over one input, the normed rows over the other
        other = "residual" if over == "x" else "x"
        moe.moe_add_rmsnorm(a["x"], a["residual"], w, out=a[over], stream_out=a[other])
        assert torch.equal(a[over], y) and torch.equal(a[other], s)
    y = moe.moe_add_rmsnorm(x, None, w)[1]
    assert torch.equal(moe.moe_add_rmsnorm(x, None, w, out=x)[1], y)


def test_overlaps_raise():
    x = torch.randn(8, 64, device=DEV).bfloat16()
    keep = x.clone()
    both = torch.zeros(9, 64, device=DEV, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_add_rmsnorm_backward(x, x, dx=x),
                 lambda: moe.moe_add_rmsnorm(both[:8], out=both[1:]),
                 lambda: moe.moe_add_rmsnorm(x, x.clone(), stream_out=x, out=x)):
        with pytest.raises(moe.MoeError, match="overlap"):
            call()
    assert torch.equal(x, keep)
