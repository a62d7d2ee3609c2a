"""The norm (16-bit, int8, E4M3 outputs; backward) against plain 64-bit
formulas, and the pre-norm layer against its parts.

Tolerances, with u half a step of the output type: the stream is exact (the
fp32 sum of two 16-bit values rounds like the exact sum).  y: u for its
rounding; the fp32 mean of H squares is off by at most (H + 2) 2^-24, its root
by half of that, rsqrt and the products by 2^-21 together.  A code is off by
at most half a step of its format plus those errors.  Gradients: the same
terms, with the mean's error relative to the sum of the absolute products;
dweight: T fp32 additions of products, each relative 2^-24.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV, layer0_weights
from group_limited_routed_moe_b200 import moe, synth

pytestmark = pytest.mark.gpu

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half the smallest step


def _u(dt):
    return torch.finfo(dt).eps / 2


def _rel_y(H):
    return (H + 2) * 2.0 ** -25 + 2.0 ** -21


def _inputs(T, H, dt, seed, residual=True, weight=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dt)
    r = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dt) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(dt) if weight else None
    return x, r, w


def _ref(x, r, w):
    s = x if r is None else (x.double() + r.double()).to(x.dtype)
    sd = s.double()
    rstd = 1 / torch.sqrt((sd * sd).mean(1, keepdim=True) + EPS)
    n = sd * rstd
    return s, rstd, n, n if w is None else n * w.double()


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


SHAPES = [(1, 1), (1, 1536), (3, 7), (2, 8), (5, 127), (4, 129), (7, 1531), (3, 4096), (2, 8200), (1, 32768),
          (2, 32767), (2, 16385), (300, 1536)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_same(T, H, dtype):
    dt = TYPES[dtype]
    x, r, w = _inputs(T, H, dt, T * 100003 + H)
    s, _, _, y = _ref(x, r, w)
    gs, gy, gsc = moe.moe_add_rmsnorm(*_dev(x, r, w), eps=EPS)
    assert gsc is None
    assert torch.equal(gs.cpu(), s)
    assert ((gy.cpu().double() - y).abs() <= y.abs() * (_u(dt) + _rel_y(H)) + TINY[dt]).all()


def _check_codes(q, scales, y, group, fmt, H):
    T = y.shape[0]
    top = 127.0 if fmt == "int8" else 448.0
    size = group or H
    rel = _rel_y(H) + 2.0 ** -22
    assert scales.shape == (T, -(-H // size))
    for g in range(scales.shape[1]):
        part = y[:, g * size:(g + 1) * size]
        sc = scales[:, g:g + 1].double()
        want = (part.abs().amax(1, keepdim=True) / top).clamp_min(2.0 ** -126)
        assert ((sc - want).abs() <= want * rel).all()
        got = q[:, g * size:(g + 1) * size].double() * sc
        z = part / sc
        if fmt == "int8":
            step = torch.ones_like(z)
        else:  # three mantissa bits; subnormal step 2^-9
            step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
        # the codes' clamp at the top cuts at most the scale's own error
        assert ((got - part).abs() <= sc * (0.5 * step + z.abs() * 3 * rel)).all()
        if fmt == "int8":
            assert q[:, g * size:(g + 1) * size].double().abs().max() <= 127


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 1536), (3, 7), (5, 127), (4, 129), (3, 136), (7, 1531), (3, 4096),
                                 (2, 8200), (1, 32768), (2, 32767), (130, 1536)])
def test_codes(T, H, group, fmt):
    x, r, w = _inputs(T, H, torch.bfloat16, T + H)
    s, _, _, y = _ref(x, r, w)
    gs, q, sc = moe.moe_add_rmsnorm(*_dev(x, r, w), eps=EPS, out_format=fmt, group=group)
    assert q.dtype == (torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    assert torch.equal(gs.cpu(), s)
    _check_codes(q.cpu(), sc.cpu(), y, group, fmt, H)


def test_without_residual_or_weight():
    x, _, _ = _inputs(9, 520, torch.float16, 5, residual=False, weight=False)
    _, _, _, y = _ref(x, None, None)
    xd = x.to(DEV)
    s, gy, _ = moe.moe_add_rmsnorm(xd)
    assert s is xd
    assert ((gy.cpu().double() - y).abs() <= y.abs() * (_u(x.dtype) + _rel_y(520)) + TINY[x.dtype]).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", [256, 257])
def test_zero_rows_and_values_that_are_not_finite(H, group):
    """A zero row has code 0 and the smallest scale; a NaN or an infinity marks
    its own row (or group), and no other."""
    x, r, w = _inputs(5, H, torch.bfloat16, 11)
    x[1], r[1] = 0, 0
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    s, _, _, y = _ref(x, r, w)
    gs, q, sc = moe.moe_add_rmsnorm(*_dev(x, r, w), eps=EPS, out_format="int8", group=group)
    gs, q, sc = gs.cpu(), q.cpu().float(), sc.cpu()
    assert torch.equal(gs.isnan(), s.isnan()) and torch.equal(gs[~s.isnan()], s[~s.isnan()])
    assert (q[1] == 0).all() and (sc[1] == 2.0 ** -126).all()
    assert sc[2].isnan().all()                     # a NaN in the row: its mean is NaN
    per = sc[3:4].repeat_interleave(group or H, dim=1)[0, :H]
    v = q[3] * per
    assert v[200].isnan()                          # infinity times 1 / infinity
    if group:
        assert (v[:128] == 0).all()                # finite over infinite
    _check_codes(q[[0, 4]], sc[[0, 4]], y[[0, 4]], group, "int8", H)
    gy = moe.moe_add_rmsnorm(*_dev(x, r, w), eps=EPS)[1].cpu()
    assert gy[2].isnan().all() and gy[3, 200].isnan() and (gy[1] == 0).all()
    assert torch.isfinite(gy[[0, 1, 4]]).all()


def test_tiny_and_large_values():
    """Rows near the ends of the type's range, where amax / top is subnormal
    or squares are large, against 64 bits."""
    x = torch.tensor([[1e-30] * 64, [3e18] * 64, [1e-38] * 64], dtype=torch.bfloat16)
    x[:, 5] *= -2
    w = torch.full((64,), 1e-30, dtype=torch.bfloat16)
    s, _, _, y = _ref(x, None, None)
    gy = moe.moe_add_rmsnorm(x.to(DEV), eps=EPS)[1].cpu()
    assert ((gy.double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133).all()
    _, _, _, y = _ref(x, None, w)
    _, q, sc = moe.moe_add_rmsnorm(x.to(DEV), None, w.to(DEV), eps=EPS, out_format="int8")
    got = q.cpu().double() * sc.cpu().double()
    assert ((got - y).abs() <= sc.cpu().double() * 0.501 + y.abs() * 2.0 ** -18).all()


@pytest.mark.parametrize("which", ["x", "residual"])
def test_stream_in_place(which):
    x, r, w = _inputs(33, 1000, torch.bfloat16, 3)
    want_s, want_y, _ = moe.moe_add_rmsnorm(*_dev(x, r, w))
    xd, rd, wd = _dev(x, r, w)
    target = xd if which == "x" else rd
    s, y, _ = moe.moe_add_rmsnorm(xd, rd, wd, stream_out=target)
    assert s is target and torch.equal(s, want_s) and torch.equal(y, want_y)


def test_rows_behind_the_last_stay():
    x, r, w = _dev(*_inputs(5, 264, torch.bfloat16, 3))
    s, y = (torch.full((9, 264), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_add_rmsnorm(x, r, w, stream_out=s[:5], out=y[:5])
    q = torch.full((9, 264), 7, dtype=torch.int8, device=DEV)
    sc = torch.full((9, 3), 7.0, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, out_format="int8", group=128, out=q[:5], scales=sc[:5])
    for t in (s, y, q, sc):
        assert (t[5:].float() == 7).all() and not (t[:5].float() == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dstream", [True, False])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 1536), (3, 7), (601, 136), (1300, 257), (40, 4096), (3, 16385),
                                 (2, 32768)])
def test_backward(T, H, dstream, dtype):
    dt = TYPES[dtype]
    x, _, w = _inputs(T, H, dt, T * 7 + H, residual=False)
    g = torch.Generator().manual_seed(H)
    dy = torch.randn(T, H, generator=g).to(dt)
    ds = torch.randn(T, H, generator=g).to(dt) if dstream else None
    _, rstd, n, _ = _ref(x, None, w)
    dn = dy.double() * w.double()
    m = (dn * n).mean(1, keepdim=True)
    want = rstd * (dn - n * m) + (ds.double() if dstream else 0)
    gdx, gdw = moe.moe_add_rmsnorm_backward(*_dev(dy, x, w), eps=EPS, dstream=None if ds is None else ds.to(DEV))
    rel = 2 * _rel_y(H) + 2.0 ** -21
    em = rel * (dn * n).abs().mean(1, keepdim=True) + 2 * H * 2.0 ** -24 * (dn * n).abs().mean(1, keepdim=True)
    tol = _u(dt) * want.abs() + rstd * (rel * (dn.abs() + (n * m).abs()) + n.abs() * em) + 2.0 ** -22 * want.abs()
    if dstream:
        tol = tol + 2.0 ** -23 * ds.double().abs()
    assert ((gdx.cpu().double() - want).abs() <= tol + TINY[dt]).all()
    wdw = (dy.double() * n).sum(0)
    tdw = (dy.double() * n).abs().sum(0) * (rel + (T + 8) * 2.0 ** -24) + 1e-30
    assert ((gdw.cpu().double() - wdw).abs() <= tdw).all()
    again = moe.moe_add_rmsnorm_backward(*_dev(dy, x, w), eps=EPS, dstream=None if ds is None else ds.to(DEV))
    assert torch.equal(again[0], gdx) and torch.equal(again[1], gdw)  # a fixed order


def test_backward_against_differences():
    x, _, w = _inputs(6, 96, torch.float16, 2, residual=False)
    g = torch.Generator().manual_seed(4)
    dy, vx, vw = (torch.randn(6, 96, generator=g).half(), torch.randn(6, 96, generator=g).double(),
                  torch.randn(96, generator=g).double())
    dx, dw = moe.moe_add_rmsnorm_backward(*_dev(dy, x, w), eps=EPS)

    def loss(a):
        s, ww = x.double() + a * vx, w.double() + a * vw
        return (dy.double() * s * ww / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)).sum()
    d = 1e-4
    want = (loss(d) - loss(-d)) / (2 * d)  # error d^2 times a third derivative of order 1e3
    got = (dx.cpu().double() * vx).sum() + (dw.cpu().double() * vw).sum()
    # each of the 576 dx is rounded by at most 2^-11 of itself
    assert abs(got - want) <= 2.0 ** -11 * (dx.cpu().double() * vx).abs().sum() + 1e-4


def test_backward_parts():
    x, _, _ = _inputs(5, 40, torch.bfloat16, 2, residual=False)
    dy = torch.randn(5, 40).to(torch.bfloat16)
    full = moe.moe_add_rmsnorm_backward(*_dev(dy, x))
    part = moe.moe_add_rmsnorm_backward(*_dev(dy, x), need_dweight=False)
    assert part[1] is None and torch.equal(part[0], full[0])
    dw = torch.full((40,), 3.0, device=DEV)
    e = torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    moe.moe_add_rmsnorm_backward(e, e, dweight=dw)
    assert (dw == 0).all()  # the gradient of no tokens


def test_streams_and_capture():
    """Another stream than the current one, and a captured and replayed call on
    changed inputs."""
    x, r, w = _dev(*_inputs(64, 1536, torch.bfloat16, 3))
    want = moe.moe_add_rmsnorm(x, r, w, out_format="int8")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = moe.moe_add_rmsnorm(x, r, w, out_format="int8", stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    dy = torch.randn_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s, q, sc = moe.moe_add_rmsnorm(x, r, w, out_format="int8")
        dx, dw = moe.moe_add_rmsnorm_backward(dy, s, w)
    x.copy_(torch.randn_like(x))
    want = moe.moe_add_rmsnorm(x, r, w, out_format="int8") + moe.moe_add_rmsnorm_backward(
        dy, moe.moe_add_rmsnorm(x, r, w)[0], w)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (s, q, sc, dx, dw)))


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    for bad in ({"residual": x.half()}, {"residual": x[:3]}, {"weight": x[0, :32]}, {"weight": x[0].cpu()},
                {"out_format": "int4"}, {"group": 128}, {"group": 64, "out_format": "int8"},
                {"out": x.float()}, {"residual": x.t().contiguous().t()},
                {"scales": x, "out_format": "int8"}):
        with pytest.raises(ValueError):
            moe.moe_add_rmsnorm(x, **bad)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x.float())
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm_backward(x, x, workspace=torch.empty(8, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x.reshape(-1)[4:68].view(1, 64))  # 8 bytes off


@pytest.mark.parametrize("T", [0, 1, 5, 77, 300])
@pytest.mark.parametrize("residual", [True, False])
def test_layer_normed_is_its_parts(T, residual):
    """Bit for bit the norm followed by moe_layer_routed with the stream as
    residual, whose own parity tests hold the layer to the oracle."""
    W = layer0_weights()
    g = torch.Generator().manual_seed(T)
    x, r, w = _dev(*_inputs(T, 1536, torch.bfloat16, T + 1, residual=residual))
    wr = (0.05 * torch.randn(1536, 128, generator=g)).to(torch.bfloat16).to(DEV)
    router = moe.moe_pack_router(wr)
    bias = torch.from_numpy(synth.make_tokens(4, seed=0).bias).to(DEV)
    s, out = moe.moe_layer_normed(x, r, w, EPS, router, bias, W.packed)
    assert out.shape == (T, 1536)
    if T == 0:
        return
    ws, n, _ = moe.moe_add_rmsnorm(x, r, w, EPS)
    want = moe.moe_layer_routed(n, router, bias, W.packed, residual=ws)
    assert torch.equal(s, ws) and torch.equal(out, want)
    # in place: the stream over the residual, the output over the input
    rr = x if r is None else r.clone()
    s2, out2 = moe.moe_layer_normed(x, None if r is None else rr, w, EPS, router, bias, W.packed,
                                    stream_out=None if r is None else rr, out=x)
    assert torch.equal(out2, want)
    assert moe.get_device_status(0) == moe.MOE_OK
