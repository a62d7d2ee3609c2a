"""The int8 product and the gated feed-forward block (forward and backward)
against plain 64-bit formulas, element by element, and a run of the norm, the
block and the 8-bit product together.

Tolerances.  u is half a step of the 16-bit type.  A product of K terms in fp32
is off by at most K 2^-23 of the sum of the absolute products (an addition
that cuts instead of rounding loses up to 2^-23).  Every rounding to 16 bits
adds u of its value; errors of an operand go through the next product with the
absolute values of the other.  |silu'| <= 1.1 and |silu''| <= 0.5; the saved
pre-activations are cut at 2^-15 of themselves; exp and division add 2^-19.
"""
import pytest
import torch

from gpu_helpers import DEV
from group_limited_routed_moe_b200 import moe

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def _u(dt):
    return torch.finfo(dt).eps / 2


def _round_err(v, dt):
    return _u(dt) * v.abs() + TINY[dt]


def _acc(K):
    return K * 2.0 ** -23


# ----------------------------------------------------------------- int8

INT8_SHAPES = [(1, 1, 16), (1, 8192, 1536), (2, 129, 16), (5, 64, 4096), (16, 1531, 1008), (17, 300, 144),
               (33, 1000, 272), (64, 128, 128), (65, 257, 1536), (128, 130, 640), (129, 127, 48), (200, 1531, 1008),
               (256, 256, 128), (257, 513, 144), (1000, 1536, 512), (700, 4104, 400), (2500, 2000, 1536),
               (300, 1531, 4096), (700, 520, 2064), (257, 200, 3200), (1500, 264, 1280)]


def _int8_inputs(T, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)
    b = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sa = torch.exp(torch.randn(T, generator=g)) * 0.01
    sb = torch.exp(torch.randn(N, generator=g)) * 0.01
    return a, sa, b, sb, torch.randn(N, generator=g)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,N,K", INT8_SHAPES)
def test_int8(T, N, K, bias, out):
    dt = TYPES[out]
    a, sa, b, sb, bi = _int8_inputs(T, N, K, T + N + K)
    if out == "f16":
        sb = sb * 0.01  # inside fp16's range
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    tol = want.abs() * 2.0 ** -22  # the sum's conversion and two products
    if bias:
        want = want + bi.double()
        tol = tol + want.abs() * 2.0 ** -24
    args = [t.to(DEV) for t in (a, sa, b, sb)]
    got = moe.moe_int8_matmul(*args, bias=bi.to(DEV) if bias else None, out_dtype=dt)
    assert got.dtype == dt and got.shape == (T, N)
    err = (got.cpu().double() - want).abs()
    assert (err <= tol + _round_err(want, dt)).all(), float((err / (tol + _round_err(want, dt) + 1e-300)).max())


def test_int8_sums_are_exact():
    """The largest sums there are: K = 131056 of (-128)^2, above 2^24 and just
    below 2^31, with scales of 1 in fp32."""
    K = 131056
    for T in (1, 130):
        a = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
        b = torch.full((9, K), -128, dtype=torch.int8, device=DEV)
        b[3] = 127
        b[4, 0] = -127  # 128 below the full sum: still a multiple of the fp32 step
        one = torch.ones(130, device=DEV)
        y = moe.moe_int8_matmul(a, one[:T], b, one[:9], out_dtype=torch.float32)
        full = float(K * 128 * 128)
        assert (y[:, 0] == full).all() and (y[:, 3] == -float(K * 128 * 127)).all()
        assert (y[:, 4] == full - 128).all()


def test_int8_scales_that_are_not_finite_stay_in_their_row():
    a, sa, b, sb, _ = _int8_inputs(40, 50, 64, 1)
    sa[3], sb[7] = float("nan"), float("inf")
    y = moe.moe_int8_matmul(*(t.to(DEV) for t in (a, sa, b, sb)), out_dtype=torch.float32).cpu()
    assert y[3].isnan().all()
    keep = torch.ones(40, 50, dtype=torch.bool)
    keep[3], keep[:, 7] = False, False
    assert torch.isfinite(y[keep]).all()


@pytest.mark.parametrize("T,N", [(5, 100), (5, 99), (150, 200), (150, 199)])
def test_int8_rows_behind_the_last_stay(T, N):
    a, sa, b, sb, _ = (t.to(DEV) for t in _int8_inputs(T, N, 64, 1))
    out = torch.full(((T + 3) * N,), 7.0, device=DEV)
    moe.moe_int8_matmul(a, sa, b, sb, out_dtype=torch.float32, out=out[:T * N].view(T, N))
    assert (out[T * N:] == 7).all()


def test_int8_refusals():
    a, sa, b, sb, bi = (t.to(DEV) for t in _int8_inputs(4, 32, 64, 1))
    for args, kw in (((a, sa[:3], b, sb), {}), ((a, sa, b[:, :32], sb), {}), ((a, sa, b, sb[:8]), {}),
                     ((a.float(), sa, b, sb), {}), ((a, sa.half(), b, sb), {}), ((a, sa, b.t(), sb), {}),
                     ((a, sa, b, sb), {"bias": bi[:4]}), ((a, sa, b, sb), {"out_dtype": torch.int32}),
                     ((a, sa, b, sb), {"out": torch.empty(4, 32, device=DEV)}), ((a, sa, b.cpu(), sb), {})):
        with pytest.raises(ValueError):
            moe.moe_int8_matmul(*args, **kw)
    with pytest.raises(moe.MoeError):
        moe.moe_int8_matmul(a[:, :24].contiguous(), sa, b[:, :24].contiguous(), sb)


# ----------------------------------------------------------------- gated block

def _ffn_inputs(T, H, I, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, r, dy = mk(T, H).to(dt), mk(T, H).to(dt), mk(T, H).to(dt)
    wg, wu = ((scale / H ** 0.5 * mk(H, I)).to(dt) for _ in range(2))
    return x, wg, wu, (scale / I ** 0.5 * mk(I, H)).to(dt), r, dy


class Ref:
    """Values and error bounds of the block in 64 bits."""

    def __init__(self, x, wg, wu, wd, r=None, dy=None):
        dt = x.dtype
        H, I = wg.shape
        T = x.shape[0]
        X, G, U, D = (t.double() for t in (x, wg, wu, wd))
        g, u = X @ G, X @ U
        eg, eu = _acc(H) * (X.abs() @ G.abs()), _acc(H) * (X.abs() @ U.abs())
        sig = torch.sigmoid(g)
        act = g * sig
        h = act * u
        eh = 1.1 * u.abs() * eg + act.abs() * eu + 2.0 ** -19 * h.abs()
        eh = eh + _round_err(h, dt) + _u(dt) * eh
        self.y = h @ D + (0 if r is None else r.double())
        ey = eh @ D.abs() + _acc(I) * (h.abs() @ D.abs()) + 2.0 ** -24 * self.y.abs()
        self.ty = ey + _round_err(self.y, dt) + _u(dt) * ey
        if dy is None:
            return
        Y = dy.double()
        eg, eu = eg + 2.0 ** -15 * g.abs(), eu + 2.0 ** -15 * u.abs()
        dh = Y @ D.t()
        edh = _acc(H) * (Y.abs() @ D.abs().t())
        ds = sig + act * (1 - sig)
        du, dg = dh * act, dh * u * ds
        edu = act.abs() * edh + 1.1 * dh.abs() * eg + 2.0 ** -19 * du.abs()
        edg = ((u * ds).abs() * edh + (dh * ds).abs() * eu + 0.5 * (dh * u).abs() * eg
               + 2.0 ** -18 * (dh * u).abs())
        edu = edu + _round_err(du, dt) + _u(dt) * edu
        edg = edg + _round_err(dg, dt) + _u(dt) * edg

        def product(a, ea, b, eb, K):
            return a @ b, ea @ b.abs() + a.abs() @ eb + ea @ eb + _acc(K) * (a.abs() @ b.abs())
        zx, zw = torch.zeros_like(X), torch.zeros_like(G)
        v1, e1 = product(dg, edg, G.t(), zw.t(), 2 * I)
        v2, e2 = product(du, edu, U.t(), zw.t(), 2 * I)
        outs = [(v1 + v2, e1 + e2), product(X.t(), zx.t(), dg, edg, T), product(X.t(), zx.t(), du, edu, T),
                product(h.t(), eh.t(), Y, zx, T)]
        self.grads = [v for v, _ in outs]
        self.tgrads = [e + _round_err(v, dt) + _u(dt) * e for v, e in outs]


def _ok(got, want, tol, what=""):
    err = (got.cpu().double() - want).abs()
    assert err.shape == want.shape
    assert (err <= tol).all(), f"{what}: {float((err / (tol + 1e-300)).max()):.3g} times the bound"


FFN_SHAPES = [(1, 8, 8), (1, 1536, 512), (1, 72, 4104), (2, 136, 64), (15, 512, 136), (16, 256, 264), (17, 64, 1032),
              (40, 520, 1048), (64, 128, 128), (100, 328, 200), (128, 264, 72), (129, 64, 64), (200, 136, 520),
              (256, 256, 256), (300, 392, 264), (515, 1000, 136), (1100, 264, 648),
              (300, 1536, 520), (1000, 520, 2056), (257, 1032, 1544)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,I", FFN_SHAPES)
def test_ffn(T, H, I, dtype):
    dt = TYPES[dtype]
    x, wg, wu, wd, r, _ = _ffn_inputs(T, H, I, dt, T + H + I)
    xd, *wsd = (t.to(DEV) for t in (x, wg, wu, wd))
    y = moe.moe_gated_ffn(xd, *wsd)
    ref = Ref(x, wg, wu, wd)
    _ok(y, ref.y, ref.ty, "y")
    ref = Ref(x, wg, wu, wd, r)
    y = moe.moe_gated_ffn(xd, *wsd, residual=r.to(DEV))
    _ok(y, ref.y, ref.ty, "y with residual")
    again, _ = moe.moe_gated_ffn(xd, *wsd, residual=r.to(DEV), save=True)
    assert torch.equal(again, y)  # a fixed order, and saving changes nothing


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,I", FFN_SHAPES)
def test_ffn_backward(T, H, I, dtype):
    dt = TYPES[dtype]
    x, wg, wu, wd, _, dy = _ffn_inputs(T, H, I, dt, T + H + I, scale=1.5)
    ref = Ref(x, wg, wu, wd, dy=dy)
    xd, wgd, wud, wdd, dyd = (t.to(DEV) for t in (x, wg, wu, wd, dy))
    _, saved = moe.moe_gated_ffn(xd, wgd, wud, wdd, save=True)
    got = moe.moe_gated_ffn_backward(dyd, xd, wgd, wud, wdd, saved)
    for name, a, v, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), got, ref.grads, ref.tgrads):
        _ok(a, v, e, name)
    again = moe.moe_gated_ffn_backward(dyd, xd, wgd, wud, wdd, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # parts: each output alone is the same, and nothing else is written
    for i in range(4):
        need = [j == i for j in range(4)]
        part = moe.moe_gated_ffn_backward(dyd, xd, wgd, wud, wdd, saved, need=need)
        assert [p is not None for p in part] == need and torch.equal(part[i], got[i])


def test_ffn_backward_against_differences():
    T, H, I = 9, 40, 48
    x, wg, wu, wd, _, dy = _ffn_inputs(T, H, I, torch.float16, 3)
    xd = [t.to(DEV) for t in (x, wg, wu, wd)]
    _, saved = moe.moe_gated_ffn(*xd, save=True)
    grads = moe.moe_gated_ffn_backward(dy.to(DEV), *xd, saved)
    g = torch.Generator().manual_seed(8)
    vs = [torch.randn(t.shape, generator=g).double() for t in (x, wg, wu, wd)]

    def loss(a):
        X, G, U, D = (t.double() + a * v for t, v in zip((x, wg, wu, wd), vs))
        z = X @ G
        return ((z * torch.sigmoid(z) * (X @ U)) @ D * dy.double()).sum()
    d = 1e-5
    want = (loss(d) - loss(-d)) / (2 * d)
    got = sum((a.cpu().double() * v).sum() for a, v in zip(grads, vs))
    ref = Ref(x, wg, wu, wd, dy=dy)
    tol = sum((e * v.abs()).sum() for e, v in zip(ref.tgrads, vs))
    assert abs(got - want) <= tol + 1e-4 * abs(want)


@pytest.mark.parametrize("T", [3, 150])
def test_ffn_saturated_and_not_finite(T):
    """Gates far out on both sides give the limits of silu; a token that is not
    finite stays in its own row."""
    H, I = 64, 72
    dt = torch.bfloat16
    x, wg, wu, wd, _, dy = _ffn_inputs(T, H, I, dt, 5)
    x[0] = x[0] * 1e4  # |g| up to 1e4 and more
    ref = Ref(x, wg, wu, wd, dy=dy)
    args = [t.to(DEV) for t in (x, wg, wu, wd)]
    y, saved = moe.moe_gated_ffn(*args, save=True)
    _ok(y, ref.y, ref.ty, "y")
    for a, v, e in zip(moe.moe_gated_ffn_backward(dy.to(DEV), *args, saved), ref.grads, ref.tgrads):
        _ok(a, v, e)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    y = moe.moe_gated_ffn(x.to(DEV), *args[1:]).cpu()
    assert y[1].isnan().all() and not torch.isfinite(y[2]).any()
    rest = [0] + list(range(3, T))
    _ok(y[rest], ref.y[rest], ref.ty[rest])


@pytest.mark.parametrize("T", [5, 150])
def test_ffn_in_place_and_rows_behind(T):
    H, I = 136, 264
    x, wg, wu, wd, r, _ = (t.to(DEV) for t in _ffn_inputs(T, H, I, torch.bfloat16, 9))
    want = moe.moe_gated_ffn(x, wg, wu, wd, residual=r)
    buf = torch.full((T + 4, H), 7.0, dtype=torch.bfloat16, device=DEV)
    hbuf = torch.full((T + 4, I), 7.0, dtype=torch.bfloat16, device=DEV)
    buf[:T] = r
    got = moe.moe_gated_ffn(x, wg, wu, wd, residual=buf[:T], y=buf[:T], h=hbuf[:T])
    assert torch.equal(got, want) and (buf[T:] == 7).all() and (hbuf[T:] == 7).all()
    want = moe.moe_gated_ffn(x, wg, wu, wd, residual=x)
    assert torch.equal(moe.moe_gated_ffn(x, wg, wu, wd, residual=x, y=x), want)


def test_ffn_no_tokens():
    _, wg, wu, wd, _, _ = (t.to(DEV) for t in _ffn_inputs(1, 64, 72, torch.bfloat16, 9))
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    y, saved = moe.moe_gated_ffn(e, wg, wu, wd, save=True)
    assert y.shape == (0, 64)
    full = [torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV) for s in ((64, 72), (64, 72), (72, 64))]
    dx, *dws = moe.moe_gated_ffn_backward(e, e, wg, wu, wd, saved, dw_gate=full[0], dw_up=full[1], dw_down=full[2])
    assert dx.shape == (0, 64) and all((d == 0).all() for d in dws)


def test_ffn_refusals():
    x, wg, wu, wd, r, dy = (t.to(DEV) for t in _ffn_inputs(4, 64, 72, torch.bfloat16, 9))
    for args, kw in (((x, wg, wu, wd.t()), {}), ((x, wg.half(), wu, wd), {}), ((x, wg, wu[:, :64], wd), {}),
                     ((x, wg, wu, wd), {"residual": r[:3]}), ((x, wg, wu, wd.cpu()), {}),
                     ((x.float(), wg, wu, wd), {}), ((x, wg, wu, wd), {"y": x.float()})):
        with pytest.raises(ValueError):
            moe.moe_gated_ffn(*args, **kw)
    with pytest.raises(moe.MoeError):  # I not a multiple of 8
        moe.moe_gated_ffn(x, wg[:, :68].contiguous(), wu[:, :68].contiguous(), wd[:68].contiguous())
    _, saved = moe.moe_gated_ffn(x, wg, wu, wd, save=True)
    with pytest.raises(ValueError):
        moe.moe_gated_ffn(x, wg, wu, wd, save=True, h=torch.empty(4, 72, dtype=x.dtype, device=DEV))
    with pytest.raises(ValueError):
        moe.moe_gated_ffn_backward(dy[:3], x, wg, wu, wd, saved)
    with pytest.raises(ValueError):
        moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved[:-16])
    with pytest.raises(ValueError):
        moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved, need=(True, True))
    with pytest.raises(moe.MoeError):
        moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("T", [1, 33, 300])
def test_capture_and_replay(T):
    """A training step captured into a graph and replayed on changed inputs."""
    x, wg, wu, wd, r, dy = (t.to(DEV) for t in _ffn_inputs(T, 256, 520, torch.bfloat16, 9))

    def step():
        y, saved = moe.moe_gated_ffn(x, wg, wu, wd, residual=r, save=True)
        return [y, *moe.moe_gated_ffn_backward(dy, x, wg, wu, wd, saved)]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    x.copy_(torch.randn_like(x))
    wg.mul_(1.25)
    want = step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    """Calls on two streams share no state: results as when run alone."""
    cases = [_ffn_inputs(T, 256, 1032, torch.bfloat16, T) for T in (3, 400)]
    cases = [[t.to(DEV) for t in c] for c in cases]
    want = [moe.moe_gated_ffn(*c[:4], residual=c[4]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate(cases):
            got[i].append(moe.moe_gated_ffn(*c[:4], residual=c[4], stream=streams[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, t) for t in g)
    assert moe.get_device_status(0) == moe.MOE_OK


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("T", [1, 37, 300])
def test_eight_bit_layer(T):
    """Norm with int8 rows, then the 8-bit product on them: the product of the
    codes is exact, so the bound is the norm's codes against the true rows."""
    H, N = 1536, 520
    g = torch.Generator().manual_seed(T)
    x, r = (torch.randn(T, H, generator=g).bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16()
    wt = 0.02 * torch.randn(N, H, generator=g)
    sb = wt.abs().amax(1) / 127
    b = torch.round(wt / sb[:, None]).to(torch.int8)
    s, q, sc = moe.moe_add_rmsnorm(x.to(DEV), r.to(DEV), w.to(DEV), out_format="int8")
    y = moe.moe_int8_matmul(q, sc, b.to(DEV), sb.to(DEV))
    sd = s.cpu().double()
    n = sd * w.double() / torch.sqrt((sd * sd).mean(1, keepdim=True) + 1e-6)
    B = b.double() * sb.double()[:, None]
    want = n @ B.t()
    step = n.abs().amax(1, keepdim=True) / 127
    tol = 0.501 * step * B.abs().sum(1) + 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -15 * (n.abs() @ B.abs().t())
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_training_step_of_a_dense_layer(T, dtype):
    """stream = x + residual; y = stream + FFN(norm(stream)); gradients of all
    of it against 64-bit autograd.  Along any path a gradient passes at most
    five roundings (normed rows, h, dg or du, the normed rows' gradient, the
    result), each u relative to values whose sums the next step passes on
    with gains below 2: relative 2-norm error at most 12 u."""
    dt = TYPES[dtype]
    H, I = 264, 520
    x, wg, wu, wd, r, dy = _ffn_inputs(T, H, I, dt, T)
    w = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(dt)
    xd, wgd, wud, wdd, rd, dyd, nwd = (t.to(DEV) for t in (x, wg, wu, wd, r, dy, w))
    s, n, _ = moe.moe_add_rmsnorm(xd, rd, nwd)
    y, saved = moe.moe_gated_ffn(n, wgd, wud, wdd, residual=s, save=True)
    dn, dwg, dwu, dwd = moe.moe_gated_ffn_backward(dyd, n, wgd, wud, wdd, saved)
    dx, dw = moe.moe_add_rmsnorm_backward(dn, s, nwd, dstream=dyd)
    leaves = [t.double().requires_grad_() for t in (s.cpu(), w, wg, wu, wd)]
    S, W, G, U, D = leaves
    N = S * W / torch.sqrt((S * S).mean(1, keepdim=True) + 1e-6)
    Y = S + (torch.nn.functional.silu(N @ G) * (N @ U)) @ D
    want = torch.autograd.grad(Y, leaves, dy.double())
    for name, a, v in zip(("y", "dx", "dw", "dwg", "dwu", "dwd"), (y, dx, dw, dwg, dwu, dwd), (Y.detach(), *want)):
        err = float((a.cpu().double() - v).norm() / v.norm())
        assert err <= 12 * _u(dt), f"{name}: {err:.3g}"


@pytest.mark.parametrize("T", [1, 37, 300])
def test_back_to_back(T):
    """A run of different calls without a wait between them (each may start
    while the one before finishes) gives what it gives with a wait after each."""
    from gpu_helpers import layer0_weights
    H, I = 1536, 1032
    x, wg, wu, wd, r, dy = (t.to(DEV) for t in _ffn_inputs(T, H, I, torch.bfloat16, T))
    g = torch.Generator().manual_seed(T)
    router = moe.moe_pack_router((0.05 * torch.randn(H, 128, generator=g)).bfloat16().to(DEV))
    b = torch.randint(-127, 128, (H, H), generator=g, dtype=torch.int8).to(DEV)
    sb = torch.full((H,), 1e-4, device=DEV)
    packed = layer0_weights().packed

    def run(wait):
        outs, s = [], x
        for _ in range(3):
            s, n, _ = moe.moe_add_rmsnorm(s, r)
            wait()
            y, saved = moe.moe_gated_ffn(n, wg, wu, wd, residual=s, save=True)
            wait()
            grads = moe.moe_gated_ffn_backward(dy, n, wg, wu, wd, saved)
            wait()
            dx, dw = moe.moe_add_rmsnorm_backward(grads[0], s, dstream=dy)
            wait()
            _, q, sc = moe.moe_add_rmsnorm(y, r, out_format="int8")
            wait()
            z = moe.moe_int8_matmul(q, sc, b, sb)
            wait()
            s, out = moe.moe_layer_normed(z, y, None, 1e-6, router, None, packed)
            wait()
            outs += [y, *grads, dx, dw, z, s, out]
            s = out
        return outs
    want = run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for _ in range(5):
        got = run(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
    assert moe.get_device_status(0) == moe.MOE_OK


def test_beside_the_routed_layer():
    """Dense products on one stream while routed layers run on another: neither
    waits for the other for good, and both give what they give alone."""
    from gpu_helpers import layer0_weights
    from group_limited_routed_moe_b200 import synth
    packed = layer0_weights().packed
    jobs = []
    for T in (2, 300):
        tok = synth.make_tokens(T, seed=1)
        lx = torch.from_numpy(tok.x_bits.view("int16")).to(DEV).view(torch.bfloat16)
        lg, bias = torch.from_numpy(tok.logits).to(DEV), torch.from_numpy(tok.bias).to(DEV)
        jobs.append(lambda lx=lx, lg=lg, bias=bias: moe.moe_layer(lx, lg, bias, packed))
    dense = []
    for T in (1, 50, 400):
        x, wg, wu, wd, r, dy = (t.to(DEV) for t in _ffn_inputs(T, 512, 1032, torch.bfloat16, T))
        dense.append(lambda x=x, wg=wg, wu=wu, wd=wd, r=r: moe.moe_gated_ffn(x, wg, wu, wd, residual=r))
    want = [[f() for f in jobs], [f() for f in dense]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, fs in enumerate((jobs, dense)):
            with torch.cuda.stream(streams[i]):
                got[i].append([f() for f in fs])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, c) for run in got[i] for a, c in zip(want[i], run))
    assert moe.get_device_status(0) == moe.MOE_OK
