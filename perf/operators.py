"""The operators around a dense feed-forward layer, as they are measured.

norm        residual addition and root-mean-square norm, its output in 8 bits with scales
norm_train  the same norm with a 16-bit output, forward and backward
int8        matrix product in 8-bit integers with a scale for each token and each channel
ffn         the gated (SwiGLU) feed-forward block of any width, forward
ffn_train   the same block, forward and backward

`run` computes a case in its plain form, or, where `own` is true, by the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of an 8-bit layer while one stream decodes: latency
        {"name": "norm_int8_T1", "op": "norm", "T": 1, "H": 1536, "dtype": "bf16", "fmt": "int8", "group": 0},
        # the same in front of a long prompt, with a scale for every 128 columns
        {"name": "norm_e4m3_T8189", "op": "norm", "T": 8189, "H": 1536, "dtype": "bf16", "fmt": "e4m3", "group": 128},
        # a training step's norm: a wide model's rows, and a ragged batch of odd rows
        {"name": "norm_train_T8189", "op": "norm_train", "T": 8189, "H": 4096, "dtype": "bf16"},
        {"name": "norm_train_T333", "op": "norm_train", "T": 333, "H": 1531, "dtype": "f16"},
        # an 8-bit layer's product: four decoding streams, a ragged batch with an odd number of
        # channels, a long prompt
        {"name": "int8_T4", "op": "int8", "T": 4, "N": 8192, "K": 1536, "out": "bf16", "bias": False},
        {"name": "int8_T203", "op": "int8", "T": 203, "N": 1531, "K": 1008, "out": "f16", "bias": True},
        {"name": "int8_T8189", "op": "int8", "T": 8189, "N": 8192, "K": 1536, "out": "bf16", "bias": False},
        # a dense layer: one decoding stream, a batch of them at another width, a long prompt
        {"name": "ffn_T1", "op": "ffn", "T": 1, "H": 1536, "I": 4096, "dtype": "bf16", "residual": True},
        {"name": "ffn_T16", "op": "ffn", "T": 16, "H": 2048, "I": 5632, "dtype": "f16", "residual": False},
        {"name": "ffn_T8189", "op": "ffn", "T": 8189, "H": 1536, "I": 4096, "dtype": "bf16", "residual": True},
        # a training step of it: a small ragged one, and a whole batch
        {"name": "ffn_train_T77", "op": "ffn_train", "T": 77, "H": 520, "I": 1048, "dtype": "f16"},
        {"name": "ffn_train_T8189", "op": "ffn_train", "T": 8189, "H": 1536, "I": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "int8", "ffn", "ffn_train"])
    dtype = rng.choice(["bf16", "f16"])
    T = _log(rng, 1, 8192)
    if op in ("norm", "norm_train"):
        H = _log(rng, 64, 8192)
        T = min(T, (8189 * 4096) // H)
        if op == "norm_train":
            return {"op": op, "T": T, "H": H, "dtype": dtype}
        return {"op": op, "T": T, "H": H, "dtype": dtype, "fmt": rng.choice(["int8", "e4m3"]),
                "group": rng.choice([0, 128])}
    if op == "int8":
        K, N = 16 * _log(rng, 4, 512), _log(rng, 64, 8192)
        T = max(1, min(T, (8189 * 8192 * 1536) // (N * K)))
        return {"op": op, "T": T, "N": N, "K": K, "out": rng.choice(["bf16", "f16", "f32"]),
                "bias": rng.choice([False, True])}
    H, I = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1024)
    T = max(1, min(T, (8189 * 1536 * 4096) // (H * I)))
    if op == "ffn":
        return {"op": op, "T": T, "H": H, "I": I, "dtype": dtype, "residual": rng.choice([False, True])}
    return {"op": op, "T": T, "H": H, "I": I, "dtype": dtype}


def _stream(T, H, g):
    """Rows of a residual stream: unit noise, rows of different size, a few channels that stand out."""
    loud = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.01).float()
    size = torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
    return torch.randn((T, H), generator=g, device="cuda") * loud * size


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op, T = case["op"], case["T"]
    st = {"case": case}
    if op in ("norm", "norm_train"):
        H, dt = case["H"], TYPES[case["dtype"]]
        st["x"] = rnd(T, H).to(dt)
        st["residual"] = _stream(T, H, g).to(dt)
        st["weight"] = (1.0 + 0.1 * rnd(H)).to(dt)
        if op == "norm_train":
            st["dy"] = rnd(T, H).to(dt)
            st["dstream"] = rnd(T, H).to(dt)
    elif op == "int8":
        N, K = case["N"], case["K"]
        a, b = rnd(T, K), 0.02 * rnd(N, K)
        st["a_scale"] = a.abs().amax(dim=1) / 127
        st["b_scale"] = b.abs().amax(dim=1) / 127
        st["a"] = torch.round(a / st["a_scale"][:, None]).to(torch.int8)
        st["b"] = torch.round(b / st["b_scale"][:, None]).to(torch.int8)
        st["bias"] = 0.1 * rnd(N) if case["bias"] else None
    else:
        H, I, dt = case["H"], case["I"], TYPES[case["dtype"]]
        st["x"] = rnd(T, H).to(dt)
        for name, shape in (("w_gate", (H, I)), ("w_up", (H, I)), ("w_down", (I, H))):
            st[name] = (0.02 * rnd(*shape)).to(dt)
        if op == "ffn":
            st["residual"] = rnd(T, H).to(dt) if case["residual"] else None
        else:
            st["dy"] = rnd(T, H).to(dt)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    return {"norm": _norm, "norm_train": _norm_train, "int8": _int8, "ffn": _ffn,
            "ffn_train": _ffn_train}[c["op"]](st, c)


def _values(q, scales, group, dtype):
    """What 8-bit codes [T, H] with their scales stand for, in the activations' type."""
    T, H = q.shape
    if q.dtype != torch.int8:
        q = q.to(dtype)  # every e4m3 value is one of bf16 and of fp16
    if group == 0:
        return torch.mul(q, scales, out=torch.empty((T, H), dtype=dtype, device=q.device))
    if H % group == 0:
        out = torch.empty((T, H // group, group), dtype=dtype, device=q.device)
        return torch.mul(q.view(out.shape), scales[:, :, None], out=out).view(T, H)
    return torch.mul(q, scales.repeat_interleave(group, dim=1)[:, :H],
                     out=torch.empty((T, H), dtype=dtype, device=q.device))


def _normed(x, residual, weight):
    """The new stream, rounded once, and the norm of what was stored, in 32 bits."""
    s = (x.float() + residual.float()).to(x.dtype)
    sf = s.float()
    rstd = torch.rsqrt((sf * sf).mean(dim=1, keepdim=True) + EPS)
    return s, sf, rstd, sf * rstd * weight.float()


def _norm(st, c):
    x, group, dt = st["x"], c["group"], TYPES[c["dtype"]]
    if own:
        from group_limited_routed_moe_b200 import moe
        s, q, scales = moe.moe_add_rmsnorm(x, st["residual"], st["weight"], EPS, out_format=c["fmt"],
                                           group=group)
        return {"stream": s, "values": _values(q, scales, group, dt), "scales": scales}
    s, _, _, y = _normed(x, st["residual"], st["weight"])
    T, H = y.shape
    top = 127.0 if c["fmt"] == "int8" else 448.0
    n = -(-H // group) if group else 1
    wide = torch.nn.functional.pad(y, (0, n * group - H)) if group else y
    scales = (wide.view(T, n, -1).abs().amax(dim=2) / top).clamp_min(2.0 ** -126)
    z = y / (scales.repeat_interleave(group, dim=1)[:, :H] if group else scales)
    q = torch.round(z).to(torch.int8) if c["fmt"] == "int8" else z.clamp(-448, 448).to(torch.float8_e4m3fn)
    return {"stream": s, "values": _values(q, scales, group, dt), "scales": scales}


def _norm_train(st, c):
    x, w, dy = st["x"], st["weight"], st["dy"]
    if own:
        from group_limited_routed_moe_b200 import moe
        s, y, _ = moe.moe_add_rmsnorm(x, st["residual"], w, EPS)
        dx, dw = moe.moe_add_rmsnorm_backward(dy, s, w, EPS, dstream=st["dstream"])
        return {"stream": s, "y": y, "dx": dx, "dweight": dw}
    s, sf, rstd, y = _normed(x, st["residual"], w)
    n, d = sf * rstd, dy.float()
    dn = d * w.float()
    dx = rstd * (dn - n * (dn * n).mean(dim=1, keepdim=True)) + st["dstream"].float()
    return {"stream": s, "y": y.to(x.dtype), "dx": dx.to(x.dtype), "dweight": (d * n).sum(dim=0)}


def _int8(st, c):
    dt = TYPES[c["out"]]
    if own:
        from group_limited_routed_moe_b200 import moe
        return moe.moe_int8_matmul(st["a"], st["a_scale"], st["b"], st["b_scale"], bias=st["bias"],
                                   out_dtype=dt)
    y = st["a"].float() @ st["b"].float().t()
    y = y * st["a_scale"][:, None] * st["b_scale"]
    return (y if st["bias"] is None else y + st["bias"]).to(dt)


def _ffn(st, c):
    x = st["x"]
    if own:
        from group_limited_routed_moe_b200 import moe
        return moe.moe_gated_ffn(x, st["w_gate"], st["w_up"], st["w_down"], residual=st["residual"])
    xf = x.float()
    g, u = xf @ st["w_gate"].float(), xf @ st["w_up"].float()
    y = (g / (1 + torch.exp(-g)) * u) @ st["w_down"].float()
    return (y if st["residual"] is None else y + st["residual"].float()).to(x.dtype)


def _ffn_train(st, c):
    x, dy, ws = st["x"], st["dy"], (st["w_gate"], st["w_up"], st["w_down"])
    if own:
        from group_limited_routed_moe_b200 import moe
        y, saved = moe.moe_gated_ffn(x, *ws, save=True)
        dx, dwg, dwu, dwd = moe.moe_gated_ffn_backward(dy, x, *ws, saved)
        return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
    dt = x.dtype
    x, dy, (wg, wu, wd) = x.float(), dy.float(), (w.float() for w in ws)
    g, u = x @ wg, x @ wu
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig
    h = a * u
    y = h @ wd
    dh = dy @ wd.t()
    dg, du = dh * u * (sig + a * (1 - sig)), dh * a
    out = {"y": y, "dx": dg @ wg.t() + du @ wu.t(), "dw_gate": x.t() @ dg, "dw_up": x.t() @ du,
           "dw_down": h.t() @ dy}
    return {k: v.to(dt) for k, v in out.items()}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_train"):
        H = case["H"]
        if op == "norm":
            n = -(-H // case["group"]) if case["group"] else 1
            return {"bytes": T * H * (2 + 2 + 2 + 1) + 4 * T * n + 2 * H, "flops": 8 * T * H}
        return {"bytes": T * H * 2 * 7 + 6 * H, "flops": 18 * T * H}
    if op == "int8":
        N, K = case["N"], case["K"]
        width = 4 if case["out"] == "f32" else 2
        return {"bytes": T * K + N * K + 4 * T + 4 * N * (2 if case["bias"] else 1) + width * T * N,
                "flops": 2 * T * N * K}
    H, I = case["H"], case["I"]
    if op == "ffn":
        return {"bytes": 2 * (T * H * (3 if case["residual"] else 2) + 3 * H * I), "flops": 6 * T * H * I}
    return {"bytes": 2 * (4 * T * H + 6 * H * I), "flops": 18 * T * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits

def _round_to(v, dtype):
    """The nearest values of a 16-bit type, ties to even, from 64 bits in one step."""
    bits, low, top = (8, -126, math.inf) if dtype == torch.bfloat16 else (11, -14, 65504.0)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=low + 1) - bits)
    r = torch.round(v / step) * step
    return torch.where(r.abs() > top, torch.sign(r) * math.inf, r)


def _e4m3(v):
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=-5) - 4)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def exact(case, seed):
    st = {k: v.double() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items()}
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_train"):
        H, w = case["H"], st["weight"]
        s = _round_to(st["x"] + st["residual"], TYPES[case["dtype"]])
        if op == "norm_train":
            s, w = s.requires_grad_(), w.requires_grad_()
        y = s * w / torch.sqrt(torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / H + EPS)
        if op == "norm_train":
            dx, dw = torch.autograd.grad(y, (s, w), st["dy"])
            return {"stream": s.detach(), "y": y.detach(), "dx": dx + st["dstream"], "dweight": dw}
        group, top = case["group"] or H, 127.0 if case["fmt"] == "int8" else 448.0
        scales = torch.stack([p.abs().amax(dim=1) for p in y.split(group, dim=1)], dim=1) / top
        per = scales[:, torch.arange(H, device=y.device) // group]
        codes = torch.round(y / per) if case["fmt"] == "int8" else _e4m3(y / per)
        return {"stream": s, "values": codes * per, "scales": scales}
    if op == "int8":
        y = torch.einsum("tk,nk->tn", st["a"], st["b"]) * torch.outer(st["a_scale"], st["b_scale"])
        return y if st["bias"] is None else y + st["bias"]
    leaves = [st[k].requires_grad_(op == "ffn_train") for k in ("x", "w_gate", "w_up", "w_down")]
    x, wg, wu, wd = leaves
    g = torch.einsum("th,hi->ti", x, wg)
    y = torch.einsum("ti,ih->th", g * torch.sigmoid(g) * torch.einsum("th,hi->ti", x, wu), wd)
    if op == "ffn":
        return y if st["residual"] is None else y + st["residual"]
    dx, dwg, dwu, dwd = torch.autograd.grad(y, leaves, st["dy"])
    return {"y": y.detach(), "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
