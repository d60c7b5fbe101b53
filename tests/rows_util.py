"""The per-row operators in 64 bits, with bounds on what rounding may do to a kernel's result.

u is half a step of a type relative to the value (2^-24 fp32, 2^-8 bf16, 2^-11 fp16). A kernel's
fp32 sum of n terms is off by at most n ACC times the sum of the terms' magnitudes; ACC = 2^-23
allows accumulators that truncate. Activations are off by 1.13 times (the largest slope of silu and
gelu) what their argument is, plus a few fp32 roundings of their own; slopes by 0.8 times (the
largest curvature) plus the same. Values held in the type between products (hidden values and
their gradients) and results are off by u more, or by half of fp16's smallest step. Each bound is
the sum of these, carried through the formulas in magnitudes.
"""
import math

import torch

U32 = 2.0 ** -24
ACC = 2.0 ** -23
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def act(a, kind):
    """act, act' in 64 bits."""
    if kind == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    p = torch.special.ndtr(a)
    return a * p, p + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)


def _held(v, e, dt):
    """Bound after rounding a value v known to e to the type."""
    return e + U[dt] * (v.abs() + e) + TINY[dt]


def lookup_ref(table, ids, scale):
    t, ids = table.double(), ids.long()
    ok = (ids >= 0) & (ids < t.shape[0])
    out = torch.zeros((ids.shape[0], t.shape[1]), dtype=torch.float64)
    out[ok] = t[ids[ok]] * scale
    dt = table.dtype
    return out, _held(out, U32 * out.abs(), dt)


def lookup_grad_ref(dout, ids, N, scale):
    d, ids = dout.double(), ids.long()
    ok = (ids >= 0) & (ids < N)
    out = torch.zeros((N, d.shape[1]), dtype=torch.float64)
    mag, cnt = torch.zeros_like(out), torch.zeros(N, dtype=torch.float64)
    out.index_add_(0, ids[ok], d[ok])
    mag.index_add_(0, ids[ok], d[ok].abs())
    cnt.index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    out, mag = out * scale, mag * abs(scale)
    return out, _held(out, (cnt[:, None] + 1) * U32 * mag, dout.dtype)


def ffn_ref(x, wg, wu, wd, kind, dy=None):
    """{name: (value, bound)} for y, and for the gradients when dy is given."""
    dt = x.dtype
    x, wu, wd = x.double(), wu.double(), wd.double()
    M, D = x.shape
    F, O = wu.shape[0], wd.shape[0]
    u = x @ wu.T
    eu = D * ACC * (x.abs() @ wu.abs().T)
    if wg is None:
        a, ea = u, eu
    else:
        wg = wg.double()
        a = x @ wg.T
        ea = D * ACC * (x.abs() @ wg.abs().T)
    f, s = act(a, kind)
    ef = 1.13 * ea + 8 * U32 * a.abs() * (1 + a.abs())
    es = 0.8 * ea + 8 * U32 * (1 + a.abs()) ** 2
    if wg is None:
        h, eh = f, ef
    else:
        h = f * u
        eh = ef * u.abs() + f.abs() * eu + ef * eu + U32 * h.abs()
    eh = _held(h, eh, dt)
    y = h @ wd.T
    ey = eh @ wd.abs().T + F * ACC * ((h.abs() + eh) @ wd.abs().T)
    out = {"y": (y, _held(y, ey, dt))}
    if dy is None:
        return out
    dy = dy.double()
    dh = dy @ wd
    edh = O * ACC * (dy.abs() @ wd.abs())
    up, eup = (torch.ones_like(u), 0.0) if wg is None else (u, eu)
    da = dh * up * s
    eda = ((edh + dh.abs()) * (up.abs() + eup) * (s.abs() + es) - da.abs()).clamp_min(0)
    eda = _held(da, eda + 3 * U32 * da.abs(), dt)
    dwd = dy.T @ h
    ewd = dy.abs().T @ eh + M * ACC * (dy.abs().T @ (h.abs() + eh))
    out["dw_down"] = (dwd, _held(dwd, ewd, dt))

    def weight(d, ed):
        v = d.T @ x
        e = ed.T @ x.abs() + M * ACC * ((d.abs() + ed).T @ x.abs())
        return v, _held(v, e, dt)

    if wg is None:
        dx = da @ wu
        edx = eda @ wu.abs() + F * ACC * ((da.abs() + eda) @ wu.abs())
        out["dw_up"] = weight(da, eda)
    else:
        du = dh * f
        edu = ((edh + dh.abs()) * (f.abs() + ef) - du.abs()).clamp_min(0)
        edu = _held(du, edu + U32 * du.abs(), dt)
        dx = da @ wg + du @ wu
        edx = (eda @ wg.abs() + edu @ wu.abs()
               + 2 * F * ACC * ((da.abs() + eda) @ wg.abs() + (du.abs() + edu) @ wu.abs()))
        out["dw_gate"] = weight(da, eda)
        out["dw_up"] = weight(du, edu)
    out["dx"] = (dx, _held(dx, edx, dt))
    return out


def close(got, ref, what=""):
    value, bound = ref
    err = (got.detach().cpu().double() - value).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"
    return worst
