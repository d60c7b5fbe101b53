"""Measured cases of the per-row operators: scaled table lookup and feed-forward block, each with
its gradient.

``run`` computes a case either in its plain form (elementary torch operations in 32 bits or more,
rounded once at the end) or, with ``own`` true, through the framework's entry points. ``exact``
gives the same outputs in 64 bits, straight from the definitions:

  lookup       out_i = s table[ids_i]                (a zero row where ids_i is outside the table)
  lookup_grad  dtable_n = s sum of dout_i over i with ids_i = n
  ffn          y = (act(x Wg^T) * (x Wu^T)) Wd^T     (no gate: act(x Wu^T) Wd^T)
  ffn_grad     dx, dWg, dWu, dWd of the same from dy
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    """The workloads behind the cases are the scenes of this repository: 4,096 Gaussians with SH
    degree 1 (token rows of 21 values), 19,456 anchors with 16 Gaussians each, 917,504 pixel-aligned
    Gaussians with SH degree 2 (rows of 36) and 5,898,240 with SH degree 3 (rows of 57); up to 64
    attribute channels are composited."""
    return [
        # one anchor's 16 Gaussians: latency alone counts
        dict(name="lookup one anchor", op="lookup", type="f32", N=19456, M=16, C=32,
             ids="anchors", masked=0.0, pad=0),
        # every Gaussian fetches its anchor's feature row
        dict(name="lookup anchors", op="lookup", type="bf16", N=19456, M=311296, C=32,
             ids="anchors", masked=0.0, pad=0),
        # pixel-aligned Gaussians take their SH rows (16 x 3) from a codebook; some have none
        dict(name="lookup codebook", op="lookup", type="f32", N=4096, M=917504, C=48,
             ids="skewed", masked=0.05, pad=0),
        # gradient of the anchors' rows: ids already in order, 16 of each
        dict(name="lookup_grad anchors", op="lookup_grad", type="f32", N=19456, M=311296, C=32,
             ids="anchors", masked=0.0, pad=0),
        # gradient of a codebook: a few rows are used by a large part of the Gaussians
        dict(name="lookup_grad codebook", op="lookup_grad", type="bf16", N=4096, M=917504, C=48,
             ids="skewed", masked=0.05, pad=0),
        # the largest scene, Gaussians in no order, 19 odd channels in rows of a wider array
        dict(name="lookup_grad scene", op="lookup_grad", type="f16", N=368640, M=5898240, C=19,
             ids="uniform", masked=0.0, pad=5),
        # one token row: latency
        dict(name="ffn one token", op="ffn", type="f32", M=1, D=57, F=256, O=64, act="gelu",
             gated=True, pad=0),
        # score tokens of the small scene to error features, without a gate, in full precision
        dict(name="ffn tokens small", op="ffn", type="f32", M=4096, D=21, F=256, O=64, act="gelu",
             gated=False, pad=0),
        # score tokens of the pixel-aligned scene in mixed precision
        dict(name="ffn tokens", op="ffn", type="bf16", M=917504, D=36, F=256, O=64, act="silu",
             gated=True, pad=0),
        # score tokens of the largest scene
        dict(name="ffn largest", op="ffn", type="bf16", M=5898240, D=57, F=128, O=64, act="silu",
             gated=True, pad=0),
        # training a decoder of anchor rows: the widest block
        dict(name="ffn_grad anchors", op="ffn_grad", type="f16", M=19456, D=128, F=512, O=128,
             act="gelu", gated=True, pad=0),
        # training the attribute decoder of every Gaussian, rows of a wider array
        dict(name="ffn_grad attributes", op="ffn_grad", type="bf16", M=311296, D=35, F=128, O=48,
             act="silu", gated=True, pad=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "ffn", "ffn_grad"])
    case = dict(op=op, type=rng.choice(["f32", "bf16", "f16"]))
    if op.startswith("lookup"):
        N, M, C = _log_int(rng, 1, 400000), _log_int(rng, 1, 5898240), _log_int(rng, 1, 512)
        M = max(1, min(M, 180000000 // C))
        case.update(N=N, M=M, C=C, ids=rng.choice(["anchors", "skewed", "uniform"]),
                    masked=rng.choice([0.0, 0.05, 0.5]), pad=rng.choice([0, 0, 3, 8]))
    else:
        M, D = _log_int(rng, 1, 1000000), _log_int(rng, 1, 128)
        F, O = _log_int(rng, 1, 1024), _log_int(rng, 1, 128)
        # at most the largest listed call's products, the gradient's factor of about 3 included
        M = max(1, min(M, 130000000000 // (F * (2 * D + O) * (3 if op == "ffn_grad" else 1))))
        M = max(1, min(M, 500000000 // F))
        case.update(M=M, D=D, F=F, O=O, act=rng.choice(["silu", "gelu"]),
                    gated=rng.random() < 0.75, pad=rng.choice([0, 0, 3, 8]))
    return case


def _rows(g, n, c, pad, dt, scale=1.0):
    """[n, c] standard normal rows of an array `pad` columns wider."""
    t = torch.empty((n, c + pad), dtype=torch.float32, device="cuda").normal_(generator=g)
    return t.mul_(scale).to(dt)[:, :c]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["type"]]
    st = dict(case=case)
    if case["op"].startswith("lookup"):
        N, M, C, pad = case["N"], case["M"], case["C"], case["pad"]
        if case["ids"] == "anchors":  # in order, about M / N of each
            ids = (torch.arange(M, device="cuda") * N).div(M, rounding_mode="floor")
            if M < N:  # a few anchors' Gaussians
                start = int(torch.randint(0, N, (1,), generator=g, device="cuda"))
                ids = (torch.arange(M, device="cuda") // 16 + start) % N
        elif case["ids"] == "skewed":
            u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
            ids = (u ** 4 * N).long().clamp_(max=N - 1)
        else:
            ids = torch.randint(0, N, (M,), generator=g, device="cuda")
        if case["masked"]:
            off = torch.rand(M, generator=g, device="cuda") < case["masked"]
            ids = torch.where(off, torch.full_like(ids, -1), ids)
        st["ids"] = ids.to(torch.int32)
        st["scale"] = math.sqrt(C)
        if case["op"] == "lookup":
            st["table"] = _rows(g, N, C, pad, dt, 0.1)
            st["out"] = torch.empty((M, C), dtype=dt, device="cuda")
        else:
            st["dout"] = _rows(g, M, C, pad, dt)
            st["dtable"] = torch.empty((N, C), dtype=dt, device="cuda")
        return st
    M, D, F, O, pad = case["M"], case["D"], case["F"], case["O"], case["pad"]
    st["x"] = _rows(g, M, D, pad, dt)
    st["w_gate"] = _rows(g, F, D, 0, dt, D ** -0.5) if case["gated"] else None
    st["w_up"] = _rows(g, F, D, 0, dt, D ** -0.5)
    st["w_down"] = _rows(g, O, F, 0, dt, F ** -0.5)
    if case["op"] == "ffn":
        st["y"] = torch.empty((M, O), dtype=dt, device="cuda")
    else:
        st["dy"] = _rows(g, M, O, pad, dt)
        for k in ("x", "w_gate", "w_up", "w_down"):
            st["d" + k] = None if st[k] is None else torch.empty(
                st[k].shape, dtype=dt, device="cuda")
    return st


def _act(a, kind):
    """(act(a), act'(a)) in a's type."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
    return a * cdf, cdf + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain(st):
    case = st["case"]
    dt = _TYPES[case["type"]]
    if case["op"] == "lookup":
        ids = st["ids"].long()
        ok = (ids >= 0) & (ids < case["N"])
        rows = st["table"].float()[torch.where(ok, ids, 0)] * st["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(dt)
    if case["op"] == "lookup_grad":
        ids = st["ids"].long()
        ok = (ids >= 0) & (ids < case["N"])
        # long sums: in 64 bits; row N takes what belongs to no row
        acc = torch.zeros((case["N"] + 1, case["C"]), dtype=torch.float64, device="cuda")
        acc.index_add_(0, torch.where(ok, ids, case["N"]), st["dout"].double())
        return (acc[:-1] * st["scale"]).to(dt)
    x, wu, wd = st["x"].float(), st["w_up"].float(), st["w_down"].float()
    u = x @ wu.T
    if case["gated"]:
        wg = st["w_gate"].float()
        f, df = _act(x @ wg.T, case["act"])
        h = f * u
    else:
        h, df = _act(u, case["act"])
    if case["op"] == "ffn":
        return (h @ wd.T).to(dt)
    dy = st["dy"].float()
    dh = dy @ wd
    out = dict(dw_down=(dy.T @ h).to(dt))
    if case["gated"]:
        da, du = dh * u * df, dh * f
        out.update(dx=(da @ wg + du @ wu).to(dt), dw_gate=(da.T @ x).to(dt),
                   dw_up=(du.T @ x).to(dt))
    else:
        du = dh * df
        out.update(dx=(du @ wu).to(dt), dw_up=(du.T @ x).to(dt))
    return out


def run(state):
    if not own:
        return _plain(state)
    import gaussian_splatting_raster_b200 as P
    case = state["case"]
    if case["op"] == "lookup":
        P.lookup(state["table"], state["ids"], state["out"], scale=state["scale"])
        return state["out"]
    if case["op"] == "lookup_grad":
        P.lookup_backward(state["dout"], state["ids"], state["dtable"], scale=state["scale"])
        return state["dtable"]
    w = (state["w_gate"], state["w_up"], state["w_down"])
    if case["op"] == "ffn":
        P.ffn(state["x"], *w, state["y"], act=case["act"])
        return state["y"]
    P.ffn_backward(state["dy"], state["x"], *w, dx=state["dx"], dw_gate=state["dw_gate"],
                   dw_up=state["dw_up"], dw_down=state["dw_down"], act=case["act"])
    return {k: state[k] for k in ("dw_down", "dx", "dw_gate", "dw_up") if state[k] is not None}


def work(case):
    e = 4 if case["type"] == "f32" else 2
    M = case["M"]
    if case["op"].startswith("lookup"):
        N, C = case["N"], case["C"]
        read, written = (min(N, M), M) if case["op"] == "lookup" else (M, N)
        return {"bytes": 4 * M + e * C * (read + written), "flops": C * M}
    D, F, O = case["D"], case["F"], case["O"]
    two = 2 if case["gated"] else 1
    weights = F * (two * D + O)
    if case["op"] == "ffn":
        return {"bytes": e * (M * (D + O) + weights), "flops": 2 * M * weights}
    # a and u again, dh, dx, the weights' gradients
    return {"bytes": e * (M * (2 * D + O) + 2 * weights),
            "flops": 2 * M * F * (3 * two * D + 2 * O)}


def _sigma(kind, a):
    """act and its derivative from the error function and the logistic function of torch, in 64
    bits."""
    if kind == "silu":
        s = torch.sigmoid(a)
        return s * a, s + a * s * torch.sigmoid(-a)
    p = torch.special.ndtr(a)
    return p * a, p + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lookup":
        ids = st["ids"].cpu().long()
        table = st["table"].cpu().double()
        out = torch.zeros((case["M"], case["C"]), dtype=torch.float64)
        ok = torch.nonzero((ids >= 0) & (ids < case["N"]))[:, 0]
        out[ok] = table.index_select(0, ids[ok]) * st["scale"]
        return out
    if case["op"] == "lookup_grad":
        # running sums over the rows in the order of their ids, read at each id's ends
        order = torch.argsort(st["ids"], stable=True)
        ids = st["ids"][order].long()
        sums = torch.zeros((case["M"] + 1, case["C"]), dtype=torch.float64, device="cuda")
        torch.cumsum(st["dout"][order].double(), 0, out=sums[1:])
        n = torch.arange(case["N"], device="cuda")
        lo, hi = torch.searchsorted(ids, n), torch.searchsorted(ids, n, right=True)
        return (sums[hi] - sums[lo]) * st["scale"]
    wg = None if st["w_gate"] is None else st["w_gate"].double()
    wu, wd = st["w_up"].double(), st["w_down"].double()
    ys, dxs = [], []
    dwg = torch.zeros_like(wu)
    dwu, dwd = torch.zeros_like(wu), torch.zeros_like(wd)
    step = max(1, (1 << 27) // case["F"])
    for r in range(0, case["M"], step):
        x = st["x"][r:r + step].double()
        u = x.matmul(wu.t())
        a = u if wg is None else x.matmul(wg.t())
        f, df = _sigma(case["act"], a)
        up = torch.ones_like(u) if wg is None else u
        if case["op"] == "ffn":
            ys.append((f * up).matmul(wd.t()))
            continue
        dy = st["dy"][r:r + step].double()
        dh = dy.matmul(wd)
        da = dh * df * up
        dwd += dy.t().matmul(f * up)
        if wg is None:
            dxs.append(da.matmul(wu))
            dwu += da.t().matmul(x)
        else:
            du = dh * f
            dxs.append(da.matmul(wg) + du.matmul(wu))
            dwg += da.t().matmul(x)
            dwu += du.t().matmul(x)
    if case["op"] == "ffn":
        return torch.cat(ys)
    out = dict(dw_down=dwd, dx=torch.cat(dxs), dw_gate=dwg, dw_up=dwu)
    if wg is None:
        del out["dw_gate"]
    return out
