"""Device-memory plumbing around the C ABI: move a scene's arrays into CUDA tensors, allocate the
outputs, and issue the calls in order. No arithmetic of the method happens here."""
from __future__ import annotations

import dataclasses

from . import Workspace, token_dim


@dataclasses.dataclass
class DeviceScene:
    means: "object"
    log_scales: "object"
    quats: "object"
    opac: "object"
    sh: "object"
    viewmats: "object"
    intrin: "object"
    bg: "object"
    H: int
    W: int

    @property
    def G(self):
        return int(self.means.shape[0])

    @property
    def V(self):
        return int(self.viewmats.shape[0])

    @property
    def deg(self):
        return {1: 0, 4: 1, 9: 2, 16: 3}[int(self.sh.shape[1])]


def to_device(scene, device="cuda") -> DeviceScene:
    import torch

    def t(a):
        return torch.as_tensor(a, dtype=torch.float32).contiguous().to(device)
    return DeviceScene(t(scene.means), t(scene.log_scales), t(scene.quats), t(scene.opac),
                       t(scene.sh), t(scene.viewmats), t(scene.intrin), t(scene.bg), scene.H,
                       scene.W)


@dataclasses.dataclass
class Outputs:
    img: "object"
    T: "object"
    n_contrib: "object"
    tokens: "object"


def alloc_outputs(ds: DeviceScene, device="cuda") -> Outputs:
    import torch
    V, H, W = ds.V, ds.H, ds.W
    return Outputs(torch.empty((V, H, W, 3), dtype=torch.float32, device=device),
                   torch.empty((V, H, W), dtype=torch.float32, device=device),
                   torch.empty((V, H, W), dtype=torch.int32, device=device),
                   torch.empty((ds.G, token_dim(ds.deg)), dtype=torch.float32, device=device))


def render(ws: Workspace, ds: DeviceScene, out: Outputs, stream=None) -> list[int]:
    ws.project(ds.means, ds.log_scales, ds.quats, ds.opac, ds.sh, ds.viewmats, ds.intrin, ds.H,
               ds.W, stream)
    n = ws.bin_sort(stream)
    ws.render(ds.bg, out.img, out.T, out.n_contrib, stream)
    return n


def render_and_score(ws: Workspace, ds: DeviceScene, obs, out: Outputs, lam: float = 1.0,
                     stream=None, fused: bool = True) -> list[int]:
    """Project, bin, render and score. fused: render and replay through splat_render_score (one
    kernel); otherwise splat_render, then splat_score_replay."""
    if not fused:
        n = render(ws, ds, out, stream)
        ws.score_replay(obs, out.tokens, lam, stream)
        return n
    ws.project(ds.means, ds.log_scales, ds.quats, ds.opac, ds.sh, ds.viewmats, ds.intrin, ds.H,
               ds.W, stream)
    n = ws.bin_sort(stream)
    ws.render_score(ds.bg, obs, out.img, out.T, out.n_contrib, out.tokens, lam, stream)
    return n


def render_and_backward(ws: Workspace, ds: DeviceScene, obs, out: Outputs, grads: dict,
                        stream=None) -> list[int]:
    """Render, then the renderer backward into the variants named in `grads` (raw, detached,
    support, pscale -> [G, 11 + 3d] fp32 tensors)."""
    n = render(ws, ds, out, stream)
    ws.backward(obs, ds.log_scales, ds.quats, ds.sh, stream=stream, **grads)
    return n


@dataclasses.dataclass
class FeedForward:
    """Weights of a feed-forward block: w_gate (None: no gate) and w_up [F, D], w_down [O, F]."""
    w_gate: "object"
    w_up: "object"
    w_down: "object"
    act: str = "gelu"

    def zeros_like(self) -> "FeedForward":
        import torch
        return FeedForward(None if self.w_gate is None else torch.zeros_like(self.w_gate),
                           torch.zeros_like(self.w_up), torch.zeros_like(self.w_down), self.act)


def token_features(out: Outputs, block: FeedForward, feats, stream=None):
    """The score tokens' projection (feats [G, O] from the tokens of the last score replay; the
    rendering calls are fp32, so a bf16 or fp16 block gets its tokens rounded first)."""
    import torch
    from . import ffn
    with torch.cuda.stream(stream):  # None: the current stream
        ffn(out.tokens.to(block.w_up.dtype), block.w_gate, block.w_up, block.w_down, feats,
            block.act)


@dataclasses.dataclass
class Decoded:
    """What decode_and_render keeps for its gradient: the looked-up rows [G, D] and the attributes
    [G, C], in the table's type."""
    rows: "object"
    feats: "object"


def decode_and_render(ws: Workspace, table, ids, scale: float, block: FeedForward, maps,
                      stream=None) -> Decoded:
    """Attribute maps of Gaussians that share table rows (anchors, a codebook): row ids[g] of table
    [N, D], times scale, decoded by the block to C attributes per Gaussian and composited by the
    last render into maps [V, H, W, C]."""
    import torch
    from . import ffn, lookup
    G, C = ids.shape[0], block.w_down.shape[0]
    with torch.cuda.stream(stream):  # None: the current stream
        d = Decoded(torch.empty((G, table.shape[1]), dtype=table.dtype, device=table.device),
                    torch.empty((G, C), dtype=table.dtype, device=table.device))
        lookup(table, ids, d.rows, scale)
        ffn(d.rows, block.w_gate, block.w_up, block.w_down, d.feats, block.act)
        ws.render_features(d.feats.float(), maps)
    return d


def decode_backward(ws: Workspace, ids, scale: float, block: FeedForward, d: Decoded, dmaps,
                    dtable, dblock: FeedForward, stream=None):
    """Gradients of decode_and_render with the render held, from dmaps [V, H, W, C]: into dtable
    [N, D] and the weights of dblock."""
    import torch
    from . import ffn_backward, lookup_backward
    with torch.cuda.stream(stream):
        dfeats = torch.empty(d.feats.shape, dtype=torch.float32, device=d.feats.device)
        ws.scatter(dmaps, dfeats)
        drows = torch.empty_like(d.rows)
        ffn_backward(dfeats.to(d.feats.dtype), d.rows, block.w_gate, block.w_up, block.w_down,
                     dx=drows, dw_gate=dblock.w_gate, dw_up=dblock.w_up, dw_down=dblock.w_down,
                     act=block.act)
        lookup_backward(drows, ids, dtable, scale)


def workspace_for(ds: DeviceScene, lib=None) -> Workspace:
    return Workspace(max(ds.G, 1), ds.V, ds.H, ds.W, ds.deg, lib=lib)
