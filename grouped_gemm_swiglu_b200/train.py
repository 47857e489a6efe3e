"""The expert layer with its gradient: one training pass over the library's calls.

    layer = MoETraining(dims, w1, w2, expert_drop=0.1)
    out, saved = layer.forward(logits, x, rng=rng)
    grads = layer.backward(saved, dout)        # dx, dlogits, dw1, dw2

Forward: moe_route_topk, moe_permute, moe_ffn_forward, moe_combine, and moe_dropout where
dropout of the output or a residual sum is wanted. Backward: the same steps in reverse.
Everything runs on torch's current stream and is capturable in a CUDA graph; nothing is
read back by the host.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from ._lib import (MOE_WDTYPE_BF16, MOE_WS_COMBINE, MOE_WS_FFN_BACKWARD, MOE_WS_FFN_FORWARD, MOE_WS_PERMUTE, MoeDims,
                   alloc_workspace, moe_combine, moe_combine_backward, moe_dropout, moe_ffn_backward, moe_ffn_forward,
                   moe_permute, moe_read_status, moe_route_topk)


@dataclass
class MoESaved:
    """What a forward pass keeps for its backward pass."""
    dims: MoeDims
    logits: torch.Tensor
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    shared_w: torch.Tensor | None
    offsets: torch.Tensor
    inv_perm: torch.Tensor
    x_perm: torch.Tensor
    gu: torch.Tensor
    h: torch.Tensor
    y: torch.Tensor
    rng: torch.Tensor | None


class MoETraining:
    """A bf16 expert layer that is trained: w1 [G,2I,H] and w2 [G,H,I] belong to the caller (an
    optimiser may change them between passes), workspaces for `max_tokens` tokens to this object.

    There is no autograd function: `out` has no grad_fn, whether or not an input requires a
    gradient, and the gradients are what backward() returns.

    gate_scale, up_scale, limits: optional fp32 [G]; router_bias: optional fp32 [E] (sigmoid
    scoring; it ranks only and has no gradient). expert_drop drops elements of the experts'
    activation h, out_drop elements of the layer's output before the residual sum; both draw
    their masks from `rng` int64 [2, 2] on the device, {seed, offset} of the experts' and of the
    output's mask, which the caller changes from pass to pass (in place, for a captured graph)
    and leaves alone between a forward pass and its backward pass.

    One pass at a time uses an object: passes that overlap on the GPU (other streams, other
    graphs) need objects of their own, which may share the weights.
    """

    def __init__(self, dims: MoeDims, w1, w2, gate_scale=None, up_scale=None, limits=None, router_bias=None,
                 max_tokens: int | None = None, expert_drop: float = 0.0, out_drop: float = 0.0):
        if dims.wdtype != MOE_WDTYPE_BF16:
            raise ValueError("MoETraining: bf16 layers only")
        self.dims, self.w1, self.w2 = dims, w1, w2
        self.gate_scale, self.up_scale, self.limits, self.router_bias = gate_scale, up_scale, limits, router_bias
        self.max_tokens = dims.T if max_tokens is None else max_tokens
        self.expert_drop, self.out_drop = expert_drop, out_drop
        sized = self._dims(self.max_tokens)
        kinds = (MOE_WS_PERMUTE, MOE_WS_FFN_FORWARD, MOE_WS_FFN_BACKWARD, MOE_WS_COMBINE)
        self.ws = {kind: alloc_workspace(sized, kind, device=w1.device) for kind in kinds}
        # dx of a token is the plain sum over its copies
        self.ones = torch.ones((self.max_tokens, dims.k), device=w1.device)
        self.sink_ones = torch.ones((self.max_tokens, dims.n_sink), device=w1.device) if dims.n_sink else None

    def _dims(self, T: int) -> MoeDims:
        d = MoeDims.from_buffer_copy(self.dims)
        d.T = T
        return d

    def _rngs(self, rng):
        if self.expert_drop == 0.0 and self.out_drop == 0.0:
            return None, None
        if rng is None or rng.shape != (2, 2) or rng.dtype != torch.int64:
            raise ValueError("MoETraining: dropout needs rng, int64 [2, 2]: {seed, offset} of the experts' and the output's mask")
        return (rng[0] if self.expert_drop else None), (rng[1] if self.out_drop else None)

    def _check_inputs(self, *tensors) -> None:
        """What the routing and permuting calls, which take addresses on trust, are handed."""
        for name, t, dtype, shape in tensors:
            if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != self.w1.device):
                raise ValueError(f"MoETraining.forward: {name} must be a contiguous {dtype} tensor of shape {shape} on {self.w1.device}")

    def forward(self, logits, x, residual=None, rng=None):
        """out [T,H] bf16 (plus residual where one is given), and what backward() needs. `logits` and
        the weights must still hold the same values then."""
        T, dev, bf = x.shape[0], x.device, torch.bfloat16
        if T > self.max_tokens:
            raise ValueError(f"T={T} exceeds the workspace size ({self.max_tokens} tokens)")
        d = self._dims(T)
        self._check_inputs(("logits", logits, torch.float32, (T, d.E + d.n_sink)), ("x", x, bf, (T, d.H)),
                           ("residual", residual, bf, (T, d.H)), ("router_bias", self.router_bias, torch.float32, (d.E,)))
        r_exp, r_out = self._rngs(rng)
        A, k = d.A, d.k
        with torch.cuda.device(dev):
            i32 = dict(dtype=torch.int32, device=dev)
            ids, inv = torch.empty((T, k), **i32), torch.empty((T, k), **i32)
            offsets, perm = torch.empty(d.G + 1, **i32), torch.empty(A, **i32)
            w = torch.empty((T, k), device=dev)
            sw = torch.empty((T, d.n_sink), device=dev) if d.n_sink else None
            xp, gu, h, y = (torch.empty((A, n), dtype=bf, device=dev) for n in (d.H, 2 * d.I, d.I, d.H))
            out = torch.empty((T, d.H), dtype=bf, device=dev)
            moe_route_topk(logits, d, self.router_bias, ids, w, sw)
            moe_permute(ids, x, d, offsets, perm, inv, xp, None, self.ws[MOE_WS_PERMUTE])
            moe_ffn_forward(xp, offsets, self.w1, self.gate_scale, self.up_scale, self.limits, self.w2, self.expert_drop,
                            r_exp, d, gu, h, y, self.ws[MOE_WS_FFN_FORWARD])
            moe_combine(y, offsets, inv, w, sw, d, out, self.ws[MOE_WS_COMBINE])
            if self.out_drop or residual is not None:
                moe_dropout(out, residual, out, self.out_drop, r_out)
        return out, MoESaved(d, logits, ids, w, sw, offsets, inv, xp, gu, h, y, rng)

    def backward(self, saved: MoESaved, dout):
        """Gradients of a forward pass: dx [T,H], dlogits [T,E+n_sink] (fp32), dw1, dw2. The residual's is dout."""
        d, dev = saved.dims, dout.device
        r_exp, r_out = self._rngs(saved.rng)
        with torch.cuda.device(dev):
            if self.out_drop:
                dropped = torch.empty_like(dout)
                moe_dropout(dout, None, dropped, self.out_drop, r_out)
                dout = dropped
            dy, dxp = torch.empty_like(saved.y), torch.empty_like(saved.x_perm)
            dw = torch.empty_like(saved.topk_w)
            dsw = torch.empty_like(saved.shared_w) if d.n_sink else None
            dlogits = torch.empty_like(saved.logits)
            dx = torch.empty_like(dout)
            dw1, dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
            moe_combine_backward(dout, saved.y, saved.offsets, saved.inv_perm, saved.topk_ids, saved.topk_w, saved.shared_w,
                                 saved.logits, d, dy, dw, dsw, dlogits, self.ws[MOE_WS_COMBINE])
            moe_ffn_backward(dy, saved.x_perm, saved.gu, saved.h, saved.offsets, self.w1, self.gate_scale, self.up_scale,
                             self.limits, self.w2, self.expert_drop, r_exp, d, dxp, dw1, dw2, self.ws[MOE_WS_FFN_BACKWARD])
            moe_combine(dxp, saved.offsets, saved.inv_perm, self.ones[:d.T], self.sink_ones[:d.T] if d.n_sink else None, d,
                        dx, self.ws[MOE_WS_COMBINE])
        return dict(dx=dx, dlogits=dlogits, dw1=dw1, dw2=dw2)

    def status(self) -> int:
        """The first device-side error of the passes so far (MOE_OK if none). Synchronises."""
        return next((s for s in map(moe_read_status, self.ws.values()) if s), 0)
