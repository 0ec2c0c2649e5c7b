"""An expert MLP under block scaling, from the router's logits to the tokens' outputs, sequenced over the C ABI.

  forward   route         logits -> each token's k experts, weights, rows; balance loss
            dispatch      x -> codes in the experts' rows (and in token order: the checkpoint)
            h  = rows W1^T                                      (grouped product)
            act           h -> codes of g = act(h) (and of h: the checkpoint)
            ye = g W2^T                                         (grouped product)
            combine       y[t] = sum_j weight[t,j] ye[row of (t,j)]
  backward  combine       dye = weight dy in the experts' rows, dweight = <dy, ye>
            dye -> codes along the rows and transposed
            dg = dye W2                                         (grouped product)
            dact          dg, kept h -> codes of dh along the rows and transposed, transposed codes of g
            dW2 = dye^T g,  dxr = dh W1
            recode        kept x -> transposed codes of the experts' rows
            dW1 = dh^T x
            combine       dx[t] = sum_j dxr[row of (t,j)]
            route         dlogits from dweight and the balance loss

Between the passes a token keeps its input's codes once (one byte a value, whatever k is) and, for each of
its experts, the codes of h and the bf16 result ye.  The quantisation is that of blocklinear.py (one
fp32 scale per 128 values: the just-in-time scaling of "FP8 低精度训练：Transformer Engine 简析" §三.1, per
block); the gradient of the logits leaves out that the choice of experts itself may change.

The layer keeps its outputs and codes in buffers made once: an output is valid until the next call.  It
takes any number of tokens up to `tokens`, down to a single one.  need_backward=False (serving) writes nothing that a
backward pass reads; the buffers of one are there all the same.
"""
from __future__ import annotations

import torch

from . import (ACT_GEGLU, ACT_SWIGLU, E4M3, fp8_block_act, fp8_block_dact, fp8_block_dispatch, fp8_block_gemm_grouped,
               fp8_block_gemm_grouped_wgrad, fp8_block_padded_rows, fp8_block_recode, moe_combine, moe_combine_bwd, moe_route,
               moe_route_bwd, moe_route_workspace_size)
from .blocklinear import BlockTensor, BlockWeight, _blocks


class BlockMoE:
    """w1 [E x W x H] and w2 [E x H x F], W = 2F for a gated act (ACT_SWIGLU, ACT_GEGLU; the gate's half first), else F.
    Each token goes to k experts; normalize: its weights add up to 1.  Gradients' codes are E4M3, or E5M2 with
    grad_dtype=E5M2."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, tokens: int, k: int, act: int = ACT_SWIGLU, normalize: bool = True,
                 grad_dtype: int = E4M3):
        (E, W, H), F = w1.shape, w2.shape[2]
        if tuple(w2.shape) != (E, H, F) or W != (2 * F if act >= ACT_GEGLU else F):
            raise ValueError("w1 is %s, w2 %s: w1 [E x W x H] and w2 [E x H x F] are wanted, W = %s" % (
                tuple(w1.shape), tuple(w2.shape), "2F" if act >= ACT_GEGLU else "F"))
        if not 1 <= k <= min(E, 32):
            raise ValueError("k is %d: 1 to min(experts, 32)" % k)
        self.w1, self.w2, self.act, self.normalize, self.grad_dtype = w1, w2, act, normalize, grad_dtype
        self.E, self.W, self.H, self.F, self.k, self.tokens = E, W, H, F, k, tokens
        dev, R, T = w1.device, tokens * k, fp8_block_padded_rows(tokens * k, E)
        self.w1_8, self.w2_8 = BlockWeight(w1), BlockWeight(w2)
        flat = lambda n, dtype: torch.empty(n, dtype=dtype, device=dev)  # noqa: E731
        u8, bf, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
        # the routing
        self._expert, self._position, self._token = flat(R, i32), flat(R, i32), flat(R, i32)
        self._weight, self._dweight = flat(R, f32), flat(R, f32)
        self._dlogits = flat(tokens * E * 4, u8)  # of the logits' type
        self.offsets, self.counts = flat(E + 1, i32), flat(E, i32)
        self.slope, self.loss = flat(E, f32), flat(1, f32)
        self.ws = flat(moe_route_workspace_size(tokens, E), u8)
        # kept for backward()
        self._xq, self._xs = flat(tokens * H, u8), flat(tokens * _blocks(H), f32)
        self._hq, self._hs = flat(R * W, u8), flat(R * _blocks(W), f32)
        self._ye = flat(R * H, bf)
        # used within a pass
        self._rq, self._rs = flat(R * H, u8), flat(R * _blocks(H), f32)
        self._h = flat(R * W, bf)
        self._gq, self._gs = flat(R * F, u8), flat(R * _blocks(F), f32)
        self._dye, self.dye8 = flat(R * H, bf), BlockTensor(R, H, E, dev)
        self._dhq, self._dhs, self._dht, self._dhts = flat(R * W, u8), flat(R * _blocks(W), f32), flat(T * W, u8), flat(T // 128 * W, f32)
        self._gt, self._gts = flat(T * F, u8), flat(T // 128 * F, f32)
        self._xt, self._xts = flat(T * H, u8), flat(T // 128 * H, f32)
        self._y, self._dx = flat(tokens * H, bf), flat(tokens * H, bf)
        self.dw1, self.dw2 = torch.empty(w1.shape, dtype=bf, device=dev), torch.empty(w2.shape, dtype=bf, device=dev)
        self.m = -1  # tokens of the last forward that left what a backward pass needs

    def _codes(self, q: torch.Tensor, s: torch.Tensor, rows: int, cols: int):
        return q[:rows * cols].view(rows, cols), s[:rows * _blocks(cols)].view(_blocks(cols), rows)

    def _transposed(self, q: torch.Tensor, s: torch.Tensor, T: int, cols: int):
        return q[:T * cols].view(cols, T), s[:T // 128 * cols].view(T // 128, cols)

    def forward(self, x: torch.Tensor, logits: torch.Tensor, valid: torch.Tensor | None = None, stream=None,
                is_first_microbatch=None, need_backward: bool = True) -> torch.Tensor:
        """x [T x H] (bf16 or fp32), logits [T x E] (bf16 or fp32), valid [T] (bool or uint8; zero for padding, whose rows of
        the output are zeros).  After it, `loss` holds the balance loss and `counts` every expert's tokens."""
        T, k, H, F, W = x.shape[0], self.k, self.H, self.F, self.W
        if T > self.tokens or tuple(x.shape) != (T, H) or tuple(logits.shape) != (T, self.E):
            raise ValueError("x is %s and logits %s, this layer takes up to %d tokens of %d and logits of %d experts" % (
                tuple(x.shape), tuple(logits.shape), self.tokens, H, self.E))
        self.m = -1
        R = T * k
        self.expert, self.position = self._expert[:R].view(T, k), self._position[:R].view(T, k)
        self.weight, self.token = self._weight[:R].view(T, k), self._token[:R]
        self.w1_8.quantize(self.w1, is_first_microbatch, transposed=need_backward, stream=stream)
        self.w2_8.quantize(self.w2, is_first_microbatch, transposed=need_backward, stream=stream)
        moe_route(logits, self.expert, self.weight, self.position, self.token, self.offsets, counts=self.counts, slope=self.slope,
                  loss=self.loss, workspace=self.ws, valid=valid, normalize=self.normalize, stream=stream)
        rq, rs = self._codes(self._rq, self._rs, R, H)
        xq, xs = self._codes(self._xq, self._xs, T, H) if need_backward else (None, None)
        fp8_block_dispatch(x, E4M3, self.position, rq, rs, q=xq, s=xs, stream=stream)
        h = self._h[:R * W].view(R, W)
        fp8_block_gemm_grouped(rq, E4M3, rs, self.w1_8.q, E4M3, self.w1_8.s, self.offsets, h, stream=stream)
        gq, gs = self._codes(self._gq, self._gs, R, F)
        hq, hs = self._codes(self._hq, self._hs, R, W) if need_backward else (None, None)
        fp8_block_act(h, self.act, E4M3, gq, gs, h_q=hq, h_s=hs, offsets=self.offsets, stream=stream)
        ye = self._ye[:R * H].view(R, H)
        fp8_block_gemm_grouped(gq, E4M3, gs, self.w2_8.q, E4M3, self.w2_8.s, self.offsets, ye, stream=stream)
        y = self._y[:T * H].view(T, H)
        moe_combine(ye, self.position, y, weight=self.weight, stream=stream)
        if need_backward:
            self.m, self._logits = T, logits
        return y

    def backward(self, dy: torch.Tensor, dloss: torch.Tensor | None = None, stream=None):
        """(dx, dlogits, dw1, dw2) from dy (bf16 [T x H]) and dloss (fp32 [1] on the device: the balance loss's factor in the
        whole loss).  Reads the forward's logits again: they keep their values until it has run."""
        if self.m < 0:
            raise RuntimeError("backward() needs a forward() with need_backward=True before it")
        T, k, H, F, W = self.m, self.k, self.H, self.F, self.W
        if tuple(dy.shape) != (T, H) or dy.dtype is not torch.bfloat16:
            raise ValueError("dy is %s %s, the forward pass had %d tokens of %d: bfloat16 is wanted" % (dy.dtype, tuple(dy.shape), T, H))
        if dloss is not None and (dloss.dtype is not torch.float32 or dloss.shape != (1,) or dloss.device != dy.device):
            raise ValueError("dloss must be a float32 tensor of shape (1,) on the device of dy, got %s %s on %s" % (
                dloss.dtype, tuple(dloss.shape), dloss.device))
        R, gf = T * k, self.grad_dtype
        P = fp8_block_padded_rows(R, self.E)
        ye, dye, dweight = self._ye[:R * H].view(R, H), self._dye[:R * H].view(R, H), self._dweight[:R].view(T, k)
        moe_combine_bwd(dy, ye, self.position, self.weight, dy=dye, dweight=dweight, stream=stream)
        self.m = -1  # the row results' buffer is used again below
        self.dye8.quantize(dye, gf, offsets=self.offsets, stream=stream)
        dg = self._h[:R * F].view(R, F)
        fp8_block_gemm_grouped(self.dye8.row_q, gf, self.dye8.row_s, self.w2_8.q_t, E4M3, self.w2_8.s_t, self.offsets, dg, stream=stream)
        hq, hs = self._codes(self._hq, self._hs, R, W)
        dhq, dhs = self._codes(self._dhq, self._dhs, R, W)
        dht, dhts = self._transposed(self._dht, self._dhts, P, W)
        gt, gts = self._transposed(self._gt, self._gts, P, F)
        fp8_block_dact(dg, hq, E4M3, hs, self.act, gf, dh_q=dhq, dh_s=dhs, dh_qt=dht, dh_st=dhts, g_qt=gt, g_st=gts,
                       offsets=self.offsets, stream=stream)
        fp8_block_gemm_grouped_wgrad(self.dye8.col_q, gf, self.dye8.col_s, gt, E4M3, gts, self.offsets, self.dw2, stream=stream)
        dxr = ye  # its last reader was the combination's gradient
        fp8_block_gemm_grouped(dhq, gf, dhs, self.w1_8.q_t, E4M3, self.w1_8.s_t, self.offsets, dxr, stream=stream)
        xq, xs = self._codes(self._xq, self._xs, T, H)
        xt, xts = self._transposed(self._xt, self._xts, P, H)
        fp8_block_recode(xq, E4M3, xs, E4M3, xt, xts, offsets=self.offsets, index=self.token, stream=stream)
        fp8_block_gemm_grouped_wgrad(dht, gf, dhts, xt, E4M3, xts, self.offsets, self.dw1, stream=stream)
        dx = self._dx[:T * H].view(T, H)
        moe_combine(dxr, self.position, dx, stream=stream)
        dlogits = self._dlogits.view(self._logits.dtype)[:T * self.E].view(T, self.E)
        moe_route_bwd(self._logits, self.expert, self.weight, dlogits, dweight=dweight, slope=self.slope, dloss=dloss,
                      normalize=self.normalize, stream=stream)
        return dx, dlogits, self.dw1, self.dw2
