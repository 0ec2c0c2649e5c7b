"""Linear layers under block scaling (one fp32 scale per 128 values), sequenced over the C ABI.

Activations and gradients are quantised in blocks of 128 along their GEMM's reduction axis,
weights in 128 x 128 blocks, each from its own values: no amax history and no delay (the
just-in-time scaling of "FP8 低精度训练：Transformer Engine 简析" §三.1, per block).

  BlockLinear    forward   Y[M,N]  = X_row W^T + b
                 backward  dX[M,K] = dY_row W          (the weight's transposed codes)
                           dW[N,K] = dY_col X_col^T    (blocks along the tokens)
                           db      = column sums of dY, in the pass that quantises it
  BlockExperts   the same per group of rows: row m of group g meets weight g (an expert layer's
                 tokens, sorted by expert).  offsets (int32 [G + 1], on the device) hold each
                 group's first row; groups may be empty, and the host never reads them.

Both take any number of rows up to `tokens`, down to a single one, and keep their outputs and
codes in buffers made once: an output is valid until the next call.  need_backward=False
(serving) quantises the input row-wise only.

Micro-batching (te modules' is_first_microbatch): forward(..., is_first_microbatch=True)
quantises the weight and keeps its codes; later micro-batches (False) reuse them.  None (the
default) quantises the weight at every forward.  Gradients are E4M3, or E5M2 with
grad_dtype=E5M2 (the HYBRID recipe's choice).
"""
from __future__ import annotations

import torch

from . import (E4M3, fp8_block_gemm, fp8_block_gemm_grouped, fp8_block_gemm_grouped_wgrad, fp8_block_padded_rows,
               fp8_block_quantize, fp8_block_quantize_weight, fp8_cast_workspace_size)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _torch_stream(stream):
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


class BlockTensor:
    """Row-wise and transposed codes and factors of activations of up to `rows` rows; the views row_q, row_s, col_q,
    col_s are those of the last call."""

    def __init__(self, rows: int, cols: int, groups: int, device):
        T = fp8_block_padded_rows(rows, groups)
        self.rows, self.cols, self.groups = rows, cols, groups
        self._rq = torch.empty(rows * cols, dtype=torch.uint8, device=device)
        self._cq = torch.empty(T * cols, dtype=torch.uint8, device=device)
        self._rs = torch.empty(rows * _blocks(cols), device=device)
        self._cs = torch.empty(T // 128 * cols, device=device)

    def quantize(self, x: torch.Tensor, dtype: int, colwise=True, offsets=None, dbias=None, workspace=None,
                 stream=None) -> None:
        m, c, T = x.shape[0], self.cols, fp8_block_padded_rows(x.shape[0], self.groups)
        if m > self.rows or x.shape[1] != c:
            raise ValueError("x is %s, this layer takes up to %d rows of %d" % (tuple(x.shape), self.rows, c))
        self.row_q, self.row_s = self._rq[:m * c].view(m, c), self._rs[:m * _blocks(c)].view(_blocks(c), m)
        self.col_q, self.col_s = self._cq[:c * T].view(c, T), self._cs[:T // 128 * c].view(T // 128, c)
        fp8_block_quantize(x, dtype, row_q=self.row_q, row_s=self.row_s, col_q=self.col_q if colwise else None,
                           col_s=self.col_s if colwise else None, offsets=offsets, dbias=dbias, workspace=workspace,
                           stream=stream)


class BlockWeight:
    """Codes and factors of weights [N x K] or [E x N x K], and their transposed copies."""

    def __init__(self, w: torch.Tensor):
        lead, (n, k) = tuple(w.shape[:-2]), w.shape[-2:]
        u8, f32 = dict(dtype=torch.uint8, device=w.device), dict(device=w.device)
        self.q, self.s = torch.empty(lead + (n, k), **u8), torch.empty(lead + (_blocks(k), _blocks(n)), **f32)
        self.q_t, self.s_t = torch.empty(lead + (k, n), **u8), torch.empty(lead + (_blocks(n), _blocks(k)), **f32)
        self.cached = False

    def quantize(self, w: torch.Tensor, is_first_microbatch, transposed=True, stream=None) -> None:
        if is_first_microbatch is False and not self.cached:
            raise RuntimeError("is_first_microbatch=False, but no codes of the weight are cached: quantise it first "
                               "with is_first_microbatch=True")
        if is_first_microbatch is not False:
            keep = transposed or bool(is_first_microbatch)  # kept codes serve later backward passes too
            fp8_block_quantize_weight(w, E4M3, q=self.q, s=self.s, q_t=self.q_t if keep else None,
                                      s_t=self.s_t if keep else None, stream=stream)
            self.cached = bool(is_first_microbatch)


class _BlockLayer:
    def __init__(self, weight: torch.Tensor, tokens: int, groups: int, out_dtype, grad_dtype: int):
        self.w, self.N, self.K = weight, weight.shape[-2], weight.shape[-1]
        self.tokens, self.grad_dtype = tokens, grad_dtype
        dev = weight.device
        self.x8, self.dy8 = BlockTensor(tokens, self.K, groups, dev), BlockTensor(tokens, self.N, groups, dev)
        self.w8 = BlockWeight(weight)
        self._y = torch.empty(tokens * self.N, dtype=out_dtype, device=dev)
        self._dx = torch.empty(tokens * self.K, dtype=torch.bfloat16, device=dev)
        self.dw = torch.empty(weight.shape, dtype=torch.bfloat16, device=dev)
        self.m = -1  # rows of the last forward that left its codes for a backward pass

    def _check_dy(self, dy: torch.Tensor) -> None:
        if self.m < 0:
            raise RuntimeError("backward() needs a forward() with need_backward=True before it")
        if dy.shape[0] != self.m:
            raise ValueError("dy has %d rows, the forward pass had %d" % (dy.shape[0], self.m))


class BlockLinear(_BlockLayer):
    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None, tokens: int, out_dtype=torch.bfloat16,
                 grad_dtype: int = E4M3):
        super().__init__(weight, tokens, 0, out_dtype, grad_dtype)
        self.b = bias
        self.db = torch.empty(self.N, device=weight.device) if bias is not None else None
        self.ws = (torch.empty(fp8_cast_workspace_size(tokens, self.N), dtype=torch.uint8, device=weight.device)
                   if bias is not None else None)

    def forward(self, x: torch.Tensor, stream=None, is_first_microbatch=None, need_backward=True) -> torch.Tensor:
        self.m = -1
        self.w8.quantize(self.w, is_first_microbatch, transposed=need_backward, stream=stream)
        self.x8.quantize(x, E4M3, colwise=need_backward, stream=stream)
        y = self._y[:x.shape[0] * self.N].view(x.shape[0], self.N)
        fp8_block_gemm(self.x8.row_q, E4M3, self.x8.row_s, self.w8.q, E4M3, self.w8.s, y, bias=self.b, stream=stream)
        self.m = x.shape[0] if need_backward else -1
        return y

    def backward(self, dy: torch.Tensor, stream=None):
        self._check_dy(dy)
        self.dy8.quantize(dy, self.grad_dtype, dbias=self.db, workspace=self.ws, stream=stream)
        dx = self._dx[:self.m * self.K].view(self.m, self.K)
        fp8_block_gemm(self.dy8.row_q, self.grad_dtype, self.dy8.row_s, self.w8.q_t, E4M3, self.w8.s_t, dx, stream=stream)
        if self.m:
            fp8_block_gemm(self.dy8.col_q, self.grad_dtype, self.dy8.col_s, self.x8.col_q, E4M3, self.x8.col_s, self.dw,
                           stream=stream)
        else:  # no rows: a sum over nothing
            with torch.cuda.stream(_torch_stream(stream)):
                self.dw.zero_()
        return dx, self.dw, self.db


class BlockExperts(_BlockLayer):
    """weight [G x N x K]; x's rows sorted by group.  Rows outside the groups keep what the output buffers held.
    backward() reads the forward's offsets again: they keep their values until it has run.  The products are laid out
    for all of x's rows, since the host does not know how many the groups hold."""

    def __init__(self, weight: torch.Tensor, tokens: int, out_dtype=torch.bfloat16, grad_dtype: int = E4M3):
        super().__init__(weight, tokens, weight.shape[0], out_dtype, grad_dtype)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, stream=None, is_first_microbatch=None,
                need_backward=True) -> torch.Tensor:
        self.m = -1
        self.w8.quantize(self.w, is_first_microbatch, transposed=need_backward, stream=stream)
        self.x8.quantize(x, E4M3, colwise=need_backward, offsets=offsets, stream=stream)
        y = self._y[:x.shape[0] * self.N].view(x.shape[0], self.N)
        fp8_block_gemm_grouped(self.x8.row_q, E4M3, self.x8.row_s, self.w8.q, E4M3, self.w8.s, offsets, y, stream=stream)
        if need_backward:
            self.m, self.offsets = x.shape[0], offsets
        return y

    def backward(self, dy: torch.Tensor, stream=None):
        self._check_dy(dy)
        self.dy8.quantize(dy, self.grad_dtype, offsets=self.offsets, stream=stream)
        dx = self._dx[:self.m * self.K].view(self.m, self.K)
        fp8_block_gemm_grouped(self.dy8.row_q, self.grad_dtype, self.dy8.row_s, self.w8.q_t, E4M3, self.w8.s_t, self.offsets,
                               dx, stream=stream)
        fp8_block_gemm_grouped_wgrad(self.dy8.col_q, self.grad_dtype, self.dy8.col_s, self.x8.col_q, E4M3, self.x8.col_s,
                                     self.offsets, self.dw, stream=stream)
        return dx, self.dw
