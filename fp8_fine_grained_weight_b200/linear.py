"""A linear layer whose three GEMMs run in FP8 through the library's C ABI.

the-good.kr wr_id=2169793 para 3: the forward pass (Fprop), the activation gradient
(Dgrad) and the weight gradient (Wgrad) of a linear layer all run as FP8 GEMMs;
para 2 of the same post: an FP8 Wgrad lets the activations be cached in FP8 for the
backward pass.  With Y = X W^T (X [T, K] tokens x channels, W [N, K]):

  Fprop  Y  [T, N] = X W^T      A = X  (1x128 along K),  B = W    (128x128 blocks)
  Dgrad  dX [T, K] = dY W       A = dY (1x128 along N),  B = W^T  (128x128 blocks)
  Wgrad  dW [N, K] = dY^T X     A = dY^T (1x128 along T), B = X^T (1x128 along T)

Every operand is produced by the library's kernels: quant_act_dual reads X (forward) and
dY (backward) once and emits both their row and their transposed 1x128 copies;
transpose_blocks turns the 128x128 codes of W into those of W^T.  Only the FP8 copies
of X^T and of W are kept for the backward pass.  With power-of-two scales the GEMMs
apply the scales in the tensor core (gemm_blockscaled_ue8m0), otherwise they promote per
128-K group.  T, K and N must be multiples of 128.  X, W, Y, dX and dW are bf16 (the GEMM
epilogues round to bf16; the Wgrad GEMM accumulates over all T in FP32 first).

The gated layer computes H = silu(X Wg^T) * (X Wu^T) from one stacked weight W [2N, K]
(the gate's N rows, then the up projection's):

  Fprop  H  [T, N]  both products, the activation and their product in one kernel; with
                    gradients, g and u are kept in bf16
  D = [dg | du] [T, 2N]  gated_backward_quant: the elementwise gradient, quantized both ways
  Dgrad  dX [T, K] = D W       A = D (1x128 along 2N),   B = W^T (128x128 blocks)
  Wgrad  dW [2N, K] = D^T X    A = D^T (1x128 along T),  B = X^T (1x128 along T)

Any T (the products over T run on T rounded up to 128, with zero rows); K and N multiples
of 128.
"""
from typing import Optional

import torch

from . import (gated_backward_quant, gemm_blockscaled, gemm_blockscaled_gated, gemm_blockscaled_ue8m0,
               quant_act_1x128, quant_act_dual, quant_weight_128x128, transpose_blocks, workspace_bytes)


def _gemm(pow2: bool):
    return gemm_blockscaled_ue8m0 if pow2 else gemm_blockscaled


class FP8LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
        qx, sx, qxt, sxt = quant_act_dual(x.contiguous(), pow2)
        qw, sw = quant_weight_128x128(w.contiguous(), pow2)
        y = _gemm(pow2)(qx, sx, qw, sw, out_dtype=torch.bfloat16)
        ctx.save_for_backward(qxt, sxt, qw, sw)
        ctx.pow2 = pow2
        return y

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        qxt, sxt, qw, sw = ctx.saved_tensors
        pow2 = ctx.pow2
        gemm = _gemm(pow2)
        qdy, sdy, qdyt, sdyt = quant_act_dual(dy.to(torch.bfloat16).contiguous(), pow2)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            qwt, swt = transpose_blocks(qw, sw)
            dx = gemm(qdy, sdy, qwt, swt, out_dtype=torch.bfloat16)
        if ctx.needs_input_grad[1]:
            dw = gemm(qdyt, sdyt, qxt, sxt, out_dtype=torch.bfloat16, b_rowwise=True)
        return dx, dw, None


def fp8_linear(x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
    """Y = X W^T with FP8 Fprop / Dgrad / Wgrad (see the module docstring)."""
    return FP8LinearFunction.apply(x, w, pow2)


class FP8Linear(torch.nn.Module):
    """nn.Linear without bias whose forward and backward GEMMs run in FP8."""

    def __init__(self, in_features: int, out_features: int, pow2: bool = False,
                 device: Optional[torch.device] = None):
        super().__init__()
        self.pow2 = pow2
        self.weight = torch.nn.Parameter(
            torch.empty((out_features, in_features), dtype=torch.bfloat16, device=device))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fp8_linear(x, self.weight, self.pow2)


def _product(qa, sa, qb, sb, pow2: bool, b_rowwise: bool = False) -> torch.Tensor:
    """A gradient product.  The promoted GEMM's split-K workspace is this call's own: the
    buffer cached per stream would be shared by graphs captured on that stream."""
    if pow2:
        return gemm_blockscaled_ue8m0(qa, sa, qb, sb, out_dtype=torch.bfloat16, b_rowwise=b_rowwise)
    with torch.cuda.device(qa.device):
        need = workspace_bytes(qa.shape[0], qb.shape[0], qa.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device=qa.device) if need else None
    return gemm_blockscaled(qa, sa, qb, sb, out_dtype=torch.bfloat16, b_rowwise=b_rowwise,
                            split_k=need > 0, workspace=ws)


class FP8GatedLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
        T, x = x.shape[0], x.contiguous()
        qxt = sxt = None
        if ctx.needs_input_grad[1]:
            if T % 128:                                    # whole 128-row tiles of X^T
                padded = x.new_zeros((-(-T // 128) * 128, x.shape[1]))
                padded[:T] = x
                x = padded
            qx, sx, qxt, sxt = quant_act_dual(x, pow2)
            qx = qx[:T]
        else:
            qx, sx = quant_act_1x128(x, pow2)
        qw, sw = quant_weight_128x128(w.contiguous(), pow2)
        h, gu = gemm_blockscaled_gated(qx, sx, qw, sw, with_gu=True)
        ctx.save_for_backward(gu, qxt, sxt, qw, sw)
        ctx.pow2 = pow2
        return h

    @staticmethod
    def backward(ctx, dh: torch.Tensor):
        gu, qxt, sxt, qw, sw = ctx.saved_tensors
        pow2 = ctx.pow2
        T, K = gu.shape[0], qw.shape[1]
        dx = dw = None
        if T == 0:
            return (gu.new_empty((0, K)) if ctx.needs_input_grad[0] else None,
                    gu.new_zeros(qw.shape) if ctx.needs_input_grad[1] else None, None)
        qd, sd, qdt, sdt = gated_backward_quant(dh.to(torch.bfloat16).contiguous(), gu, pow2)
        if ctx.needs_input_grad[0]:
            qwt, swt = transpose_blocks(qw, sw)
            dx = _product(qd, sd, qwt, swt, pow2)
        if ctx.needs_input_grad[1]:
            dw = _product(qdt, sdt, qxt, sxt, pow2, b_rowwise=True)
        return dx, dw, None


def fp8_gated_linear(x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
    """H = silu(X Wg^T) * (X Wu^T) in FP8, W = [Wg; Wu] stacked (see the module docstring).

    x bf16 [T, K], w bf16 [2N, K] -> bf16 [T, N].  Without gradients g and u are not kept.
    """
    for t, name in ((x, "x"), (w, "w")):
        if t.dim() != 2:
            raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    if w.shape[1] != x.shape[1] or w.shape[0] % 256 or x.shape[1] % 128 or not w.numel():
        raise ValueError(f"w must be [2N, K] with N and K multiples of 128 and K the columns of x, got "
                         f"{tuple(w.shape)} for x {tuple(x.shape)}")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return FP8GatedLinearFunction.apply(x, w, pow2)
    qx, sx = quant_act_1x128(x.contiguous(), pow2)
    qw, sw = quant_weight_128x128(w.contiguous(), pow2)
    return gemm_blockscaled_gated(qx, sx, qw, sw)


class FP8GatedLinear(torch.nn.Module):
    """The gate and up projections of a feed-forward block with the activation between them,
    silu(gate(x)) * up(x), whose forward and backward GEMMs run in FP8.  ``weight`` is
    [2 out_features, in_features]: the gate's rows, then the up projection's.  An
    ``FP8Linear(out_features, in_features)`` after it is the block's down projection."""

    def __init__(self, in_features: int, out_features: int, pow2: bool = False,
                 device: Optional[torch.device] = None):
        super().__init__()
        self.pow2 = pow2
        self.weight = torch.nn.Parameter(
            torch.empty((2 * out_features, in_features), dtype=torch.bfloat16, device=device))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fp8_gated_linear(x, self.weight, self.pow2)
