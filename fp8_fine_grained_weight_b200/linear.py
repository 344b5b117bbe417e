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
of 128.  A step of a small layer is bound by the host, so each direction is one call of the
library.
"""
import ctypes
import functools
from typing import Optional

import torch

from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import (_call, _launch, _require_cuda, _same_device, gemm_blockscaled, gemm_blockscaled_gated,
               gemm_blockscaled_ue8m0, gemm_gated_ue8m0, quant_act_1x128, quant_act_dual,
               quant_weight_128x128, transpose_blocks)


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


def _packed(t: torch.Tensor) -> torch.Tensor:
    """`t` contiguous and starting on 16 bytes (a view may do neither)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _new(device, dtype, *shape) -> torch.Tensor:
    strides = (1,) if len(shape) == 1 else (shape[1], 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


@functools.lru_cache(maxsize=1024)
def _gated_bytes(device: int, T: int, N: int, K: int, for_dx: bool, for_dw: bool, pow2: bool):
    """Bytes that the layer keeps, of its forward scratch and of its backward scratch."""
    out = (ctypes.c_size_t * 3)()
    with torch.cuda.device(device):
        _call("fp8q_gated_linear_sizes", T, N, K, for_dx, for_dw, pow2, out)
    return tuple(out)


class FP8GatedLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
        x, w, pow2 = _packed(x), _packed(w), bool(pow2)
        (T, K), N, dev = x.shape, w.shape[0] // 2, x.device
        for_dx, for_dw, _ = ctx.needs_input_grad
        kept_bytes, scratch_bytes, ctx.scratch = _gated_bytes(dev.index, T, N, K, for_dx, for_dw, pow2)
        kept = _new(dev, torch.uint8, kept_bytes)          # g and u, the codes of W and of X^T
        scratch = _new(dev, torch.uint8, scratch_bytes)
        h = _new(dev, torch.bfloat16, T, N)
        _launch(x, "fp8q_gated_linear_forward", x.data_ptr(), w.data_ptr(), T, N, K, for_dw, pow2,
                kept.data_ptr(), scratch.data_ptr(), h.data_ptr())
        ctx.save_for_backward(kept)
        ctx.sizes = (T, N, K, for_dw, pow2)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh: torch.Tensor):
        if forward_ad.unpack_dual(dh).tangent is not None:
            raise NotImplementedError("fp8_gated_linear has no forward-mode derivative")
        kept, = ctx.saved_tensors
        T, N, K, kept_for_dw, pow2 = ctx.sizes
        for_dx, for_dw, _ = ctx.needs_input_grad
        dev = kept.device
        dx = _new(dev, torch.bfloat16, T, K) if for_dx else None
        dw = _new(dev, torch.bfloat16, 2 * N, K) if for_dw else None
        if T == 0:
            return dx, dw.zero_() if for_dw else None, None
        dh = _packed(dh.to(torch.bfloat16))
        # one buffer of this call's own, the split-K workspace in it: the one cached per stream would
        # be shared by graphs captured on that stream
        scratch = _new(dev, torch.uint8, ctx.scratch)
        _launch(kept, "fp8q_gated_linear_backward", dh.data_ptr(), kept.data_ptr(), T, N, K, kept_for_dw, pow2,
                scratch.data_ptr(), dx.data_ptr() if for_dx else None, dw.data_ptr() if for_dw else None)
        return dx, dw, None


def fp8_gated_linear(x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
    """H = silu(X Wg^T) * (X Wu^T) in FP8, W = [Wg; Wu] stacked (see the module docstring).

    x bf16 [T, K], w bf16 [2N, K] -> bf16 [T, N].  Without gradients the same product runs and g and u are
    not kept.
    Differentiable once, in reverse mode; a forward-mode tangent is refused.  When a backward pass is captured into a CUDA graph, no other autograd
    graph of the same leaves may be alive: autograd would run its gradient accumulators on the
    stream of that graph, outside the capture (true of every differentiable function).
    """
    for t, name in ((x, "x"), (w, "w")):
        if t.dim() != 2:
            raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    if w.shape[1] != x.shape[1] or w.shape[0] % 256 or x.shape[1] % 128 or not w.numel():
        raise ValueError(f"w must be [2N, K] with N and K multiples of 128 and K the columns of x, got "
                         f"{tuple(w.shape)} for x {tuple(x.shape)}")
    for t, name in ((x, "x"), (w, "w")):
        _require_cuda(t, name)
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    _same_device(w, x.device, "w")
    # (the function also refuses a tangent, which the calls below would drop)
    if (torch.is_grad_enabled() and (x.requires_grad or w.requires_grad)
            or any(forward_ad.unpack_dual(t).tangent is not None for t in (x, w))):
        return FP8GatedLinearFunction.apply(x, w, pow2)
    qx, sx = quant_act_1x128(_packed(x), pow2)
    qw, sw = quant_weight_128x128(_packed(w), pow2)
    return (gemm_gated_ue8m0 if pow2 else gemm_blockscaled_gated)(qx, sx, qw, sw)    # as with gradients


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
