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
of 128.  A step of a small layer is bound by the host, so the gated layer's function makes
the library's calls itself on buffers carved from one allocation per direction (half the
host time of going through the binding's functions).
"""
from typing import Optional

import torch

from torch.autograd.function import once_differentiable

from . import (BSCALE_BLOCK, BSCALE_ROW, OUT_BF16, _call, _on, _require_cuda, _same_device, _stream,
               gemm_blockscaled, gemm_blockscaled_gated, gemm_blockscaled_ue8m0, quant_act_1x128,
               quant_act_dual, quant_weight_128x128, transpose_blocks, workspace_bytes)


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


def _carve(device, sizes):
    """One allocation for buffers of the given bytes: (the tensor that owns it, their offsets)."""
    offsets, end = [], 0
    for n in sizes:
        offsets.append(end)
        end += -(-n // 256) * 256
    return torch.empty_strided((end,), (1,), dtype=torch.uint8, device=device), offsets


def _packed(t: torch.Tensor) -> torch.Tensor:
    """`t` contiguous and starting on 16 bytes (a view may do neither)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _pad128(n: int) -> int:
    return -(-n // 128) * 128


def _product(a, sa, ld_sa, b, sb, ld_sb, rowwise, out, M, N, K, pow2, ws, ws_len, stream):
    """out [M, N] = A B^T in bf16 from raw pointers, both operands with K contiguous."""
    mode = BSCALE_ROW if rowwise else BSCALE_BLOCK
    if pow2:
        _call("fp8_gemm_blockscaled_ue8m0", a, sa, ld_sa, b, sb, ld_sb, mode, out.data_ptr(), OUT_BF16,
              M, N, K, K, K, N, stream)
    else:
        _call("fp8_gemm_blockscaled_ws", a, sa, ld_sa, b, sb, ld_sb, mode, out.data_ptr(), OUT_BF16,
              M, N, K, K, K, N, ws, ws_len, stream)


class FP8GatedLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
        x, w = _packed(x), _packed(w)
        (T, K), R = x.shape, w.shape[0]                    # R = 2N
        N, Tp, pow2 = R // 2, _pad128(T), int(bool(pow2))
        for_dw = ctx.needs_input_grad[1]
        # kept for the backward pass: g and u, the codes and scales of W, those of X^T
        kept, (gu, qw, sw, qxt, sxt) = _carve(x.device, (2 * T * R, R * K, R * K // 4096,
                                                         K * Tp * for_dw, K * Tp // 32 * for_dw))
        base = kept.data_ptr()
        own, (qx, sx) = _carve(x.device, (T * K, T * K // 32))
        q, s = own.data_ptr() + qx, own.data_ptr() + sx
        h = torch.empty_strided((T, N), (N, 1), dtype=torch.bfloat16, device=x.device)
        with _on(x):
            stream = _stream(x)
            if for_dw:
                _call("fp8q_quant_act_dual" if T == Tp else "fp8q_quant_act_dual_padded", x.data_ptr(), T, K, K, q, K, s, T, base + qxt, Tp,
                      base + sxt, K, pow2, stream)
            else:
                _call("fp8q_quant_act_1x128", x.data_ptr(), T, K, K, q, K, s, T, pow2, stream)
            _call("fp8q_quant_weight_128x128", w.data_ptr(), R, K, K, base + qw, K, base + sw, pow2, stream)
            _call("fp8_gemm_blockscaled_gated", q, s, T, base + qw, base + sw, h.data_ptr(), N,
                  base + gu, R, T, N, K, K, K, stream)
        ctx.save_for_backward(kept)
        ctx.layout = (T, N, K, pow2, gu, qw, sw, qxt, sxt)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh: torch.Tensor):
        kept, = ctx.saved_tensors
        T, N, K, pow2, gu, qw, sw, qxt, sxt = ctx.layout
        for_dx, for_dw, _ = ctx.needs_input_grad
        R, Tp, dev, base = 2 * N, _pad128(T), kept.device, kept.data_ptr()
        dx = torch.empty_strided((T, K), (K, 1), dtype=torch.bfloat16, device=dev) if for_dx else None
        dw = torch.empty_strided((R, K), (K, 1), dtype=torch.bfloat16, device=dev) if for_dw else None
        if T == 0:
            return dx, dw.zero_() if for_dw else None, None
        dh = _packed(dh.to(torch.bfloat16))
        with _on(kept):
            # The promoted GEMM's split-K workspace is this call's own: the buffer cached per stream
            # would be shared by graphs captured on that stream.  Below 2048 a split saves less
            # than its extra launch costs (a group of 128 takes 0.6 us, the launch 2.5 us).
            ws_len = 0 if pow2 else max(workspace_bytes(T, K, R) if for_dx and R >= 2048 else 0,
                                        workspace_bytes(R, K, Tp) if for_dw and Tp >= 2048 else 0)
            own, offsets = _carve(dev, (T * R, T * R // 32, R * Tp, R * Tp // 32, K * R * for_dx,
                                        K * R // 4096 * for_dx, ws_len))
            qd, sd, qdt, sdt, qwt, swt, ws = (own.data_ptr() + o for o in offsets)
            stream = _stream(kept)
            _call("fp8q_gated_backward_quant", dh.data_ptr(), N, base + gu, R, T, N, qd, R, sd, T, qdt, Tp,
                  sdt, R, pow2, stream)
            if for_dx:
                _call("fp8q_transpose_blocks", base + qw, base + sw, R, K, K, qwt, swt, R, stream)
                _product(qd, sd, T, qwt, swt, 0, False, dx, T, K, R, pow2, ws, ws_len * (R >= 2048), stream)
            if for_dw:
                _product(qdt, sdt, R, base + qxt, base + sxt, K, True, dw, R, K, Tp, pow2, ws,
                         ws_len * (Tp >= 2048), stream)
        return dx, dw, None


def fp8_gated_linear(x: torch.Tensor, w: torch.Tensor, pow2: bool = False) -> torch.Tensor:
    """H = silu(X Wg^T) * (X Wu^T) in FP8, W = [Wg; Wu] stacked (see the module docstring).

    x bf16 [T, K], w bf16 [2N, K] -> bf16 [T, N].  Without gradients g and u are not kept.
    Differentiable once.  When a backward pass is captured into a CUDA graph, no other autograd
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
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return FP8GatedLinearFunction.apply(x, w, pow2)
    qx, sx = quant_act_1x128(_packed(x), pow2)
    qw, sw = quant_weight_128x128(_packed(w), pow2)
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
