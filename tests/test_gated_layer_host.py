"""The gated layer's paths on the CPU: which library calls each makes and with which arguments (the
calls recorded instead of made)."""
import pytest
import torch

import fp8_fine_grained_weight_b200 as fq
import fp8_fine_grained_weight_b200.linear as linear
from fp8_fine_grained_weight_b200.linear import fp8_gated_linear

bf16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    log = []
    for module in (fq, linear):
        monkeypatch.setattr(module, "_require_cuda", lambda t, name: None)
        monkeypatch.setattr(module, "_call", lambda name, *args: log.append((name, args)))
    monkeypatch.setattr(fq, "_stream", lambda t: 0)
    monkeypatch.setattr(linear, "_gated_bytes", lambda *a: (256, 256, 256))
    return log


def names(calls):
    return [name for name, _ in calls]


@pytest.mark.parametrize("pow2,product", [(False, "fp8_gemm_blockscaled_gated"), (True, "fp8_gemm_gated_ue8m0")])
def test_without_gradients_the_scales_choose_the_product(calls, pow2, product):
    """The product that the layer runs with gradients: FP32 scales promoted, powers of two applied by the
    tensor core."""
    x, w = torch.empty(4, 128, dtype=bf16), torch.empty(256, 128, dtype=bf16)
    assert fp8_gated_linear(x, w, pow2).shape == (4, 128)
    assert names(calls) == ["fp8q_quant_act_1x128", "fp8q_quant_weight_128x128", product]
    assert all(args[-2] == int(pow2) for _, args in calls[:2])
    calls.clear()
    w.requires_grad_(True)
    with torch.no_grad():
        fp8_gated_linear(x, w, pow2)
    assert names(calls)[-1] == product


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dual", ["x", "w"])
@pytest.mark.parametrize("grad_mode", [True, False])
def test_forward_mode_derivatives_are_refused(calls, pow2, dual, grad_mode):
    """An operand with a tangent does not require a gradient; its derivative must not come out as zero."""
    from torch.autograd import forward_ad
    ops = {"x": torch.zeros(4, 128, dtype=bf16), "w": torch.zeros(256, 128, dtype=bf16)}
    with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        fp8_gated_linear(**ops, pow2=pow2)                       # no tangent: taken
        ops[dual] = forward_ad.make_dual(ops[dual], torch.ones_like(ops[dual]))
        with pytest.raises(NotImplementedError, match="jvp"):
            fp8_gated_linear(**ops, pow2=pow2)
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda x: fp8_gated_linear(x, ops["w"], pow2), (torch.zeros(4, 128, dtype=bf16),),
                       (torch.ones(4, 128, dtype=bf16),))


def test_a_tangent_of_the_upstream_gradient_is_refused(calls):
    from torch.autograd import forward_ad
    x = torch.zeros(4, 128, dtype=bf16, requires_grad=True)
    h = fp8_gated_linear(x, torch.zeros(256, 128, dtype=bf16))
    dh = torch.zeros(4, 128, dtype=bf16)
    with forward_ad.dual_level():
        torch.autograd.grad(h, x, dh, retain_graph=True)         # no tangent: taken
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.autograd.grad(h, x, forward_ad.make_dual(dh, torch.ones_like(dh)))


def test_a_single_token_of_any_row_stride(calls):
    """A row taken out of a transposed or oddly pitched buffer stays contiguous to torch whatever its row
    stride says; the quantizers that the layer runs get a stride that the library takes."""
    w = torch.zeros(256, 128, dtype=bf16)
    for x in (torch.zeros(128, 1, dtype=bf16).t(), torch.zeros(3, 131, dtype=bf16)[1:2, 3:]):
        assert x.shape == (1, 128) and x.is_contiguous() and x.stride(0) != 128
        fp8_gated_linear(x, w)
        args = dict(calls)["fp8q_quant_act_1x128"]
        assert args[1:4] == (1, 128, 128) and args[5] == 128
        fq.quant_rowwise(x)
        assert calls[-1][1][1:4] == (1, 128, 128)
        calls.clear()


def test_quantizers_take_single_rows_of_outputs(calls):
    """Outputs with one row, or scales of one group, whose row stride is not the pitch."""
    u8, f32 = torch.uint8, torch.float32
    q, s = torch.zeros(256, 1, dtype=u8).t(), torch.zeros(2, 9, dtype=f32)
    fq.quant_act_1x128(torch.zeros(1, 256, dtype=bf16), out=(q, s))
    assert calls[-1][1][5] == 256 and calls[-1][1][7] == 9
    one_group = torch.zeros(5, 1, dtype=f32).t()                 # [1, 5], row stride 1
    fq.quant_act_1x128(torch.zeros(5, 128, dtype=bf16), out=(torch.zeros(5, 128, dtype=u8), one_group))
    assert calls[-1][1][7] >= 5
    padded = torch.zeros(1, 16, dtype=f32)                       # what ran before: its stride is the pitch
    fq.quant_act_1x128(torch.zeros(5, 128, dtype=bf16), out=(torch.zeros(5, 128, dtype=u8), padded), ld_scale=16)
    assert calls[-1][1][7] == 16
    with pytest.raises(ValueError, match="ld_scale"):
        fq.quant_act_1x128(torch.zeros(5, 128, dtype=bf16), out=(torch.zeros(5, 128, dtype=u8), padded), ld_scale=8)
