"""GPU tests of the gated layer's paths beside the training step of test_gpu_gated.py."""
import numpy as np
import pytest

import workloads
from tests._helpers import to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_fine_grained_weight_b200 as fq
    fq.lib()
    return fq


def layer_inputs(T, N, K, seed):
    rng = np.random.default_rng(seed)
    x = to_dev_bf16(workloads.normal_bf16(rng, (T, K), 1.0, 0.001))
    return x, to_dev_bf16(workloads.normal_bf16(rng, (2 * N, K), 2 * K ** -0.5))


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,N,K", [(1, 128, 256), (140, 256, 256), (300, 640, 7168), (1025, 384, 1152)])
def test_h_without_gradients_is_h_with_them(fq, T, N, K, pow2):
    """Bit for bit, by the few-row kernel and by the wide ones."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    x, w = layer_inputs(T, N, K, T + K)
    with torch.no_grad():
        h = fp8_gated_linear(x, w, pow2)
    kept = fp8_gated_linear(x, w.clone().requires_grad_(True), pow2)
    assert kept.requires_grad and torch.equal(h, kept)
    assert fq.device_error() == 0


@pytest.mark.parametrize("pow2", [False, True])
def test_one_token_of_any_row_stride(fq, pow2):
    """A token as a transposed column and as a row of an oddly pitched buffer, with and without
    gradients, and the quantizers on the same rows."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    x, w = layer_inputs(1, 128, 256, 5)
    odd = torch.zeros((3, 263), dtype=torch.bfloat16, device="cuda")
    odd[1:2, 7:] = x
    with torch.no_grad():
        h = fp8_gated_linear(x, w, pow2)
    q, s = fq.quant_act_1x128(x, pow2)
    qr, sr = fq.quant_rowwise(x, pow2)
    column = x.reshape(-1, 1).clone().t()
    aligned = torch.zeros((3, 261), dtype=torch.bfloat16, device="cuda")     # its first row, 16 bytes aligned
    aligned[:1, :256] = x
    for v in (column, odd[1:2, 7:], aligned[:1, :256]):
        assert v.shape == (1, 256) and v.stride(0) % 8 != 0 or v.stride(0) < 256
        with torch.no_grad():
            assert torch.equal(fp8_gated_linear(v, w, pow2), h)
        v1 = v.detach().requires_grad_(True)
        assert torch.equal(fp8_gated_linear(v1, w, pow2), h)
        if v.data_ptr() % 16 == 0:
            for got, want in zip((*fq.quant_act_1x128(v, pow2), *fq.quant_rowwise(v, pow2)), (q, s, qr, sr)):
                assert torch.equal(got, want)
    assert fq.device_error() == 0
