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
