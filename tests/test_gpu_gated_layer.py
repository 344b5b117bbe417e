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


def test_promoted_step_that_splits_its_products(fq):
    """Two and more thousand tokens with FP32 scales: both gradient products split their last wave along K
    into the layer's own scratch.  Each product against the oracle's of the codes it read."""
    from tests.test_gpu_gated import layer_check
    T, N, K = 2200, 1024, 256
    assert fq.workspace_bytes(T, K, 2 * N) > 0 and fq.workspace_bytes(2 * N, K, 2304) > 0
    layer_check(fq, T, N, K, False, 17)


def test_host_threads(fq):
    """Four host threads at once, each on its own stream: INT8 blocks and training steps of its own
    inputs give the bits they give alone."""
    import threading
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear

    def once(x, w, dh, pow2):
        x1, w1 = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
        h = fp8_gated_linear(x1, w1, pow2)
        grads = torch.autograd.grad(h, (x1, w1), dh)
        with torch.no_grad():
            h0 = fp8_gated_linear(x, w, pow2)
            q, s = fq.quant_int8_rowwise(x)
            h8 = fq.gemm_int8_gated(q, s, *fq.quant_int8_rowwise(w))
            y = fq.gemm_int8(q, s, *fq.quant_int8_rowwise(w), out_dtype=torch.float32)
        return [h.detach(), *grads, h0, h8, y]

    jobs = []
    for i, (T, N, K) in enumerate(((1, 128, 256), (140, 256, 384), (700, 384, 512), (2200, 1024, 256))):
        x, w = layer_inputs(T, N, K, i)
        jobs.append((x, w, to_dev_bf16(workloads.normal_bf16(np.random.default_rng(i), (T, N), 1e-3)), i % 2 == 1))
    want = [once(*job) for job in jobs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(jobs))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(30)
                for _ in range(20):
                    got = once(*jobs[i])
                    torch.cuda.current_stream().synchronize()
                    wrong.extend((i, k) for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except Exception as e:                                   # reported by the test's thread
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not wrong and not any(t.is_alive() for t in threads), wrong[:4]
    torch.cuda.synchronize()
    assert fq.device_error() == 0


def test_one_column_operands_of_the_other_entry_points(fq):
    """Scales of one token, [G, 1], with a column stride that is not 1: the block-scaled and the grouped
    products read the same scales as from a contiguous copy."""
    import torch
    x, w = layer_inputs(1, 128, 384, 9)
    qa, sa = fq.quant_act_1x128(x, True)
    qw, sw = fq.quant_weight_128x128(w, True)
    wide = torch.full((3, 4), float("nan"), device="cuda")
    wide[:, 1:2] = sa
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for scales in (sa.reshape(1, 3).t(), wide[:, 1:2], wide[:, 1::3][:, :1]):
        assert torch.equal(scales, sa)
        for f in (fq.gemm_blockscaled, fq.gemm_blockscaled_ue8m0):
            assert torch.equal(f(qa, scales, qw, sw), f(qa, sa, qw, sw))
        for f in (fq.gemm_grouped, fq.gemm_grouped_ue8m0):
            assert torch.equal(f(qa, scales, qw[None], sw[None], offsets), f(qa, sa, qw[None], sw[None], offsets))
        c, q, s = fq.gemm_blockscaled_quant(qa, scales, qw, sw)
        assert all(torch.equal(a, b) for a, b in zip((c, q, s), fq.gemm_blockscaled_quant(qa, sa, qw, sw)))
    out = torch.empty((3, 4), device="cuda")[:, ::3][:, :1]
    q, s = fq.quant_act_1x128(x, True, out=(torch.empty_like(qa), out))
    assert s is out and torch.equal(s, sa) and torch.equal(q, qa)
    assert fq.device_error() == 0
