"""Every element of every output of the 8-bit feed-forward operators is written and is a number:
outputs filled with NaN before the call, compared with the 64-bit references of test_gpu_int8.py and
test_gpu_gated.py in the form in which a NaN fails.  The tolerances are derived there."""
import numpy as np
import pytest

import oracle
import workloads
from tests._helpers import assert_gemm_close, assert_within, host, to_dev, to_dev_bf16
from tests.test_gpu_gated import grads64, operands, sigmoid
from tests.test_gpu_int8 import acc_ref, bf16_normal, codes, gated_ref, quant_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_fine_grained_weight_b200 as fq
    fq.lib()
    return fq


def nan(*shape, dtype):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def unset(*shape, dtype):
    """Codes that read as NaN (E4M3) or, for INT8, as -1."""
    import torch
    return torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda").view(dtype)


# One tile of 16, 32, 64 and 128 rows of the few-row kernel, K of one group and split over a cluster; the wide
# kernel on single CTAs and on pairs; rows of C on 16 bytes and not, part tiles both ways.
SHAPES = [(1, 128, 512), (5, 33, 40), (20, 136, 1000), (50, 64, 130), (100, 512, 2048), (150, 2049, 129),
          (300, 513, 640), (1000, 2048, 256), (2000, 1100, 384)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fp32", [False, True])
def test_gemm_int8(fq, M, N, K, fp32):
    import torch
    dtype = torch.float32 if fp32 else torch.bfloat16
    (qa, sa), (qb, sb) = codes(M, K, M + K), codes(N, K, N + 2 * K)
    C = fq.gemm_int8(qa, sa, qb, sb, out=nan(M, N, dtype=dtype))
    assert fq.device_error() == 0
    ref = host(acc_ref(qa, qb) * sa.double()[:, None] * sb.double())
    assert_within("C", host(C), ref, (3.01 * 2.0 ** -24 + (0 if fp32 else 2.0 ** -8)) * np.abs(ref))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_int8_gated(fq, M, N, K):
    import torch
    (qa, sa), (qw, sw) = codes(M, K, M + K), codes(2 * N, K, N + 2 * K)
    h = fq.gemm_int8_gated(qa, sa, qw, sw, out=nan(M, N, dtype=torch.bfloat16))
    assert fq.device_error() == 0
    ref, tol = gated_ref(qa, sa, qw, sw)
    assert_within("h", host(h), host(ref), host(tol))


@pytest.mark.parametrize("M,K", [(1, 8), (3, 7), (9, 1000), (2, 4096), (2, 8200), (2, 16391)])
def test_quant_int8(fq, M, K):
    import torch
    x = bf16_normal((M, K), K)
    for code in (-1, 77):                      # a code left alone cannot agree with both
        q, s = torch.full((M, K), code, dtype=torch.int8, device="cuda"), nan(M, dtype=torch.float32)
        fq.quant_int8_rowwise(x, out=(q, s))
        qr, sr = quant_ref(x)
        assert torch.equal(q, qr) and torch.equal(s, sr)


@pytest.mark.parametrize("entry", ["gemm_blockscaled_gated", "gemm_gated_ue8m0"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (16, 256, 1152), (30, 128, 640), (64, 384, 256), (127, 128, 384),
                                   (300, 1280, 640), (600, 2560, 128), (1025, 384, 512), (2500, 1280, 256)])
def test_fp8_gated(fq, entry, M, N, K):
    import torch
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, entry == "gemm_gated_ue8m0", M + N + K)
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    args = [to_dev(t) for t in (qa, sa, qw, sw)]
    product = getattr(fq, entry)
    h, gu = product(*args, with_gu=True, out=(nan(M, N, dtype=torch.bfloat16), nan(M, 2 * N, dtype=torch.bfloat16)))
    h2 = product(*args, out=nan(M, N, dtype=torch.bfloat16))
    assert fq.device_error() == 0
    assert_gemm_close("gu", host(gu), C, T, bf16=True)
    g, u, Tg, Tu = C[:, :N], C[:, N:], T[:, :N], T[:, N:]
    silu = g * sigmoid(g)
    tol = (2e-5 * (1.1 * Tg * np.abs(u) + np.abs(silu) * Tu) * (1 + 2.0 ** -8) + 1e-30
           + (2.0 ** -8 + 2.0 ** -23 * (8 + 2.7 * np.abs(g))) * np.abs(silu * u) + 1.2e-36 * np.abs(u))
    assert_within("h with g and u", host(h), silu * u, tol)
    assert_within("h", host(h2), silu * u, tol)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,N", [(1, 128), (127, 128), (130, 384), (300, 128)])
def test_gated_backward_quant(fq, M, N, pow2):
    import torch
    rng = np.random.default_rng(M + N)
    dh = workloads.normal_bf16(rng, (M, N), 1e-3)
    gu = workloads.normal_bf16(rng, (M, 2 * N), 3.0, 0.01)
    Mp = -(-M // 128) * 128
    out = (unset(M, 2 * N, dtype=torch.uint8), nan(2 * N // 128, M, dtype=torch.float32),
           unset(2 * N, Mp, dtype=torch.uint8), nan(Mp // 128, 2 * N, dtype=torch.float32))
    fq.gated_backward_quant(to_dev_bf16(dh), to_dev_bf16(gu), pow2, out=out)
    assert fq.device_error() == 0
    f = lambda b: workloads.bf16_bits_to_fp32(b).astype(np.float64)
    D, e = grads64(f(dh), f(gu))
    pad = ((0, Mp - M), (0, 0))
    for name, D, e, q, s in (("rows", D, e, *out[:2]), ("columns", np.pad(D, pad).T, np.pad(e, pad).T, *out[2:])):
        sc = np.repeat(host(s).T.astype(np.float64), 128, axis=1)
        values = oracle.decode_table()[host(q)].astype(np.float64) * sc
        tol = e + (2.0 ** -8 + 2.0 ** -4 * (1 + 2.0 ** -8)) * (np.abs(D) + e) + 2.0 ** -10 * sc + 1e-37
        assert_within(name, values, D, tol)


# ------------------------------------------------------------------------ what the layer allocates

def fill_free_memory(byte):
    """The allocator's free blocks, small and large, hold `byte` afterwards: the blocks go from large to
    small, so that each size takes what the last one left beside tensors that live."""
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [1 << 26] * 4 + [1 << 23] * 8 + [1 << 21] * 32 + [1 << 19] * 128 + [1 << k for k in range(18, 8, -1)]
    held = [torch.full((n,), byte, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(1 if n >> 19 else 32)]
    del held
    for n in (1 << 10, 1 << 18, 1 << 22, 1 << 25):
        assert (torch.empty(n, dtype=torch.uint8, device="cuda").cpu() == byte).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (200, 256, 384), (513, 128, 640), (2200, 1024, 256)])
def test_layer_does_not_read_what_its_memory_held(fq, T, N, K, pow2):
    """Results on memory full of NaN (0xFF bytes in every type) are those on zeroed memory: the buffers
    kept, the scratch with its split-K workspace, and the outputs."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    xb, wb, _, _ = operands(T, N, K, pow2, T + K)
    x, w = to_dev_bf16(xb).requires_grad_(True), to_dev_bf16(wb).requires_grad_(True)
    dh = to_dev_bf16(workloads.normal_bf16(np.random.default_rng(T), (T, N), 1e-3))
    results = []
    for byte in (0, 0xFF):
        fill_free_memory(byte)
        h = fp8_gated_linear(x, w, pow2)
        got = [h.detach(), *torch.autograd.grad(h, (x, w), dh)]
        with torch.no_grad():
            got.append(fp8_gated_linear(x, w, pow2))
        assert all(torch.isfinite(t).all() for t in got)
        results.append([t.cpu() for t in got])
        del h, got
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert fq.device_error() == 0
