"""GPU tests of the gated FP8 projections, forward and backward, against the oracle and 64-bit
arithmetic.

Forward: g and u are within the GEMM tests' band of the oracle's products, 2e-5 T with
T = sum |a b|; |silu'| <= 1.1, so h is within 2e-5 (1.1 Tg |u| + |silu(g)| Tu) of silu(g) u,
plus the roundings of the epilogue ((8 + 2.7 |g|) 2^-23 relative, counted in the INT8 tests)
and of bf16 (2^-8).

Backward: D = [dg | du] in FP32.  With sg = 1 / (1 + exp(-g)): the exponential is within
2 + 1.173 |g| units of 2^-23, the sum, the quotient (2 units) and each product round, so sg is
within 5 + 1.2 |g| units relative; du adds two products: 6 + 1.2 |g|.  dg = dh u sg t with
t = 1 + g (1 - sg): sg's error moves t by |g| sg (5 + 1.2 |g|) units absolutely and the
subtraction and the FMA round: |g| / 2 + |t| / 2.  Then bf16 (2^-8 of the value), then E4M3
with the tile's scale: half a step, 2^-4 of the value or 2^-10 s among its subnormals.
"""
import numpy as np
import pytest

import oracle
import workloads
from tests._helpers import assert_bytes_equal, assert_gemm_close, host, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_fine_grained_weight_b200 as fq
    fq.lib()
    return fq


def sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def check_h(h, C, T):
    """h (host, float) against the oracle's products C of all 2N rows and their scale T."""
    N = C.shape[1] // 2
    g, u, Tg, Tu = C[:, :N], C[:, N:], T[:, :N], T[:, N:]
    silu = g * sigmoid(g)
    ref = silu * u
    tol = (2e-5 * (1.1 * Tg * np.abs(u) + np.abs(silu) * Tu) * (1 + 2.0 ** -8) + 1e-30
           + (2.0 ** -8 + 2.0 ** -23 * (8 + 2.7 * np.abs(g))) * np.abs(ref) + 1.2e-36 * np.abs(u))
    bad = np.abs(h.astype(np.float64) - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


def operands(M, N, K, pow2, seed):
    rng = np.random.default_rng(seed)
    a = workloads.normal_bf16(rng, (M, K), 1.0, 0.001)
    w = workloads.normal_bf16(rng, (2 * N, K), 2 * K ** -0.5)
    return a, w, oracle.quant_act_1x128(a, pow2), oracle.quant_weight_128x128(w, pow2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (2, 256, 640), (16, 128, 1152), (17, 384, 256), (64, 256, 2048),
                                   (100, 128, 384), (127, 256, 128), (129, 640, 512), (300, 256, 1280),
                                   (513, 128, 384), (1025, 384, 128)])
def test_forward(fq, M, N, K, pow2):
    import torch
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, pow2, M + N + K)
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    args = [to_dev(t) for t in (qa, sa, qw, sw)]
    h, gu = fq.gemm_blockscaled_gated(*args, with_gu=True)
    h2 = fq.gemm_blockscaled_gated(*args)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    check_h(host(h), C, T)
    check_h(host(h2), C, T)
    assert_gemm_close("gu", host(gu), C, T, bf16=True)


def test_forward_of_one_group_and_of_one_token(fq):
    """Scales [1, M] and [G, 1] as a transpose leaves them, with strides that say nothing."""
    import torch
    for M, K in ((70, 128), (1, 384), (1, 128)):
        _, _, (qa, sa), (qw, sw) = operands(M, 128, K, False, M + K)
        C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
        s = to_dev(np.ascontiguousarray(sa.T)).t()
        check_h(host(fq.gemm_blockscaled_gated(to_dev(qa), s, to_dev(qw), to_dev(sw))), C, T)
    assert fq.device_error() == 0


def test_forward_many_tiles(fq):
    """More tiles than SMs and both tile orders, with and without the kept g and u."""
    import torch
    for M, N in ((2500, 1280), (130, 10240)):
        _, _, (qa, sa), (qw, sw) = operands(M, N, 256, False, M)
        C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
        args = [to_dev(t) for t in (qa, sa, qw, sw)]
        h, gu = fq.gemm_blockscaled_gated(*args, with_gu=True)
        check_h(host(h), C, T)
        assert torch.equal(h, fq.gemm_blockscaled_gated(*args))
        assert_gemm_close("gu", host(gu), C, T, bf16=True)
    assert fq.device_error() == 0


@pytest.mark.parametrize("M", [3, 50, 140])
def test_forward_strides_and_guards(fq, M):
    """Padded operands and outputs inside larger buffers, whose other elements stay."""
    import torch
    N, K = 256, 384
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, False, M)
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    A = torch.full((M, K + 32), 0x7F, dtype=torch.uint8, device="cuda")
    A[:, :K] = to_dev(qa)
    W = torch.full((2 * N, K + 16), 0x7F, dtype=torch.uint8, device="cuda")
    W[:, :K] = to_dev(qw)
    S = torch.full((K // 128, M + 7), float("nan"), device="cuda")
    S[:, :M] = to_dev(sa)
    H = torch.full((M + 2, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    GU = torch.full((M + 2, 2 * N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    h, gu = H[1:M + 1, 8:8 + N], GU[1:M + 1, 8:8 + 2 * N]
    fq.gemm_blockscaled_gated(A[:, :K], S, W[:, :K], to_dev(sw), with_gu=True, out=(h, gu))
    check_h(host(h), C, T)
    assert_gemm_close("gu", host(gu.contiguous()), C, T, bf16=True)
    h2 = torch.empty_like(h)
    fq.gemm_blockscaled_gated(A[:, :K], S, W[:, :K], to_dev(sw), out=h2)
    check_h(host(h2), C, T)
    h.fill_(7.0)
    gu.fill_(7.0)
    assert (H == 7).all() and (GU == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (65, 128, 640), (100, 256, 512), (127, 384, 128), (129, 640, 1152),
                                   (300, 256, 1280), (513, 128, 384), (1025, 896, 256), (2500, 1280, 256),
                                   (130, 10240, 128)])
def test_forward_of_powers_of_two(fq, M, N, K):
    """Scales inside the tensor core: part groups of a scale slot, column tiles that end inside a
    tile of 96 and weight blocks that begin inside one, more tiles than SMs, both tile orders."""
    import torch
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, True, M + N + K)
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    args = [to_dev(t) for t in (qa, sa, qw, sw)]
    h, gu = fq.gemm_gated_ue8m0(*args, with_gu=True)
    h2 = fq.gemm_gated_ue8m0(*args)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    check_h(host(h), C, T)
    assert torch.equal(h, h2)
    assert_gemm_close("gu", host(gu), C, T, bf16=True)


@pytest.mark.parametrize("M", [3, 70, 140])
def test_forward_of_powers_of_two_strides_and_guards(fq, M):
    import torch
    N, K = 256, 384
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, True, M)
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    A = torch.full((M, K + 32), 0x7F, dtype=torch.uint8, device="cuda")
    A[:, :K] = to_dev(qa)
    W = torch.full((2 * N, K + 16), 0x7F, dtype=torch.uint8, device="cuda")
    W[:, :K] = to_dev(qw)
    S = torch.full((K // 128, M + 7), float("nan"), device="cuda")
    S[:, :M] = to_dev(sa)
    H = torch.full((M + 2, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    GU = torch.full((M + 2, 2 * N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    h, gu = H[1:M + 1, 8:8 + N], GU[1:M + 1, 8:8 + 2 * N]
    fq.gemm_gated_ue8m0(A[:, :K], S, W[:, :K], to_dev(sw), with_gu=True, out=(h, gu))
    assert fq.device_error() == 0
    check_h(host(h), C, T)
    assert_gemm_close("gu", host(gu.contiguous()), C, T, bf16=True)
    h2 = torch.empty_like(h)
    fq.gemm_gated_ue8m0(A[:, :K], S, W[:, :K], to_dev(sw), out=h2)
    assert torch.equal(h, h2)
    h.fill_(7.0)
    gu.fill_(7.0)
    assert (H == 7).all() and (GU == 7).all()


def test_forward_of_powers_of_two_reports_other_scales(fq):
    """A scale that is no power of two, of a token, of the gate's rows or of the up projection's."""
    import torch
    _, _, (qa, sa), (qw, sw) = operands(200, 128, 256, True, 4)
    for which, at in ((0, (1, 150)), (1, (0, 1)), (1, (1, 0))):
        scales = [sa.copy(), sw.copy()]
        scales[which][at] *= 1.5
        a = [to_dev(t) for t in (qa, scales[0], qw, scales[1])]
        fq.gemm_gated_ue8m0(*a)
        assert fq.device_error() == (8 << 8) | 7
        fq.gemm_gated_ue8m0(*[to_dev(t) for t in (qa, sa, qw, sw)])
        assert fq.device_error() == 0


def test_forward_of_powers_of_two_below_the_smallest_scale(fq):
    """A tile whose scale is a power of two under 2^-127 is reported and counts with 2^-127: g and u
    are off by at most 448 2^-127 sum |w| for it, the other rows' by nothing."""
    import torch
    M, N, K = 300, 256, 512
    _, _, (qa, sa), (qw, sw) = operands(M, N, K, True, 6)
    sa[2, 7], sa[0, 299] = 2.0 ** -130, 2.0 ** -149
    C, T = oracle.gemm_blockscaled_ref(qa, sa, qw, sw)
    h, gu = fq.gemm_gated_ue8m0(*[to_dev(t) for t in (qa, sa, qw, sw)], with_gu=True)
    assert fq.device_error() == (8 << 8) | 7
    wmax = 448 * float(sw.max())
    C = C.astype(np.float64)
    tol = 2e-5 * T * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(C) + 128 * 448 * 2.0 ** -127 * wmax + 1e-30
    assert (np.abs(host(gu).astype(np.float64) - C) <= tol).all()
    check_h(host(h), C, T)


# -------------------------------------------------------------------------------- backward

def grads64(dh, gu):
    N = dh.shape[1]
    g, u = gu[:, :N], gu[:, N:]
    sg = sigmoid(g)
    t = 1 + g * (1 - sg)
    du, dg = dh * g * sg, dh * u * sg * t
    units = 2.0 ** -23
    e_du = units * (6 + 1.2 * np.abs(g)) * np.abs(du)
    e_dg = units * ((8 + 1.2 * np.abs(g)) * np.abs(dg)
                    + np.abs(dh * u * sg) * (np.abs(g) * sg * (5 + 1.2 * np.abs(g)) + np.abs(g) / 2 + np.abs(t)))
    # exp(-g) past 2^126: sg is flushed
    tiny = 1.2e-38 * np.abs(dh) * (1 + np.abs(g)) * (1 + np.abs(u))
    return np.concatenate([dg, du], 1), np.concatenate([e_dg + tiny, e_du + tiny], 1)


def check_codes(D, e, q, s, pow2):
    """q [R, C] and s [C / 128, R] as the 1x128 quantization of a D within e (before the rounding
    to bf16)."""
    vals = oracle.decode_table()[q].astype(np.float64)
    sc = np.repeat(s.T.astype(np.float64), 128, axis=1)
    lo = np.maximum(np.abs(D) - e, 0) * (1 - 2.0 ** -8)
    hi = (np.abs(D) + e) * (1 + 2.0 ** -8)
    R, Cn = D.shape
    amax_lo = lo.reshape(R, Cn // 128, 128).max(2) / 448 * (1 - 2.0 ** -23)
    amax_hi = hi.reshape(R, Cn // 128, 128).max(2) / 448 * (1 + 2.0 ** -23)
    st = s.T
    zero = (amax_hi < 1e-37) | ((amax_lo <= 0) & (st == 1))     # a tile that may be all zeros
    if pow2:
        ok = (st >= amax_lo) & (st < 2 * amax_hi)
        assert (np.frexp(st)[0] == 0.5).all()
    else:
        ok = (st >= amax_lo) & (st <= amax_hi)
    assert (ok | zero).all(), np.argwhere(~(ok | zero))[:4]
    tol = e + (2.0 ** -8 + 2.0 ** -4 * (1 + 2.0 ** -8)) * (np.abs(D) + e) + 2.0 ** -10 * sc + 1e-37
    bad = np.abs(vals * sc - D) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,N", [(1, 128), (5, 256), (127, 128), (128, 384), (130, 256), (300, 128)])
def test_backward_quant(fq, M, N, pow2):
    import torch
    rng = np.random.default_rng(M + N)
    dh = workloads.normal_bf16(rng, (M, N), 1e-3)
    gu = workloads.normal_bf16(rng, (M, 2 * N), 3.0, 0.01)
    q, s, qt, st = fq.gated_backward_quant(to_dev_bf16(dh), to_dev_bf16(gu), pow2)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    Mp = -(-M // 128) * 128
    assert q.shape == (M, 2 * N) and s.shape == (2 * N // 128, M)
    assert qt.shape == (2 * N, Mp) and st.shape == (Mp // 128, 2 * N)
    f = lambda b: workloads.bf16_bits_to_fp32(b).astype(np.float64)
    D, e = grads64(f(dh), f(gu))
    check_codes(D, e, host(q), host(s), pow2)
    pad = ((0, Mp - M), (0, 0))
    check_codes(np.pad(D, pad).T, np.pad(e, pad).T, host(qt), host(st), pow2)
    assert (host(qt)[:, M:] & 0x7F == 0).all()


@pytest.mark.parametrize("pow2", [False, True])
def test_backward_quant_is_bit_exact_where_the_gradient_is(fq, pow2):
    """g = 0: sg = 1/2 exactly, dg = dh u / 2 rounded once to bf16, du = 0.  Codes and scales of D
    and of its transpose equal the oracle's."""
    rng = np.random.default_rng(8)
    M, N = 256, 256
    dh = workloads.normal_bf16(rng, (M, N), 1e-2)
    gu = workloads.normal_bf16(rng, (M, 2 * N), 2.0, 0.01)
    gu[:, :N] = 0
    f = workloads.bf16_bits_to_fp32
    dg = (f(dh) * f(gu[:, N:]) * np.float32(0.5)).astype(np.float32)      # exact in FP32
    D = np.concatenate([workloads.fp32_to_bf16_bits(dg), np.zeros((M, N), np.uint16)], 1)
    # du = dh 0 keeps the sign of dh
    D[:, N:] = dh & 0x8000
    got = [host(t) for t in fq.gated_backward_quant(to_dev_bf16(dh), to_dev_bf16(gu), pow2)]
    qr, sr = oracle.quant_act_1x128(D, pow2)
    qtr, str_ = oracle.quant_act_1x128(np.ascontiguousarray(D.T), pow2)
    for name, a, b in zip(("q", "s", "qt", "st"), got, (qr, sr, qtr, str_)):
        assert_bytes_equal(name, a, b)


def test_backward_formula_against_differences():
    """The gradient that the tests above hold the kernel to, against central differences."""
    rng = np.random.default_rng(4)
    g, u, dh = (rng.normal(0, 3, (1, 128)) for _ in range(3))
    D, _ = grads64(dh, np.concatenate([g, u], 1))
    f = lambda g, u: g * sigmoid(g) * u
    d = 1e-5
    dg = dh * (f(g + d, u) - f(g - d, u)) / (2 * d)
    du = dh * (f(g, u + d) - f(g, u - d)) / (2 * d)
    # truncation d^2 / 6 |f'''| < 1e-9 and cancellation 2^-52 |f| / d < 1e-9
    assert np.abs(D - np.concatenate([dg, du], 1)).max() < 1e-8


def test_backward_quant_guards(fq):
    """Outputs inside larger buffers; nothing outside them is written, and no row past M."""
    import torch
    M, N = 70, 256
    rng = np.random.default_rng(5)
    dh = to_dev_bf16(workloads.normal_bf16(rng, (M, N), 1e-3))
    gu = to_dev_bf16(workloads.normal_bf16(rng, (M, 2 * N), 2.0))
    want = fq.gated_backward_quant(dh, gu)
    DH = torch.full((M + 1, N + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    GU = torch.full((M + 1, 2 * N + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    DH[:M, :N], GU[:M, :2 * N] = dh, gu
    bufs = [torch.full((M + 60, 2 * N + 8), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((2 * N // 128 + 1, M + 9), 7.0, device="cuda"),
            torch.full((2 * N + 1, 128 + 16), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((2, 2 * N + 3), 7.0, device="cuda")]
    shapes = [(M, 2 * N), (2 * N // 128, M), (2 * N, 128), (1, 2 * N)]
    views = [b[:r, :c] for b, (r, c) in zip(bufs, shapes)]
    fq.gated_backward_quant(DH[:M, :N], GU[:M, :2 * N], out=tuple(views))
    for v, w in zip(views, want):
        assert torch.equal(v, w)
        v.fill_(7.0 if v.dtype == torch.float32 else 0x5A)
    for b in bufs:
        assert (b == (7.0 if b.dtype == torch.float32 else 0x5A)).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (100, 256), (128, 256), (129, 384), (300, 128)])
def test_dual_quantizer_for_any_rows(fq, M, K, pow2):
    """Codes and scales of X and of X^T padded with zeros, bit for bit; nothing beside them."""
    import torch
    xb = workloads.normal_bf16(np.random.default_rng(M), (M, K), 1.0, 0.001)
    Mp = -(-M // 128) * 128
    x = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, :K] = to_dev_bf16(xb)
    q = torch.full((M + 30, K + 8), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((K // 128, M + 5), 7.0, device="cuda")
    qt = torch.full((K + 1, Mp + 16), 0x5A, dtype=torch.uint8, device="cuda")
    st = torch.full((Mp // 128 + 1, K + 3), 7.0, device="cuda")
    assert fq.lib().fp8q_quant_act_dual_padded(
        x.data_ptr(), M, K, x.stride(0), q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0), qt.data_ptr(),
        qt.stride(0), st.data_ptr(), st.stride(0), int(pow2), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    padded = np.zeros((Mp, K), xb.dtype)
    padded[:M] = xb
    qr, sr = oracle.quant_act_1x128(xb, pow2)
    qtr, str_ = oracle.quant_act_1x128(np.ascontiguousarray(padded.T), pow2)
    for name, got, want in (("q", q[:M, :K], qr), ("s", s[:, :M], sr), ("qt", qt[:K, :Mp], qtr),
                            ("st", st[:Mp // 128, :K], str_)):
        assert_bytes_equal(name, host(got.contiguous()), want)
        got.fill_(0x5A if got.dtype == torch.uint8 else 7.0)
    assert all((t == (0x5A if t.dtype == torch.uint8 else 7.0)).all() for t in (q, s, qt, st))


# --------------------------------------------------------------------------- the whole layer

def layer_check(fq, T, N, K, pow2, seed):
    """One forward and backward, each product against the oracle's product of the codes it
    read (the gradient's codes from gated_backward_quant on the same g and u, which is
    tested above)."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    xb, wb, (qx, sx), (qw, sw) = operands(T, N, K, pow2, seed)
    dhb = workloads.normal_bf16(np.random.default_rng(seed + 1), (T, N), 1e-3)
    x, w, dh = to_dev_bf16(xb).requires_grad_(True), to_dev_bf16(wb).requires_grad_(True), to_dev_bf16(dhb)
    h = fp8_gated_linear(x, w, pow2)
    dx, dw = torch.autograd.grad(h, (x, w), dh)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    assert h.dtype == dx.dtype == dw.dtype == torch.bfloat16 and dx.shape == x.shape and dw.shape == w.shape
    C, Tm = oracle.gemm_blockscaled_ref(qx, sx, qw, sw)
    check_h(host(h), C, Tm)
    gated = fq.gemm_gated_ue8m0 if pow2 else fq.gemm_blockscaled_gated          # as the layer
    _, gu = gated(*[to_dev(t) for t in (qx, sx, qw, sw)], with_gu=True)
    q, s, qt, st = (host(t) for t in fq.gated_backward_quant(dh, gu, pow2))
    qwt, swt = oracle.quant_weight_128x128(np.ascontiguousarray(wb.T), pow2)
    C, Tm = oracle.gemm_blockscaled_ref(q, s, qwt, swt)
    assert_gemm_close("dx", host(dx), C, Tm, bf16=True)
    Tp = -(-T // 128) * 128
    xt = np.zeros((K, Tp), xb.dtype)
    xt[:, :T] = xb.T
    qxt, sxt = oracle.quant_act_1x128(xt, pow2)
    C, Tm = oracle.gemm_blockscaled_ref(qt, st, qxt, sxt, b_rowwise=True)
    assert_gemm_close("dw", host(dw), C, Tm, bf16=True)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (200, 256, 384), (256, 384, 256), (513, 128, 640)])
def test_layer(fq, T, N, K, pow2):
    layer_check(fq, T, N, K, pow2, T + N + K)


def test_layer_needs_only_what_is_asked(fq):
    """Gradients of x alone and of w alone are those of both; without gradients the same h."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    xb, wb, _, _ = operands(140, 256, 256, False, 3)
    x, w = to_dev_bf16(xb), to_dev_bf16(wb)
    dh = to_dev_bf16(workloads.normal_bf16(np.random.default_rng(9), (140, 256), 1e-3))
    x1, w1 = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    h = fp8_gated_linear(x1, w1)
    dx, dw = torch.autograd.grad(h, (x1, w1), dh)
    hx = fp8_gated_linear(x1, w)
    assert torch.equal(torch.autograd.grad(hx, x1, dh)[0], dx) and torch.equal(hx, h)
    hw = fp8_gated_linear(x, w1)
    assert torch.equal(torch.autograd.grad(hw, w1, dh)[0], dw) and torch.equal(hw, h)
    with torch.no_grad():
        assert torch.equal(fp8_gated_linear(x1, w1), h)
    assert torch.equal(fp8_gated_linear(x, w), h)
    # an expanded (broadcast) upstream gradient, and the same graph walked twice
    h = fp8_gated_linear(x1, w1)
    a = torch.autograd.grad(h.float().sum(), (x1, w1), retain_graph=True)
    b = torch.autograd.grad(h, (x1, w1), torch.ones_like(h))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_layer_takes_views(fq):
    """Operands and an upstream gradient that are transposed, sliced or off 16 bytes."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    xb, wb, _, _ = operands(70, 128, 256, False, 12)
    x, w = to_dev_bf16(xb), to_dev_bf16(wb)
    dh = to_dev_bf16(workloads.normal_bf16(np.random.default_rng(2), (70, 128), 1e-3))

    def off(t):                                # the same values starting 2 bytes further
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    want = None
    for f in (lambda t: t.clone(), lambda t: t.t().contiguous().t(), off):
        x1, w1 = f(x).requires_grad_(True), f(w).requires_grad_(True)
        h = fp8_gated_linear(x1, w1)
        got = (h.detach(), *torch.autograd.grad(h, (x1, w1), f(dh)))
        with torch.no_grad():
            assert torch.equal(fp8_gated_linear(x1, w1), got[0])
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(RuntimeError):          # no second derivative
        h = fp8_gated_linear(x1, w1)
        g = torch.autograd.grad(h, x1, dh.clone().requires_grad_(True), create_graph=True)[0]
        torch.autograd.grad(g.float().sum(), x1)


def test_empty_batch(fq):
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.ones((256, 128), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    h = fp8_gated_linear(x, w)
    dx, dw = torch.autograd.grad(h, (x, w), torch.empty_like(h))
    assert h.shape == (0, 128) and dx.shape == (0, 128) and (dw == 0).all()


@pytest.mark.parametrize("pow2", [False, True])
def test_feed_forward_block(fq, pow2):
    """The gated layer and a down projection together: outputs and gradients of the block follow
    the FP32 block on the same weights.  E4M3 rounds by at most 2^-4 (its error on average is
    2^-4 / sqrt(3) per operand = 3.6%, two operands per product, four products deep:
    3.6% sqrt(8) = 10%)."""
    import torch
    from fp8_fine_grained_weight_b200.linear import FP8GatedLinear, FP8Linear
    torch.manual_seed(1)
    up, down = FP8GatedLinear(512, 384, pow2, device="cuda"), FP8Linear(384, 512, pow2, device="cuda")
    x = torch.randn(256, 512, device="cuda").to(torch.bfloat16).requires_grad_(True)
    y = down(up(x))
    dy = torch.randn_like(y)
    y.backward(dy)
    xf, wu, wd = (t.detach().float().requires_grad_(True) for t in (x, up.weight, down.weight))
    gu = xf @ wu.t()
    yf = (torch.nn.functional.silu(gu[:, :384]) * gu[:, 384:]) @ wd.t()
    yf.backward(dy.float())
    for got, want in ((y, yf), (x.grad, xf.grad), (up.weight.grad, wu.grad), (down.weight.grad, wd.grad)):
        d = (got.detach().float() - want.detach()).norm() / want.detach().norm()
        assert float(d) < 0.10
    assert fq.device_error() == 0


def test_layer_in_graphs_and_on_a_stream(fq):
    """Forward and backward captured twice and replayed at the same time; and on a side stream."""
    import torch
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    sets = []
    for seed in (1, 2):
        xb, wb, _, _ = operands(200, 256, 384, False, seed)
        dh = workloads.normal_bf16(np.random.default_rng(seed), (200, 256), 1e-3)
        sets.append((to_dev_bf16(xb).requires_grad_(True), to_dev_bf16(wb).requires_grad_(True), to_dev_bf16(dh)))

    def step(x, w, dh):
        h = fp8_gated_linear(x, w)
        return (h.detach(), *torch.autograd.grad(h, (x, w), dh))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [step(*s) for s in sets]
    side.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(step(*s), w))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    other = torch.cuda.Stream()
    for _ in range(10):
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert fq.device_error() == 0
