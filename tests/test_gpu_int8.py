"""GPU tests of the per-row INT8 quantizer and the INT8 products, against 64-bit arithmetic.

The quantizer is bit-exact with its definition.  The products' sums are exact, so every
tolerance counts roundings only (each at most half a step: 2^-24 relative in FP32, 2^-8 in
bf16):

  product   acc -> FP32, times sa, times sb: 3 roundings; bf16 output one more.
  gated     g and u carry 3 FP32 roundings each.  silu(g) = g / (1 + exp(-g)): a relative
            error d of g moves it by |1 + g (1 - sg)| d <= (1 + |g|) d; the exponential is
            within 2 + 1.173 |g| units of 2^-23 (as CUDA's __expf) and enters 1 + e with weight
            e / (1 + e) <= 1; the sum rounds once, the quotient is within 2 units, the product
            with u rounds once.  In units of 2^-23: 1.5 (1 + |g|) + 2 + 1.173 |g| + 0.5 + 2 +
            0.5 + 1.5 <= 8 + 2.7 |g|.  Below g = -87.3 the quotient may be flushed: 1.2e-36 |u|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_fine_grained_weight_b200 as fq
    fq.lib()
    return fq


def quant_ref(x):
    """Definition of the quantizer in 64 bits (scale and reciprocal are FP32 by definition)."""
    import torch
    x = x.double()
    a = x.abs().amax(dim=1)
    finite = torch.isfinite(x).all(dim=1)
    zero = a < 2.0 ** -100
    a1 = torch.where(finite & ~zero, a, torch.ones_like(a))
    s = torch.where(zero, torch.ones_like(a), (a1 / 127.0).float().double())
    s = torch.where(finite, s, torch.full_like(s, float("nan")))
    r = (127.0 / a1).float().double()
    q = torch.round(torch.where(torch.isfinite(x), x, torch.zeros_like(x)) * r[:, None])
    q = torch.where((finite & ~zero)[:, None], q, torch.zeros_like(q))
    return q.to(torch.int8), s.float()


def bf16_normal(shape, seed, std=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def codes(rows, K, seed, pitch=None):
    """int8 codes over the whole range, -128 among them, rows `pitch` bytes apart."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pitch = -(-K // 16) * 16 if pitch is None else pitch
    q = torch.randint(-128, 128, (rows, pitch), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand((rows,), generator=g, device="cuda") * 0.01 + 0.001
    return q[:, :K], s


# ------------------------------------------------------------------------------- quantizer

@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (1, 8), (5, 64), (9, 1000), (17, 1024), (2, 1032), (4, 2047),
                                 (3, 7168), (2, 8192), (2, 8200), (1, 16384), (2, 16391), (1, 40001), (300, 129)])
def test_quant_is_bit_exact(fq, M, K):
    import torch
    x = bf16_normal((M, K), M * 1000 + K)
    x[:, 0] *= 50
    q, s = fq.quant_int8_rowwise(x)
    qr, sr = quant_ref(x)
    assert torch.equal(q, qr) and torch.equal(s, sr)
    assert q.stride(0) % 16 == 0


def test_quant_ties_and_extremes(fq):
    """Halves of the largest value (ties up to the rounding of 127 / a), every bf16
    magnitude in one row, rows of zeros, of tiny, huge and non-finite values."""
    import torch
    pats = torch.arange(0x0080, 0x7F80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    rows = torch.zeros((9, pats.numel() + 1), dtype=torch.bfloat16, device="cuda")
    rows[0, :-1] = pats
    rows[1, :-1] = -pats
    k = torch.arange(254, device="cuda", dtype=torch.float32)
    rows[2, :254] = (k / 2 - 63).to(torch.bfloat16)
    rows[2, 300] = 127.0
    rows[4, 5] = 2.0 ** -101
    rows[5, 6] = -(2.0 ** -100)
    rows[6, 7] = float("inf")
    rows[7, 8] = float("nan")
    rows[8, 9], rows[8, 10] = float("-inf"), 3.0
    for x in (rows, rows[:, 1:], rows[:, :-2]):
        q, s = fq.quant_int8_rowwise(x)
        qr, sr = quant_ref(x)
        assert torch.equal(q, qr)
        assert torch.equal(s.nan_to_num(nan=-7.0), sr.nan_to_num(nan=-7.0))
    assert torch.isnan(s[6]) and torch.isnan(s[7]) and torch.isnan(s[8]) and s[3] == 1.0 and s[4] == 1.0


@pytest.mark.parametrize("K,off,pitch", [(512, 1, 520), (513, 3, 777), (4096, 0, 4100), (96, 8, 128), (30, 2, 33)])
def test_quant_strided_rows_and_guards(fq, K, off, pitch):
    """Any row start and pitch; the bytes around the codes and scales stay as they were."""
    import torch
    M = 37
    buf = bf16_normal((M + 1, pitch + off), K)
    x = buf.view(-1)[off:off + M * pitch].view(M, pitch)[:, :K]
    qbuf = torch.full((M + 2, K + 24), 99, dtype=torch.int8, device="cuda")
    sbuf = torch.full((M + 5,), -3.0, device="cuda")
    fq.quant_int8_rowwise(x, out=(qbuf[1:M + 1, :K], sbuf[2:M + 2]))
    qr, sr = quant_ref(x)
    assert torch.equal(qbuf[1:M + 1, :K], qr) and torch.equal(sbuf[2:M + 2], sr)
    assert (qbuf[0] == 99).all() and (qbuf[M + 1] == 99).all() and (qbuf[:, K:] == 99).all()
    assert (sbuf[:2] == -3).all() and (sbuf[M + 2:] == -3).all()


# -------------------------------------------------------------------------------- products

def acc_ref(qa, qb):
    return qa.double() @ qb.double().t()


def check_product(C, qa, sa, qb, sb):
    import torch
    ref = acc_ref(qa, qb) * sa.double()[:, None] * sb.double()
    tol = 3.01 * 2.0 ** -24 + (2.0 ** -8 if C.dtype == torch.bfloat16 else 0.0)
    bad = (C.double() - ref).abs() > tol * ref.abs()
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


SHAPES = [(1, 1, 1), (1, 16, 16), (2, 7, 33), (16, 128, 128), (17, 130, 129), (1, 7168, 2048), (64, 96, 4096),
          (65, 2047, 300), (127, 256, 128), (128, 264, 1024), (129, 1000, 2047), (300, 513, 640), (700, 4096, 512), (513, 300, 200), (1000, 2047, 129), (2500, 1100, 1300)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fp32", [False, True])
def test_gemm_int8(fq, M, N, K, fp32):
    import torch
    qa, sa = codes(M, K, 11 * M + K)
    qb, sb = codes(N, K, 13 * N + K)
    C = fq.gemm_int8(qa, sa, qb, sb, out_dtype=torch.float32 if fp32 else torch.bfloat16)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    check_product(C, qa, sa, qb, sb)


@pytest.mark.parametrize("M", [1, 33, 200])
def test_gemm_int8_sums_to_the_int32_limit(fq, M):
    """The longest K with codes of one sign: the sums come within 2^14 of 2^31 and are exact
    (unit scales; the FP32 output is the sum's rounding)."""
    import torch
    K = 131071
    buf = torch.full((M + 40, 131072), -128, dtype=torch.int8, device="cuda")
    qa, qb = buf[:M, :K], buf[M:, :K]
    one = torch.ones(M + 40, device="cuda")
    C = fq.gemm_int8(qa, one, qb, one, out_dtype=torch.float32)
    assert (C == float(np.float32(131071 * 16384))).all()
    with pytest.raises(fq.Fp8qError):
        fq.gemm_int8(buf[:M], one, buf[M:], one)


def gated_ref(qa, sa, qw, sw):
    import torch
    N = qw.shape[0] // 2
    c = acc_ref(qa, qw) * sa.double()[:, None] * sw.double()
    g, u = c[:, :N], c[:, N:]
    h = g * torch.special.expit(g) * u
    tol = (2.0 ** -8 + 2.0 ** -23 * (8 + 2.7 * g.abs())) * h.abs() + 1.2e-36 * u.abs() + 2.0 ** -134
    return h, tol


def check_gated(h, qa, sa, qw, sw):
    ref, tol = gated_ref(qa, sa, qw, sw)
    bad = (h.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_int8_gated(fq, M, N, K):
    import torch
    qa, sa = codes(M, K, 17 * M + K)
    qw, sw = codes(2 * N, K, 19 * N + K)
    h = fq.gemm_int8_gated(qa, sa, qw, sw)
    torch.cuda.synchronize()
    assert fq.device_error() == 0
    check_gated(h, qa, sa, qw, sw)


@pytest.mark.parametrize("M", [2, 40, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_int8_strides_and_guards(fq, M, gated):
    """Padded operands and an output inside a larger buffer, its rows on 16 bytes and not;
    what lies around the output stays as it was."""
    import torch
    N, K = 136, 200
    qa, sa = codes(M, K, 5, pitch=256)
    qb, sb = codes(2 * N if gated else N, K, 6, pitch=208)
    for pitch, off in ((160, 8), (139, 1)):
        for dtype in (torch.bfloat16,) if gated else (torch.bfloat16, torch.float32):
            buf = torch.full((M + 2, pitch + off), 7.0, dtype=dtype, device="cuda")
            out = buf[1:M + 1, off:off + N]
            f = fq.gemm_int8_gated if gated else fq.gemm_int8
            f(qa, sa, qb, sb, out=out)
            (check_gated if gated else check_product)(out, qa, sa, qb, sb)
            out.fill_(7.0)
            assert (buf == 7.0).all()


def test_int8_row_without_finite_scale_is_nan_and_alone(fq):
    """A row of the activations with Inf or NaN gives NaN in its own output row only."""
    import torch
    x = bf16_normal((140, 256), 3)
    x[5, 3] = float("inf")
    x[139, 0] = float("nan")
    w = bf16_normal((2 * 128, 256), 4)
    q, s = fq.quant_int8_rowwise(x)
    qw, sw = fq.quant_int8_rowwise(w)
    for rows in (slice(0, 140), slice(130, 140), slice(0, 8)):
        for C in (fq.gemm_int8(q[rows], s[rows], qw, sw), fq.gemm_int8_gated(q[rows], s[rows], qw, sw)):
            bad = torch.zeros(140, dtype=torch.bool, device="cuda")
            bad[5] = bad[139] = True
            assert torch.equal(torch.isnan(C).any(1), bad[rows]) and torch.equal(torch.isnan(C).all(1), bad[rows])


def test_int8_feed_forward_for_serving(fq):
    """quantize -> gated -> quantize -> product, as a serving block runs it, for a prompt and for
    single tokens: each step against the definition on the step's own inputs, and a token alone
    gives the bits it gives inside the batch."""
    import torch
    T, N, K = 150, 384, 640
    x = bf16_normal((T, K), 21)
    qw, sw = fq.quant_int8_rowwise(bf16_normal((2 * N, K), 22, K ** -0.5))
    qd, sd = fq.quant_int8_rowwise(bf16_normal((K, N), 23, N ** -0.5))

    def block(x):
        q, s = fq.quant_int8_rowwise(x)
        h = fq.gemm_int8_gated(q, s, qw, sw)
        q2, s2 = fq.quant_int8_rowwise(h)
        return q, s, h, q2, s2, fq.gemm_int8(q2, s2, qd, sd)

    q, s, h, q2, s2, y = block(x)
    check_gated(h, q, s, qw, sw)
    qr, sr = quant_ref(h)
    assert torch.equal(q2, qr) and torch.equal(s2, sr)
    check_product(y, q2, s2, qd, sd)
    for t in (0, 77, 149):
        one = block(x[t:t + 1])
        assert torch.equal(one[2], h[t:t + 1]) and torch.equal(one[5], y[t:t + 1])
    assert torch.equal(block(x[:40])[5], y[:40])


def test_int8_on_a_side_stream_and_in_graphs(fq):
    """On another stream, captured, and two captured graphs replayed at the same time."""
    import torch
    qw, sw = fq.quant_int8_rowwise(bf16_normal((512, 2048), 31))
    xs = [bf16_normal((3, 2048), 32), bf16_normal((3, 2048), 33)]
    want = []
    for x in xs:
        q, s = fq.quant_int8_rowwise(x)
        want.append((fq.gemm_int8(q, s, qw, sw), fq.gemm_int8_gated(q, s, qw, sw)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, s = fq.quant_int8_rowwise(xs[0])
        got = fq.gemm_int8(q, s, qw, sw)
    side.synchronize()
    assert torch.equal(got, want[0][0])
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q, s = fq.quant_int8_rowwise(x)
            outs.append((fq.gemm_int8(q, s, qw, sw), fq.gemm_int8_gated(q, s, qw, sw)))
        graphs.append(g)
    other = torch.cuda.Stream()
    for _ in range(20):
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    assert fq.device_error() == 0


def test_int8_empty_batch(fq):
    import torch
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q, s = fq.quant_int8_rowwise(x)
    qw, sw = fq.quant_int8_rowwise(bf16_normal((64, 256), 1))
    assert fq.gemm_int8(q, s, qw, sw).shape == (0, 64)
    assert fq.gemm_int8_gated(q, s, qw, sw).shape == (0, 32)
