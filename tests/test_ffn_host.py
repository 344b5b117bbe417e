"""The 8-bit feed-forward operators on the CPU: the C ABI's refusals (validation returns before any
CUDA call), the binding's operand checks and marshalling (the library call recorded instead
of made), and the gated layer's checks."""
import ctypes

import pytest
import torch

import fp8_fine_grained_weight_b200 as fq
from fp8_fine_grained_weight_b200.linear import fp8_gated_linear

bf16, u8, i8, f32 = torch.bfloat16, torch.uint8, torch.int8, torch.float32
P16, P_MIS, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4097), ctypes.c_void_p(0)
OK, ENULL, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from fp8_fine_grained_weight_b200 import build
    build.build()
    return fq.lib()


def caller(f, **defaults):
    return lambda **kw: f(*dict(defaults, **kw).values())


def test_quant_int8_refusals(L):
    call = caller(L.fp8q_quant_int8_rowwise, x=P16, M=4, K=100, ldx=100, q=P16, ldq=112, s=P16, stream=NULL)
    assert call(M=0) == OK and call(K=0) == OK
    assert call(M=-1) == SHAPE and call(K=-1) == SHAPE
    assert call(x=NULL) == call(q=NULL) == call(s=NULL) == ENULL
    assert call(ldx=99) == SHAPE and call(ldq=99) == SHAPE and call(M=1 << 31) == SHAPE
    assert call(x=P_MIS) == ALIGN and call(s=P_MIS) == ALIGN


def int8_caller(L):
    return caller(L.fp8q_gemm_int8, A=P16, sA=P16, B=P16, sB=P16, C=P16, out=0, M=4, N=9, K=100, lda=112, ldb=112,
                  ldc=9, stream=NULL)


def test_gemm_int8_refusals(L):
    call = int8_caller(L)
    assert call(M=0) == OK
    assert call(M=-1) == call(N=-1) == call(K=-1) == SHAPE
    assert call(N=0) == call(K=0) == SHAPE
    for p in ("A", "sA", "B", "sB", "C"):
        assert call(**{p: NULL}) == ENULL
    assert call(out=2) == UNSUPPORTED
    assert call(K=131072, lda=131072, ldb=131072) == SHAPE        # the sums could pass INT32
    assert call(lda=96) == call(ldb=96) == call(ldc=8) == SHAPE
    assert call(lda=104) == call(ldb=120) == ALIGN                # rows start on 16 bytes
    assert call(A=P_MIS) == call(B=P_MIS) == call(C=P_MIS) == call(sA=P_MIS) == ALIGN
    assert call(C=ctypes.c_void_p(4098), out=1) == ALIGN          # FP32 output on 2 bytes
    assert call(M=1 << 30) == call(N=1 << 30, ldc=1 << 30) == SHAPE


def test_gemm_int8_gated_refusals(L):
    call = caller(L.fp8q_gemm_int8_gated, A=P16, sA=P16, W=P16, sW=P16, H=P16, M=4, N=9, K=100, lda=112, ldw=112,
                  ldh=9, stream=NULL)
    assert call(M=0) == OK
    assert call(N=0) == call(K=131072, lda=131072, ldw=131072) == call(ldh=8) == SHAPE
    assert call(W=NULL) == call(H=NULL) == ENULL
    assert call(ldw=100) == call(H=P_MIS) == ALIGN


@pytest.mark.parametrize("entry", ["fp8_gemm_blockscaled_gated", "fp8_gemm_gated_ue8m0"])
def test_gemm_blockscaled_gated_refusals(L, entry):
    call = caller(getattr(L, entry), A=P16, sA=P16, ld_sa=4, W=P16, sW=P16, H=P16, ldh=256, GU=P16,
                  ldgu=512, M=4, N=256, K=128, lda=128, ldw=128, stream=NULL)
    assert call(M=0) == OK
    assert call(N=200) == call(K=100) == call(M=-1) == call(N=1 << 30, ldh=1 << 30) == SHAPE
    assert call(ld_sa=3) == call(ldh=128) == call(ldgu=511) == call(lda=64) == SHAPE
    for p in ("A", "sA", "W", "sW", "H"):
        assert call(**{p: NULL}) == ENULL
    assert call(GU=P_MIS) == call(ldgu=516) == call(ldh=260) == call(A=P_MIS) == call(lda=136) == ALIGN


def test_gated_backward_refusals(L):
    call = caller(L.fp8q_gated_backward_quant, dH=P16, lddh=256, GU=P16, ldgu=512, M=130, N=256, q=P16, ldq=512, s=P16,
                  ld_s=130, qt=P16, ldqt=256, st=P16, ld_st=512, pow2=0, stream=NULL)
    assert call(M=0) == OK and call(N=0) == OK
    assert call(M=-1) == call(N=200) == call(N=1 << 30) == SHAPE
    for p in ("dH", "GU", "q", "s", "qt", "st"):
        assert call(**{p: NULL}) == ENULL
    assert call(lddh=248) == call(ldgu=504) == call(ldq=504) == call(ld_s=129) == call(ld_st=511) == SHAPE
    assert call(ldqt=240) == SHAPE                                # covers M rounded up to 128
    assert call(lddh=260) == call(ldgu=516) == call(ldq=516) == call(ldqt=264) == ALIGN
    assert call(dH=P_MIS) == call(GU=P_MIS) == call(q=P_MIS) == call(qt=P_MIS) == call(s=P_MIS) == ALIGN


def test_quant_act_dual_padded_refusals(L):
    call = caller(L.fp8q_quant_act_dual_padded, x=P16, M=130, K=256, ldx=256, q=P16, ldq=256, s=P16, ld_s=130, qt=P16,
                  ldqt=256, st=P16, ld_st=256, pow2=0, stream=NULL)
    assert call(M=0) == OK and call(K=0) == OK
    assert call(M=-1) == call(K=200) == call(ldx=128) == call(ldq=248) == call(ld_s=129) == call(ld_st=255) == SHAPE
    assert call(ldqt=240) == SHAPE and call(M=1 << 30, ld_s=1 << 30, ldqt=1 << 30) == SHAPE
    for p in ("x", "q", "s", "qt", "st"):
        assert call(**{p: NULL}) == ENULL
    assert call(ldx=260) == call(ldq=260) == call(ldqt=264) == call(x=P_MIS) == call(qt=P_MIS) == call(s=P_MIS) == ALIGN


def sizes(L, *args):
    out = (ctypes.c_size_t * 3)()
    assert L.fp8q_gated_linear_sizes(*args, out) == OK
    return list(out)


def test_gated_linear_sizes_and_refusals(L):
    """Every buffer of the layer is inside the bytes that it asks for: kept holds g, u (bf16), W's
    codes and scales and X^T's; the scratches the codes and scales of X, and of D, D^T and W^T."""
    up = lambda *n: sum(-(-b // 256) * 256 for b in n)
    for T, N, K in ((1, 128, 128), (200, 256, 384), (256, 384, 640)):
        R, Tp = 2 * N, -(-T // 128) * 128
        w = (R * K, R * K // 4096)
        d = (T * R, T * R // 32, R * Tp, R * Tp // 32)
        assert sizes(L, T, N, K, 1, 1, 1) == [up(2 * T * R, *w, K * Tp, K * Tp // 32), up(T * K, T * K // 32),
                                              up(*d, K * R, K * R // 4096)]
        assert sizes(L, T, N, K, 0, 1, 0)[2] == up(*d)            # (no split-K below 2048)
        assert sizes(L, T, N, K, 1, 0, 0)[0] == up(2 * T * R, *w)
    out = (ctypes.c_size_t * 3)()
    for T, N, K in ((-1, 128, 128), (4, 100, 128), (4, 128, 100), (4, 0, 128), (4, 128, 0), (4, 1 << 30, 128)):
        assert L.fp8q_gated_linear_sizes(T, N, K, 1, 1, 1, out) == SHAPE
    assert L.fp8q_gated_linear_sizes(4, 128, 128, 1, 1, 1, None) == ENULL
    call = caller(L.fp8q_gated_linear_forward, x=P16, w=P16, T=4, N=128, K=128, for_dw=1, pow2=0, kept=P16, scratch=P16,
                  H=P16, stream=NULL)
    assert call(N=100) == call(K=100) == call(T=-1) == SHAPE
    for p in ("x", "w", "kept", "scratch", "H"):
        assert call(**{p: NULL}) == ENULL and call(**{p: P_MIS}) == ALIGN
    call = caller(L.fp8q_gated_linear_backward, dH=P16, kept=P16, T=4, N=128, K=128, for_dw=1, pow2=1, scratch=P16, dX=P16,
                  dW=P16, stream=NULL)
    assert call(T=0) == OK
    assert call(N=100) == call(K=100) == call(T=-1) == SHAPE
    for p in ("dH", "kept", "scratch"):
        assert call(**{p: NULL}) == ENULL
    for p in ("dH", "kept", "scratch", "dX", "dW"):
        assert call(**{p: P_MIS}) == ALIGN
    assert call(for_dw=0) == ENULL                                # dW without what it needs


# ------------------------------------------------------------------------------- the binding

@pytest.fixture
def calls(monkeypatch):
    log = []
    monkeypatch.setattr(fq, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(fq, "_stream", lambda t: 0)
    monkeypatch.setattr(fq, "_call", lambda name, *args: log.append((name, args)))
    return log


def E(*shape, dtype=u8):
    return torch.empty(shape, dtype=dtype)


def test_product_path_requires_cuda_tensors():
    with pytest.raises(TypeError, match="CUDA tensor"):
        fq.quant_int8_rowwise(E(4, 128, dtype=bf16))
    with pytest.raises(TypeError, match="CUDA tensor"):
        fq.gemm_int8(E(4, 16, dtype=i8), E(4, dtype=f32), E(4, 16, dtype=i8), E(4, dtype=f32))
    with pytest.raises(TypeError, match="CUDA tensor"):
        fq.gated_backward_quant(E(4, 128, dtype=bf16), E(4, 256, dtype=bf16))


def test_calls_run_on_the_operands_device(calls, monkeypatch):
    """On a device that is not the current one, the library call is made inside that device's
    context; on the current one, without a switch."""
    entered = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *a):
            entered.append(None)

    class On(torch.Tensor):
        def get_device(self):
            return 3

    t = E(4, 128, dtype=bf16).as_subclass(On)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(fq, "_call", lambda name, *args: entered.append(name))
    fq._launch(t, "a")
    with fq._on(t):
        entered.append("b")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3)
    fq._launch(t, "c")
    with fq._on(t):
        entered.append("d")
    assert entered == [3, "a", None, 3, "b", None, "c", "d"]


def test_quant_int8_marshalling(calls):
    q, s = fq.quant_int8_rowwise(E(5, 100, dtype=bf16))
    assert q.shape == (5, 100) and q.stride() == (112, 1) and s.shape == (5,)
    assert calls[-1][0] == "fp8q_quant_int8_rowwise" and calls[-1][1][1:4] == (5, 100, 100)
    x = E(5, 120, dtype=bf16)[:, 8:108]
    fq.quant_int8_rowwise(x, out=(E(6, 128, dtype=i8), E(7, dtype=f32)))
    assert calls[-1][1][3] == 120 and calls[-1][1][5] == 128
    for bad in ((E(5, 99, dtype=i8), s), (q, E(4, dtype=f32)), (q, E(5, 1, dtype=f32)),
                (q, torch.empty(5, dtype=f32, device="meta"))):
        with pytest.raises(ValueError):
            fq.quant_int8_rowwise(E(5, 100, dtype=bf16), out=bad)
    for bad in (E(5, 100, dtype=torch.float16), E(5, 100, dtype=f32)):
        with pytest.raises(TypeError):
            fq.quant_int8_rowwise(bad)
    with pytest.raises(ValueError):
        fq.quant_int8_rowwise(E(100, 5, dtype=bf16).t())
    with pytest.raises(ValueError):
        fq.quant_int8_rowwise(E(5, 0, dtype=bf16))
    with pytest.raises(TypeError):
        fq.quant_int8_rowwise(E(5, 100, dtype=bf16), out=(E(5, 100), s))


def test_int8_products_marshalling(calls):
    qa, sa, qb, sb = E(5, 112, dtype=i8)[:, :100], E(5, dtype=f32), E(18, 112, dtype=i8)[:, :100], E(18, dtype=f32)
    C = fq.gemm_int8(qa, sa, qb, sb)
    assert C.shape == (5, 18) and C.dtype == bf16 and calls[-1][1][5:12] == (0, 5, 18, 100, 112, 112, 18)
    assert fq.gemm_int8(qa, sa, qb, sb, out_dtype=f32).dtype == f32 and calls[-1][1][5] == 1
    big = E(8, 40, dtype=f32)
    assert fq.gemm_int8(qa, sa, qb, sb, out=big) is big and calls[-1][1][11] == 40
    h = fq.gemm_int8_gated(qa, sa, qb, sb)
    assert h.shape == (5, 9) and h.dtype == bf16 and calls[-1][1][5:11] == (5, 9, 100, 112, 112, 9)
    for f in (fq.gemm_int8, fq.gemm_int8_gated):
        for bad in ((qa, sa, qb[:, :96], sb), (qa, sa[:4], qb, sb), (qa, sa, qb, sb[:17]),
                    (qa, sa, qb, E(36, dtype=f32)[::2]), (qa, sa, qb.to("meta"), sb), (qa[0], sa, qb, sb)):
            with pytest.raises(ValueError):
                f(*bad)
        for bad in ((qa.view(u8), sa, qb, sb), (qa, sa.half(), qb, sb)):
            with pytest.raises(TypeError):
                f(*bad)
        with pytest.raises(ValueError):
            f(qa, sa, qb, sb, out=E(4, 18, dtype=bf16))
    with pytest.raises(TypeError):
        fq.gemm_int8(qa, sa, qb, sb, out=E(5, 18, dtype=torch.float16))
    with pytest.raises(TypeError):
        fq.gemm_int8(qa, sa, qb, sb, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        fq.gemm_int8_gated(qa, sa, qb, sb, out=E(5, 9, dtype=f32))
    with pytest.raises(ValueError, match="even"):
        fq.gemm_int8_gated(qa, sa, qb[:17], sb)


def test_blockscaled_gated_marshalling(calls):
    qa, sa, qw, sw = E(5, 256), E(2, 9, dtype=f32), E(512, 256), E(4, 2, dtype=f32)
    h = fq.gemm_blockscaled_gated(qa, sa, qw, sw)
    assert h.shape == (5, 256) and calls[-1][1][7] is None and calls[-1][1][9:14] == (5, 256, 256, 256, 256)
    h, gu = fq.gemm_blockscaled_gated(qa.view(torch.float8_e4m3fn), sa, qw, sw, with_gu=True)
    assert gu.shape == (5, 512) and calls[-1][1][7] == gu.data_ptr() and calls[-1][1][8] == 512
    assert fq.gemm_blockscaled_gated(qa, sa, qw, sw, with_gu=True, out=(h, gu))[1] is gu
    assert fq.gemm_blockscaled_gated(qa, sa, qw, sw, out=h) is h
    for bad in (dict(out=E(4, 256, dtype=bf16)), dict(with_gu=True, out=(h, E(5, 500, dtype=bf16)))):
        with pytest.raises(ValueError):
            fq.gemm_blockscaled_gated(qa, sa, qw, sw, **bad)
    with pytest.raises(TypeError):
        fq.gemm_blockscaled_gated(qa, sa, qw, sw, out=E(5, 256, dtype=f32))
    with pytest.raises(ValueError, match="multiple of 128"):
        fq.gemm_blockscaled_gated(qa, sa, E(384, 256), E(3, 2, dtype=f32))
    with pytest.raises(ValueError):
        fq.gemm_blockscaled_gated(qa, sa, qw, E(2, 2, dtype=f32))
    with pytest.raises(ValueError):
        fq.gemm_blockscaled_gated(qa, E(2, 4, dtype=f32), qw, sw)


def test_one_column_needs_no_unit_stride(calls):
    """[G, 1] scales of a single token, transposed from [1, G], keep the strides (1, G)."""
    sa = E(1, 2, dtype=f32).t()
    assert sa.stride() == (1, 2)
    fq.gemm_blockscaled_gated(E(1, 256), sa, E(512, 256), E(4, 2, dtype=f32))
    assert calls[-1][1][2] == 1


def test_a_single_rows_stride_is_not_used(calls):
    """[1, M] scales of one K group, transposed from [M, 1], carry the row stride 1; a single row of
    codes may carry any."""
    sa = E(40, 1, dtype=f32).t()
    assert sa.stride(0) == 1
    fq.gemm_blockscaled_gated(E(40, 128), sa, E(256, 128), E(2, 1, dtype=f32))
    assert calls[-1][1][2] >= 40
    one = lambda n, dtype: E(n, 1, dtype=dtype).t()
    fq.quant_int8_rowwise(one(100, bf16))
    assert calls[-1][1][3] >= 100
    fq.gemm_int8(one(100, i8), E(1, dtype=f32), E(3, 112, dtype=i8)[:, :100], E(3, dtype=f32), out=one(3, bf16))
    assert calls[-1][1][9] == 112 and calls[-1][1][11] >= 3
    fq.gemm_int8_gated(one(100, i8), E(1, dtype=f32), E(4, 112, dtype=i8)[:, :100], E(4, dtype=f32), out=one(2, bf16))
    assert calls[-1][1][8] == 112 and calls[-1][1][10] >= 2
    fq.gated_backward_quant(one(128, bf16), one(256, bf16))
    assert calls[-1][1][1] >= 128 and calls[-1][1][3] >= 256


def test_gated_backward_marshalling(calls):
    dh, gu = E(130, 128, dtype=bf16), E(130, 256, dtype=bf16)
    bufs = fq.gated_backward_quant(dh, gu)
    assert [tuple(t.shape) for t in bufs] == [(130, 256), (2, 130), (256, 256), (2, 256)]
    fq.gated_backward_quant(dh, gu, True, out=bufs)
    assert calls[-1][1][-2] == 1
    q, s, qt, st = bufs
    for bad in ((E(129, 256), s, qt, st), (q, s, E(256, 130), st), (q, s, qt, E(1, 256, dtype=f32))):
        with pytest.raises(ValueError):
            fq.gated_backward_quant(dh, gu, out=bad)
    for bad in ((dh, gu[:, :254]), (dh[:, :100], E(130, 200, dtype=bf16)), (dh, gu[:129])):
        with pytest.raises(ValueError):
            fq.gated_backward_quant(*bad)
    with pytest.raises(TypeError):
        fq.gated_backward_quant(dh.float(), gu)


def test_gated_linear_refusals():
    ok = E(4, 128, dtype=bf16)
    for x, w in ((ok, E(256, 256, dtype=bf16)), (ok, E(128, 128, dtype=bf16)), (ok[0], E(256, 128, dtype=bf16)),
                 (E(4, 100, dtype=bf16), E(256, 100, dtype=bf16)), (ok, E(0, 128, dtype=bf16)),
                 (ok, E(2, 128, 128, dtype=bf16))):
        with pytest.raises(ValueError):
            fp8_gated_linear(x, w)
    with pytest.raises(TypeError, match="CUDA tensor"):
        fp8_gated_linear(ok, E(256, 128, dtype=bf16))


def test_gated_linear_refuses_other_types(monkeypatch):
    import fp8_fine_grained_weight_b200.linear as linear
    monkeypatch.setattr(linear, "_require_cuda", lambda t, name: None)
    for x, w in ((E(4, 128, dtype=f32), E(256, 128, dtype=bf16)), (E(4, 128, dtype=bf16), E(256, 128, dtype=f32))):
        with pytest.raises(TypeError, match="bfloat16"):
            fp8_gated_linear(x, w)
    with pytest.raises(ValueError, match="is on"):
        fp8_gated_linear(E(4, 128, dtype=bf16), E(256, 128, dtype=bf16).to("meta"))
