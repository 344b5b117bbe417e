"""The comparisons that GPU tests use turn down outputs that are not numbers."""
import numpy as np
import pytest

from tests._helpers import assert_gemm_close, assert_within


def test_assert_within():
    ref = np.linspace(-2, 2, 12).reshape(3, 4)
    tol = np.full_like(ref, 1e-3)
    assert_within("same", ref, ref, tol)
    assert_within("near", ref + 9e-4, ref, tol)
    one = ref.copy()
    one[1, 2] = np.nan
    for bad in (np.full_like(ref, np.nan), one, ref + 2e-3, np.full_like(ref, np.inf), ref[:2]):
        with pytest.raises(AssertionError):
            assert_within("bad", bad, ref, tol[:len(bad)])
    with pytest.raises(AssertionError):
        assert_within("reference", ref, one, tol)
    with pytest.raises(AssertionError):
        assert_within("infinite on both sides", np.full_like(ref, np.inf), np.full_like(ref, np.inf), tol)


@pytest.mark.parametrize("bf16", [False, True])
def test_assert_gemm_close_rejects_nan(bf16):
    ref, T = np.ones((3, 4)), np.full((3, 4), 2.0)
    one = ref.copy()
    one[2, 0] = np.nan
    assert_gemm_close("same", ref, ref, T, bf16)
    for bad in (np.full_like(ref, np.nan), one):
        with pytest.raises(AssertionError):
            assert_gemm_close("bad", bad, ref, T, bf16)
