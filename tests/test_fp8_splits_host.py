"""Refusals of the 8-bit products with given K splits (no GPU needed): every check precedes the first
CUDA call."""
import ctypes

import pytest

import bf16_activations_nvfp4_b200 as fi

P = ctypes.c_void_p


def _mm(gated, splits, m=4, k=64):
    p = [P(256 * i) for i in range(1, 8)]
    if gated:
        return fi.library().fi_mm_fp8_gated_ex(*p, 0, m, 8, k, splits, None)
    return fi.library().fi_mm_fp8_ex(*p[:5], 0, m, 8, k, splits, None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("splits", [-1, fi.MAX_FP8_SPLITS + 1, 1 << 20])
def test_splits_out_of_range(gated, splits):
    assert _mm(gated, splits) == -1 and "splits" in fi.last_error()
    assert _mm(gated, splits, m=0) == -1


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("splits", [0, 1, fi.MAX_FP8_SPLITS])
def test_splits_in_range(gated, splits):
    assert _mm(gated, splits, m=0) == 0
    assert _mm(gated, splits, k=72) == -2 and "splits" not in fi.last_error()
