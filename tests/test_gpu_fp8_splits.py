"""8-bit products with the number of K splits given: an output's bits follow from its rows, k and that
number alone, whichever kernel and tile the sizes select."""
import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8

pytestmark = pytest.mark.gpu

# tiles of 16, 32, 64, 96, 128 and 256 rows, and CTA pairs
ROWS = [1, 16, 17, 40, 65, 97, 130, 256, 600, 2100]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("splits", [1, 2, 5, 8])
@pytest.mark.parametrize("n,k", [(1000, 2704), (640, 7168), (5000, 400)])
def test_bits_do_not_depend_on_the_number_of_rows(n, k, splits, gate, dtype):
    a = _fp8.cuda(_fp8.quantize(_fp8.normal(max(ROWS), k, 1, outliers=True), 1))
    w, u = (_fp8.cuda(_fp8.quantize(_fp8.normal(n, k, s, 0.02), 128)) for s in (2, 3))

    def call(rows, cols=n):
        x, g, v = (t[:rows] for t in a), *(((q[:cols], s[:-(-cols // 128)])) for q, s in (w, u))
        if gate:
            return fi.mm_fp8_gated(*x, *g, *v, out_dtype=dtype, splits=splits)
        return fi.mm_fp8(*x, *g, out_dtype=dtype, splits=splits)

    ref = call(max(ROWS))
    for rows in ROWS:
        assert torch.equal(call(rows), ref[:rows]), rows
    for cols in (1, 129, 300):
        assert torch.equal(call(77, cols), ref[:77, :cols]), cols
        assert torch.equal(call(1500, cols), ref[:1500, :cols]), cols


@pytest.mark.parametrize("splits", [1, 3, 8])
@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (77, 1030, 2704), (200, 384, 1024), (1100, 900, 656)])
def test_products_of_given_splits(m, n, k, splits):
    a = _fp8.quantize(_fp8.normal(m, k, 1, outliers=True), 1)
    w, u = (_fp8.quantize(_fp8.normal(n, k, s, 0.02), 128) for s in (2, 3))
    out = fi.mm_fp8(*_fp8.cuda(a), *_fp8.cuda(w), out_dtype=torch.float32, splits=splits)
    (g, gm), (v, vm) = _fp8.product(a, w), _fp8.product(a, u)
    _fp8.check_product(out, g, gm, k)
    out = fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(w), *_fp8.cuda(u), splits=splits)
    _fp8.check(out, *_fp8.gated(g, gm, v, vm, k))


def test_more_splits_than_blocks_and_none_given():
    a, w = (_fp8.cuda(_fp8.quantize(_fp8.normal(r, 272, s), rows)) for r, s, rows in ((9, 1, 1), (300, 2, 128)))
    three = fi.mm_fp8(*a, *w, splits=3)
    assert torch.equal(fi.mm_fp8(*a, *w, splits=8), three)
    assert torch.equal(fi.mm_fp8(*a, *w, splits=0), fi.mm_fp8(*a, *w))


def test_splits_refused():
    a, w = (_fp8.cuda(_fp8.quantize(_fp8.normal(r, 272, s), rows)) for r, s, rows in ((9, 1, 1), (300, 2, 128)))
    for call in (lambda s: fi.mm_fp8(*a, *w, splits=s), lambda s: fi.mm_fp8_gated(*a, *w, *w, splits=s)):
        for splits in (-1, 9, 1 << 40):
            with pytest.raises(fi.FiError, match="splits"):
                call(splits)
        for splits in (1.0, None, "1"):
            with pytest.raises(TypeError, match="splits"):
                call(splits)
