"""The limit of a kernel's waits counts from the end of the kernel before it. Under programmatic launch
a kernel is on the GPU while the one before it still runs; one that runs for longer than the limit must
neither run its successor's waits out nor have its successor write anything early."""
import contextlib

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8, _gpu

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000


@pytest.fixture(scope="module")
def long_call():
    """A call that lets its successor start at once and itself takes many times the limit: one long masked
    row, which one CTA goes through twice."""
    z = torch.full((1, 1 << 26), -float("inf"), dtype=torch.bfloat16, device="cuda")
    token = torch.zeros(1, dtype=torch.int64, device="cuda")
    call = lambda: fi.token_logprobs(z, token)
    call()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    call()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) * 1e6 > 3 * LIMIT_NS, start.elapsed_time(end)
    return call


@contextlib.contextmanager
def short_limit():
    fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, LIMIT_NS)
    try:
        yield
    finally:
        fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, 1_000_000_000)


def _behind(long_call, call):
    """call() alone, and right behind the long call."""
    ref = call()
    torch.cuda.synchronize()
    assert fi.get_device_error() == 0
    with short_limit():
        long_call()
        out = call()
        torch.cuda.synchronize()
        assert fi.get_device_error() == 0
    assert torch.equal(out, ref)


# the tiles of 16, 32, 64, 96, 128 and 256 rows, and CTA pairs
@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (30, 3000, 1024), (64, 3000, 1024), (80, 20480, 1024),
                                   (128, 2048, 2048), (200, 512, 1024), (256, 4096, 14336), (1024, 8192, 1024)])
@pytest.mark.parametrize("gate", [False, True])
def test_products_behind_a_long_kernel(long_call, m, n, k, gate):
    a = fi.quantize_fp8(_fp8.normal(m, k, 1).cuda())
    w = fi.pack_weights_fp8(_fp8.normal(n, k, 2, 0.02).cuda())
    _behind(long_call, lambda: fi.mm_fp8_gated(*a, *w, *w) if gate else fi.mm_fp8(*a, *w))


def test_products_in_a_row_behind_a_long_kernel(long_call):
    """The second product's predecessor is the first, which waits for the long call."""
    a = fi.quantize_fp8(_fp8.normal(40, 1024, 1).cuda())
    w = fi.pack_weights_fp8(_fp8.normal(1024, 1024, 2, 0.02).cuda())
    _behind(long_call, lambda: fi.mm_fp8(*fi.quantize_fp8(fi.mm_fp8(*a, *w)), *w))


@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (30, 3000, 1024), (64, 3000, 1024), (80, 20480, 1024),
                                   (128, 2048, 2048), (200, 512, 1024), (256, 4096, 14336), (1024, 8192, 1024)])
@pytest.mark.parametrize("gate", [False, True])
def test_nothing_is_stored_when_a_wait_ran_out(m, n, k, gate):
    mark = 2.0 ** 100  # far above what the product can give
    a = fi.quantize_fp8(_fp8.normal(m, k, 1).cuda())
    w = fi.pack_weights_fp8(_fp8.normal(n, k, 2, 0.02).cuda())
    out = torch.full((m, n), mark, dtype=torch.bfloat16, device="cuda")
    call = lambda: fi.mm_fp8_gated(*a, *w, *w, out=out) if gate else fi.mm_fp8(*a, *w, out=out)
    with short_limit():
        fi.debug_set(fi.DEBUG_STALL_PRODUCER, 1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            fi.debug_set(fi.DEBUG_STALL_PRODUCER, 0)
    assert fi.get_device_error() != 0
    assert bool((out == mark).all())
    call()
    assert fi.get_device_error() == 0 and not bool((out == mark).any())


# the GEMV's ring with and without K splits; the tensor-core path with either activation mode, and with
# the decoded weights in tensor memory (up to 128 rows) or in shared memory
@pytest.mark.parametrize("m,n,k,tactic", [
    (1, 4096, 14336, fi.make_tactic(fi.KIND_GEMV, 1, 0, 0x22)), (2, 1024, 14336, fi.make_tactic(fi.KIND_GEMV, 4, 0, 0x22)),
    (1, 4096, 14336, fi.TACTIC_DEFAULT), (8, 4096, 14336, fi.make_tactic(fi.KIND_MMA, 1, 0, 1)),
    (8, 4096, 14336, fi.make_tactic(fi.KIND_MMA, 8, 0, 2)), (200, 4096, 4096, fi.make_tactic(fi.KIND_MMA, 1, 0, 1)),
    (200, 4096, 4096, fi.TACTIC_DEFAULT)])
def test_4_bit_products_behind_a_long_kernel(long_call, m, n, k, tactic):
    weights = _gpu.device_weights(n, k, 3)
    x = _fp8.normal(m, k, 1).to(torch.bfloat16).cuda()
    _behind(long_call, lambda: fi.mm_bf16_fp4(x, *weights, tactic=tactic))
