"""The stall hook counts launches down exactly, whichever threads launch."""
import threading

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8, _gpu

pytestmark = pytest.mark.gpu

RING = fi.make_tactic(fi.KIND_GEMV, 1, 0, 0x22)  # a stalled launch leaves its output as it was


def test_launches_of_several_threads_are_counted_once():
    n, k, threads, each, stalled = 64, 1024, 8, 100, 250
    weights = _gpu.device_weights(n, k, 3)
    x = _fp8.normal(1, k, 1).to(torch.bfloat16).cuda()
    mark = 2.0 ** 100  # far above what the product can give
    outs = [torch.full((each, 1, n), mark, dtype=torch.bfloat16, device="cuda") for _ in range(threads)]
    torch.cuda.synchronize()
    start = threading.Barrier(threads)
    wrong = []

    def work(out):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for i in range(each):
                    fi.mm_bf16_fp4(x, *weights, tactic=RING, out=out[i])
        except Exception as e:  # an assertion in a thread is not seen
            wrong.append(repr(e))

    fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, 1_000_000)
    fi.debug_set(fi.DEBUG_STALL_PRODUCER, stalled)
    try:
        workers = [threading.Thread(target=work, args=(o,)) for o in outs]
        for w in workers:
            w.start()
        for w in workers:
            w.join()
        torch.cuda.synchronize()
    finally:
        fi.debug_set(fi.DEBUG_STALL_PRODUCER, 0)
        fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, 1_000_000_000)
    assert fi.get_device_error() != 0 and not wrong, wrong[:3]
    untouched = torch.stack(outs) == mark
    assert bool((untouched.all(-1) == untouched.any(-1)).all())
    assert int(untouched.all(-1).sum()) == stalled
