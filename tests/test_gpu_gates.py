"""The gated product's activation on exact gates, over the whole range of the exponential."""
import math

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8

pytestmark = pytest.mark.gpu

# every kernel: tiles of 16, 32, 64 and 128 rows, CTA pairs
SIZES = [(16, 300), (29, 129), (64, 1), (128, 640), (200, 640), (1500, 2000)]


def _operands(gates, ups):
    """(a, g, u) whose gates are gates[i] and up values ups[j], both exactly: a block of k of its own for
    each, a one in it, and the values as scales of the rows (codes times scales of powers of two for ups)."""
    m, n = len(gates), len(ups)
    aq = torch.zeros((m, 256))
    aq[:, 0] = aq[:, 128] = 1
    a_s = torch.ones((m, 2))
    a_s[:, 0] = gates
    gq, uq = torch.zeros((n, 256)), torch.zeros((n, 256))
    gq[:, 0] = 1
    uq[:, 128] = ups
    one = torch.ones((-(-n // 128), 2))
    return (aq.to(_fp8.E4M3), a_s), (gq.to(_fp8.E4M3), one), (uq.to(_fp8.E4M3), one)


def _gates(m):
    fixed = torch.tensor([-20.0, -40.0, -80.0, -86.5, -87.5, -88.0, -88.5, -89.0, -100.0, -104.0, -110.0, 0.0, 30.0, 90.0,
                          -1e4, 1e4])[:m]
    g = torch.empty(m).uniform_(-108, 30, generator=torch.Generator().manual_seed(m))
    g[:len(fixed)] = fixed
    return g


def _bound(g, u):
    """silu(g) u as g e / (1 + e) u with e = exp(-|g|) (g / (1 + e) u for g >= 0) in fp32, in steps of 2^-24:
    the exponential is off by 4 (2^-22, the instruction's bound) and 1 more for its correction, which the
    sum halves and rounds (3.5); the reciprocal is off by 2; the product g e, its scaling back, the
    product with the reciprocal and the one with u are each rounded. Below the normal numbers the
    last three of those, and an output of fp32, are each off by 2^-150 (times u)."""
    s = g / (1 + torch.exp(-g)) * u
    return s, (5 + 3.5 + 2 + 4) * 2.0 ** -24 * s.abs() + 4 * 2.0 ** -150 * (u.abs() + 1)


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_exact_gates(m, n, dtype):
    gates = _gates(m)
    ups = torch.tensor([1.0, -1.0, 448.0, 0.0, 2.0 ** -9, -20.0])[torch.arange(n) % 6]
    a, g, u = _operands(gates, ups)
    out = fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u), out_dtype=dtype)
    ref, tol = _bound(gates.double()[:, None], ups.double()[None, :])
    if dtype == torch.float32:
        off = (out.cpu().double() - ref).abs() - tol
        i = int(off.argmax())
        assert bool((off <= 0).all()), (gates[i // n].item(), ups[i % n].item(), out.flatten()[i].item(), ref.flatten()[i].item())
    else:
        _fp8.check(out, ref, tol)


def test_gates_without_end():
    """Gates that are infinite or NaN, as the formula has them: g / (1 + exp(-g)) u, here with u = g."""
    inf = float("inf")
    a, g, _ = _operands(torch.tensor([inf, -inf, float("nan"), 1.0, 3e38, -3e38]), torch.ones(5))
    u = (g[0], g[1].clone())
    u[1][:] = 2.0 ** -120
    out = fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u), out_dtype=torch.float32).cpu()
    assert bool((out[0] == inf).all()) and bool(torch.isnan(out[1:3]).all())
    silu = 1 / (1 + math.exp(-1))
    assert bool(torch.isclose(out[3], torch.tensor(silu * 2.0 ** -120), rtol=2.0 ** -20, atol=0).all())
    assert bool((out[4] == inf).all())  # 3e38 times 226
    assert bool((out[5] == 0).all())


def test_up_values_without_end_stay_in_their_rows():
    inf = float("inf")
    a, g, u = _operands(torch.tensor([inf, -inf, float("nan"), 1.0]), torch.ones(5))
    a[1][3, 0] = 3e38
    out = fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u), out_dtype=torch.float32).cpu()
    # an infinite scale makes the zero codes of the up weights NaN, too
    assert bool(torch.isnan(out[:3]).all())
    assert bool(torch.isclose(out[3], torch.tensor(3e38)).all())
