"""Token log probabilities are never above 0 and entropies never below: a row with one entry left (as
constrained decoding leaves it) has exactly 0 for both, whatever that entry's value."""
import math

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (rows, vocab): a CTA per row, of each size; a cluster of CTAs per row
SHAPES = [(700, 515), (1500, 40), (300, 40001), (3, 152064), (1, 70001)]


def _values(rows):
    """20.1, -7.3 and others, of both signs and of many mantissas."""
    g = torch.Generator().manual_seed(rows)
    v = torch.randn(rows, generator=g) * 6 + 10
    fixed = torch.tensor([20.1, -7.3, 2.0, 0.1, -0.3, 1000.7, -60000.0])[:rows]
    v[:len(fixed)] = fixed
    return v


def _signs(got):
    for name in ("logprob", "top_logprobs"):
        x = getattr(got, name)
        assert bool(((x <= 0) | torch.isnan(x)).all()), (name, x.max())
    assert bool(((got.entropy >= 0) | torch.isnan(got.entropy)).all()), got.entropy.min()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("topk", [0, 1, 20])
def test_one_entry_left(dtype, rows, vocab, topk):
    for mask in (-math.inf, torch.finfo(dtype).min):
        z = torch.full((rows, vocab), mask, dtype=dtype)
        at = torch.arange(rows) * 37 % vocab
        z[torch.arange(rows), at] = _values(rows).to(dtype)
        got = fi.token_logprobs(z.cuda(), at.cuda(), topk=topk)
        _signs(got)
        assert bool((got.logprob == 0).all()), (mask, got.logprob[got.logprob != 0][:3])
        assert bool((got.entropy == 0).all()), (mask, got.entropy[got.entropy != 0][:3])
        assert bool((got.rank == 0).all())
        if topk:
            assert bool((got.top_logprobs[:, 0] == 0).all()) and torch.equal(got.top_ids[:, 0].cpu(), at)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_nearly_certain_rows(dtype, rows, vocab):
    """One entry far above the others, by 0 to 40."""
    g = torch.Generator().manual_seed(1)
    z = torch.randn((rows, vocab), generator=g) * 0.1 + _values(rows)[:, None].clamp(-40, 40)
    at = torch.arange(rows) * 41 % vocab
    z[torch.arange(rows), at] += torch.linspace(0, 40, rows)
    z = z.to(dtype)
    got = fi.token_logprobs(z.cuda(), at.cuda(), topk=3)
    _signs(got)
    y = torch.log_softmax(z.double(), 1)
    ent = -(y * y.exp()).sum(1)
    # a certain row's: the sum of up to vocab small terms and its logarithm, as the other rows' bound
    # (vocab / 256 + 24 additions of 2^-24, 45 units of 2^-23 in the exponentials, 2^-21 of the logarithm)
    r = (vocab / 256 + 24) * 2.0 ** -24 + 45 * 2.0 ** -23 + 2.0 ** -21
    ref = y[torch.arange(rows), at]
    assert bool(((got.logprob.cpu().double() - ref).abs() <= r + 2.0 ** -22 * ref.abs()).all())
    assert bool(((got.entropy.cpu().double() - ent).abs() <= 2 * r * (math.log(vocab) + 2)).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_signs_of_ordinary_rows(dtype):
    g = torch.Generator().manual_seed(2)
    for rows, vocab, scale in ((2000, 700, 30.0), (40, 50001, 3.0), (9, 65537, 100.0), (2000, 2, 1.0), (500, 1, 9.0)):
        z = (torch.randn((rows, vocab), generator=g) * scale + 5).to(dtype).cuda()
        _signs(fi.token_logprobs(z, z.argmax(1), topk=4))
