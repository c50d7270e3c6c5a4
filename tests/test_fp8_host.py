"""Refusals of the 8-bit products and the token log probabilities (no GPU needed): every check
precedes the first CUDA call."""
import ctypes

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi

P = ctypes.c_void_p
INVALID, SHAPE = -1, -2


def _p(x):
    return P(x)


@pytest.mark.parametrize("name", ["fi_fp8_quantize", "fi_fp8_pack_weights"])
@pytest.mark.parametrize("x,dtype,rows,k,q,s,status", [
    (256, 3, 4, 64, 512, 1024, INVALID),
    (256, -1, 4, 64, 512, 1024, INVALID),
    (256, 0, -1, 64, 512, 1024, INVALID),
    (256, 0, 4, -16, 512, 1024, INVALID),
    (256, 0, 4, 40, 512, 1024, SHAPE),
    (256, 0, 1 << 40, 1 << 40, 512, 1024, SHAPE),
    (0, 0, 4, 64, 512, 1024, INVALID),
    (256, 0, 4, 64, 0, 1024, INVALID),
    (256, 0, 4, 64, 512, 0, INVALID),
    (264, 0, 4, 64, 512, 1024, INVALID),
    (256, 0, 4, 64, 520, 1024, INVALID),
    (256, 0, 4, 64, 512, 1026, INVALID),
])
def test_quantize_refusals(name, x, dtype, rows, k, q, s, status):
    assert getattr(fi.library(), name)(_p(x), dtype, rows, k, _p(q), _p(s), None) == status
    assert fi.last_error()


@pytest.mark.parametrize("name", ["fi_fp8_quantize", "fi_fp8_pack_weights"])
def test_quantize_of_nothing_is_a_no_op(name):
    fn = getattr(fi.library(), name)
    assert fn(None, 0, 0, 64, None, None, None) == 0
    assert fn(None, 2, 5, 0, None, None, None) == 0


def _mm(gated, A=256, As=512, W=1024, Ws=2048, U=4096, Us=8192, out=16384, dtype=0, m=4, n=8, k=64):
    if gated:
        return fi.library().fi_mm_fp8_gated(_p(A), _p(As), _p(W), _p(Ws), _p(U), _p(Us), _p(out), dtype, m, n, k, None)
    return fi.library().fi_mm_fp8(_p(A), _p(As), _p(W), _p(Ws), _p(out), dtype, m, n, k, None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), INVALID), (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-16), INVALID),
    (dict(k=72), SHAPE), (dict(m=1 << 40, n=1 << 40), SHAPE), (dict(A=0), INVALID), (dict(As=0), INVALID),
    (dict(W=0), INVALID), (dict(Ws=0), INVALID), (dict(out=0), INVALID), (dict(A=264), INVALID),
    (dict(W=1032), INVALID), (dict(As=514), INVALID), (dict(Ws=2049), INVALID), (dict(out=16385), INVALID),
    (dict(out=16386, dtype=2), INVALID),
])
def test_product_refusals(gated, bad, status):
    assert _mm(gated, **bad) == status
    assert fi.last_error()


@pytest.mark.parametrize("bad", [dict(U=0), dict(Us=0), dict(U=4104), dict(Us=8194)])
def test_gated_product_refusals(bad):
    assert _mm(True, **bad) == INVALID


@pytest.mark.parametrize("gated", [False, True])
def test_products_of_nothing_are_no_ops(gated):
    assert _mm(gated, m=0, A=0, out=0) == 0
    assert _mm(gated, n=0, W=0, out=0) == 0


def _lp(logits=256, dtype=0, rows=2, vocab=100, ld=100, tokens=512, topk=3, lp=1024, ent=2048, rank=4096, tl=8192, ti=16384):
    return fi.library().fi_token_logprobs(_p(logits), dtype, rows, vocab, ld, _p(tokens), topk, _p(lp), _p(ent),
                                          _p(rank), _p(tl), _p(ti), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), INVALID), (dict(rows=-1), INVALID), (dict(vocab=-1), INVALID), (dict(vocab=0), SHAPE),
    (dict(ld=99), INVALID), (dict(topk=-1), INVALID), (dict(topk=33), INVALID), (dict(vocab=1 << 31, ld=1 << 31), SHAPE),
    (dict(logits=0), INVALID), (dict(tokens=0), INVALID), (dict(lp=0), INVALID), (dict(ent=0), INVALID),
    (dict(rank=0), INVALID), (dict(tl=0), INVALID), (dict(ti=0), INVALID), (dict(logits=257), INVALID),
    (dict(logits=258, dtype=2), INVALID), (dict(tokens=516), INVALID), (dict(rank=4100), INVALID),
    (dict(ti=16388), INVALID), (dict(lp=1026), INVALID),
])
def test_logprob_refusals(bad, status):
    assert _lp(**bad) == status
    assert fi.last_error()


def test_logprobs_of_no_rows_is_a_no_op():
    assert _lp(rows=0, logits=0, tokens=0, lp=0, ent=0, rank=0, tl=0, ti=0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 64))
    q, s = torch.zeros((4, 64), dtype=torch.float8_e4m3fn), torch.zeros((4, 1))
    for call in (lambda: fi.quantize_fp8(x), lambda: fi.pack_weights_fp8(x), lambda: fi.quantize_fp8(x.int()),
                 lambda: fi.quantize_fp8("x"), lambda: fi.mm_fp8(q, s, q, s), lambda: fi.mm_fp8_gated(q, s, q, s, q, s),
                 lambda: fi.token_logprobs(x, torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


def test_binding_says_what_is_wrong():
    """The native module takes none of these; the message names the argument."""
    q, s = torch.zeros((4, 64), dtype=torch.float8_e4m3fn), torch.zeros((4, 1))
    for call, word in ((lambda: fi.quantize_fp8(torch.zeros((4, 64)), out=(q,)), "codes, scale"),
                       (lambda: fi.quantize_fp8(torch.zeros((4, 64)), out=(None, None)), "codes, scale"),
                       (lambda: fi.quantize_fp8(None), "A must be"), (lambda: fi.pack_weights_fp8(q), "W must be"),
                       (lambda: fi.mm_fp8(q, s, q, s), "Aq must be"), (lambda: fi.mm_fp8(None, s, q, s), "Aq must be"),
                       (lambda: fi.token_logprobs(None, None), "logits must be")):
        with pytest.raises(ValueError, match=word):
            call()
