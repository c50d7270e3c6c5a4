"""The Python calls of the 8-bit operators and the log probabilities: what they take, make and refuse."""
import threading

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def _operands(m=5, n=300, k=272):
    g = torch.Generator().manual_seed(3)
    a = fi.quantize_fp8(torch.randn((m, k), generator=g).cuda())
    return a, fi.pack_weights_fp8(torch.randn((n, k), generator=g).cuda()), fi.pack_weights_fp8(
        torch.randn((n, k), generator=g).cuda())


def test_outputs_are_what_was_asked_for():
    a, w, u = _operands()
    assert a[0].dtype is F8 and a[0].shape == (5, 272) and a[1].dtype is torch.float32 and a[1].shape == (5, 3)
    assert w[0].shape == (300, 272) and w[1].shape == (3, 3)
    for call in (lambda **kw: fi.mm_fp8(*a, *w, **kw), lambda **kw: fi.mm_fp8_gated(*a, *w, *u, **kw)):
        assert call().dtype is torch.bfloat16 and call().shape == (5, 300)
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            ref = call(out_dtype=dtype)
            out = torch.empty((5, 300), dtype=dtype, device="cuda")
            assert ref.dtype is dtype and not ref.requires_grad and ref.is_contiguous()
            assert call(out=out) is out or call(out=out).data_ptr() == out.data_ptr()
            assert torch.equal(out, ref) and torch.equal(call(out=out, out_dtype=dtype), ref)
    lp = fi.token_logprobs(torch.randn((3, 50), device="cuda"), torch.tensor([0, 1, 2]).cuda(), topk=4)
    assert isinstance(lp, fi.TokenLogprobs) and lp.top_ids is lp[4] and lp._asdict()["rank"].dtype is torch.int64
    with torch.inference_mode():
        assert fi.mm_fp8(*a, *w).is_inference()


def test_products_refuse():
    a, w, u = _operands()
    cases = [
        (lambda: fi.mm_fp8(a[0].float(), a[1], *w), "Aq must be"),
        (lambda: fi.mm_fp8(a[0].cpu(), a[1], *w), "Aq must be"),
        (lambda: fi.mm_fp8(a[0], a[1].double(), *w), "Ascale must be"),
        (lambda: fi.mm_fp8(a[0], a[1][:4], *w), "shape mismatch"),
        (lambda: fi.mm_fp8(a[0], a[1][:, :2].contiguous(), *w), "shape mismatch"),
        (lambda: fi.mm_fp8(*a, w[0][:, :256].contiguous(), w[1]), "shape mismatch"),
        (lambda: fi.mm_fp8(*a, w[0], w[1].t()), "Wscale must be"),
        (lambda: fi.mm_fp8(*a, *w, out_dtype=torch.float64), "bf16, f16 or fp32"),
        (lambda: fi.mm_fp8(*a, *w, out_dtype="bf16"), "bf16, f16 or fp32"),
        (lambda: fi.mm_fp8(*a, *w, out=torch.empty((5, 299), device="cuda")), "out must be"),
        (lambda: fi.mm_fp8(*a, *w, out=torch.empty((300, 5), device="cuda").t()), "out must be"),
        (lambda: fi.mm_fp8(*a, *w, out=torch.empty((5, 300))), "out must be"),
        (lambda: fi.mm_fp8(*a, *w, out=torch.empty((5, 300), device="cuda"), out_dtype=torch.float16), "bf16, f16"),
        (lambda: fi.mm_fp8_gated(*a, *w, u[0][:299], u[1]), "rows"),
        (lambda: fi.mm_fp8_gated(*a, *w, u[0], u[1].half()), "Uscale must be"),
        (lambda: fi.quantize_fp8(torch.zeros((4, 32), device="cuda").t()), "contiguous"),
        (lambda: fi.quantize_fp8(torch.zeros((4, 32), device="cuda", dtype=torch.float64)), "A must be"),
        (lambda: fi.quantize_fp8(torch.zeros((5, 272), device="cuda"), out=(a[0], a[1][:4])), "codes must be"),
        (lambda: fi.pack_weights_fp8(torch.zeros((300, 272), device="cuda"), out=(w[0], a[1])), "codes must be"),
    ]
    for i, (call, word) in enumerate(cases):
        with pytest.raises(ValueError, match=word):
            call()
            pytest.fail(f"case {i} was taken")
    with pytest.raises(fi.FiError, match="multiple of 16"):
        fi.quantize_fp8(torch.zeros((4, 24), device="cuda"))
    # codes that start off a 16-byte boundary
    off = torch.zeros(5 * 272 + 8, dtype=torch.uint8, device="cuda")[8:].view(F8).view(5, 272)
    with pytest.raises(fi.FiError, match="aligned"):
        fi.mm_fp8(off, a[1], *w)


def test_logprobs_refuse():
    z, t = torch.randn((3, 50), device="cuda"), torch.tensor([0, 1, 2]).cuda()
    for call, word in ((lambda: fi.token_logprobs(z.double(), t), "logits must be"),
                       (lambda: fi.token_logprobs(z[0], t), "logits must be"),
                       (lambda: fi.token_logprobs(z.t(), torch.zeros(50, dtype=torch.int64, device="cuda")), "adjacent"),
                       (lambda: fi.token_logprobs(z[:1].expand(3, 50), t), "overlap"),
                       (lambda: fi.token_logprobs(z, t[:2]), "tokens must be"),
                       (lambda: fi.token_logprobs(z, t.int()), "tokens must be"),
                       (lambda: fi.token_logprobs(z, t.cpu()), "tokens must be")):
        with pytest.raises(ValueError, match=word):
            call()
    for topk in (-1, 33, 1 << 70):
        with pytest.raises(fi.FiError, match="topk"):
            fi.token_logprobs(z, t, topk=topk)
    with pytest.raises(TypeError):
        fi.token_logprobs(z, t, topk=2.0)
    with pytest.raises(fi.FiError, match="vocabulary"):
        fi.token_logprobs(z[:, :0], t)


def test_calls_of_several_threads():
    """Each with a stream of its own; the calls let the others run."""
    a, w, _ = _operands(40, 700, 400)
    z, t = torch.randn((9, 3000), device="cuda"), torch.arange(9).cuda()
    ref, lp = fi.mm_fp8(*a, *w), fi.token_logprobs(z, t, topk=6)
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(50):
                    same = torch.equal(fi.mm_fp8(*a, *w), ref)
                    if not (same and all(torch.equal(x, y) for x, y in zip(fi.token_logprobs(z, t, topk=6), lp))):
                        wrong.append("another result")
        except Exception as e:  # an assertion in a thread is not seen
            wrong.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong, wrong[:3]
