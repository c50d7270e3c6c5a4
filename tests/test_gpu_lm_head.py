"""lm_head_logprobs beyond the rows of one NVFP4 product."""
import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8

pytestmark = pytest.mark.gpu


def _head(rows, vocab=1003, k=512):
    x = _fp8.normal(rows, k, 1).to(torch.bfloat16).cuda()
    w = _fp8.normal(vocab, k, 2, 0.05).cuda()
    return x, w, (torch.arange(rows) * 13 % vocab).cuda()


@pytest.mark.parametrize("rows", [256, 257, 512, 700])
@pytest.mark.parametrize("topk", [0, 4])
def test_any_number_of_rows(rows, topk):
    x, w, tokens = _head(rows)
    w8, w4 = fi.pack_weights_fp8(w), fi.pack_weights(w)
    logits4 = torch.cat([fi.mm_bf16_fp4(p, *w4) for p in x.split(256)])
    logits8 = fi.mm_fp8(*fi.quantize_fp8(x), *w8, out_dtype=torch.float32)
    for weight, logits in ((w8, logits8), (w4, logits4)):
        got = fi.lm_head_logprobs(x, weight, tokens, topk=topk)
        z = torch.log_softmax(logits.double(), 1)
        assert [tuple(t.shape) for t in got] == [(rows,)] * 3 + [(rows, topk)] * 2
        # logits of magnitude 10 at most: the bound of the small log probability tests
        assert bool((got.logprob.double() - z.gather(1, tokens[:, None])[:, 0]).abs().max() < 1e-5)
        ref = fi.token_logprobs(logits, tokens, topk=topk)
        assert torch.equal(got.rank, ref.rank) and torch.equal(got.top_ids, ref.top_ids)


def test_rows_and_tokens_have_to_agree():
    x, w, tokens = _head(300)
    w4 = fi.pack_weights(w)
    for bad in (tokens[:299], torch.cat([tokens, tokens[:1]]), tokens[:, None], tokens.int(), tokens.cpu()):
        with pytest.raises(ValueError, match="tokens"):
            fi.lm_head_logprobs(x, w4, bad)
    with pytest.raises(ValueError, match="A must be"):
        fi.lm_head_logprobs(x.float(), w4, tokens)
