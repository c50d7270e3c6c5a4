"""Token log probabilities, entropy, rank and alternatives on the GPU."""
import math

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _order(z):
    """Indices in the order (value descending, NaN first; index ascending), of 64-bit logits."""
    key = torch.where(torch.isnan(z), torch.full_like(z, INF), z)
    first = torch.isnan(z)
    idx = torch.argsort(key, dim=1, descending=True, stable=True)
    # a NaN comes before an infinity: a second stable sort by that alone
    return idx.gather(1, torch.argsort(first.gather(1, idx).to(torch.uint8), dim=1, descending=True, stable=True))


def _reference(logits, tokens, topk):
    z = logits.cpu().double()
    rows, vocab = z.shape
    t = tokens.cpu()
    inside = (t >= 0) & (t < vocab)
    tt = t.clamp(0, vocab - 1)
    empty = (z == -INF).all(1)
    # relative to the maximum first: next to one of 3e38 a logarithm is below a 64-bit step (2^75)
    d = torch.where(empty[:, None], z, z - z.amax(1, keepdim=True))
    y = torch.where(empty[:, None], z, d - d.exp().sum(1, keepdim=True).log())
    plogp = torch.where(y == -INF, 0.0, y * y.exp())
    entropy = torch.where(empty, 0.0, -plogp.sum(1))
    bad = torch.isnan(z).any(1) | (z == INF).any(1)
    y = torch.where(bad[:, None], NAN, y)
    entropy = torch.where(bad, NAN, entropy)
    order = _order(z)
    place = torch.empty_like(order).scatter_(1, order, torch.arange(vocab).expand(rows, -1))
    ids = order[:, :min(topk, vocab)]
    return {"logprob": torch.where(inside, y.gather(1, tt[:, None])[:, 0], NAN), "entropy": entropy,
            "rank": torch.where(inside, place.gather(1, tt[:, None])[:, 0], -1),
            "top_logprobs": y.gather(1, ids), "top_ids": ids}


def _check(logits, tokens, topk, got=None):
    got = (got or fi.token_logprobs(logits, tokens, topk=topk))._asdict()
    ref = _reference(logits, tokens, topk)
    vocab = logits.shape[1]
    # the sum of exponentials: a thread adds at most vocab / 256 + 8 terms in a row and 16 joins
    # follow, each off by 2^-24; each exponential by 2 units of 2^-23, twice that for its argument's
    # rounding over differences up to 40 (weighted by the exponentials themselves); the logarithm
    # by 2^-21 absolutely
    r = (vocab / 256 + 24) * 2.0 ** -24 + 4 * 2.0 ** -23 + 40 * 2.0 ** -23 + 2.0 ** -21
    for name in ("logprob", "top_logprobs", "entropy"):
        x, y = got[name].cpu().double(), ref[name]
        assert got[name].dtype == torch.float32 and x.shape == y.shape, name
        assert torch.equal(torch.isnan(x), torch.isnan(y)), (name, x, y)
        assert torch.equal(torch.isinf(x), torch.isinf(y)), (name, x, y)
        fine = torch.isfinite(y)
        # the entropy's second sum has the same relative error on a value of at most ln(vocab) + 1
        tol = r + 3 * 2.0 ** -24 * y.abs() if name != "entropy" else torch.full_like(y, 2 * r * (math.log(vocab) + 2))
        assert bool(((x - y).abs() <= tol)[fine].all()), (name, ((x - y).abs() / tol)[fine].max())
    for name in ("rank", "top_ids"):
        assert got[name].dtype == torch.int64 and torch.equal(got[name].cpu(), ref[name]), name


def _logits(rows, vocab, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, vocab), generator=g) * scale).to(dtype)


DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,topk", [(1, 1, 0), (1, 1, 1), (2, 7, 32), (3, 31, 5), (5, 32, 32), (4, 33, 32),
                                             (7, 1000, 20), (1, 4099, 32), (3, 32001, 1), (2, 65537, 20),
                                             (1, 152064, 20), (300, 5001, 7), (1500, 515, 3)])
def test_against_64_bits(dtype, rows, vocab, topk):
    z = _logits(rows, vocab, dtype, rows + vocab).cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(7)).cuda()
    _check(z, tokens, topk)


@pytest.mark.parametrize("dtype", DTYPES)
def test_greatest_and_least_tokens(dtype):
    z = _logits(6, 9001, dtype, 1).cuda()
    for tokens in (z.argmax(1), z.argmin(1), torch.zeros(6, dtype=torch.int64, device="cuda"),
                   torch.full((6,), 9000, device="cuda")):
        _check(z, tokens, 10)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [515, 40000])
def test_ties_go_to_the_lower_index(dtype, vocab):
    g = torch.Generator().manual_seed(2)
    z = torch.stack([torch.full((vocab,), 1.5), torch.randint(0, 3, (vocab,), generator=g).float(),
                     torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0), torch.arange(vocab).float().div(512).floor()])
    tokens = torch.tensor([vocab // 2, 17, 3, vocab - 1]).cuda()
    _check(z.to(dtype).cuda(), tokens, 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [2, 1300])
def test_ties_at_the_ends_of_unaligned_rows(dtype, rows):
    """Equal greatest values in the first and last elements of rows that start off a 16-byte
    boundary, against equal ones in the middle."""
    vocab = 3000
    big = torch.zeros((rows, vocab + 9)).to(dtype)
    big[:, 4:4 + vocab] = _logits(rows, vocab, dtype, 12).clamp(max=5)
    big[:, 5:9] = 6.0
    big[:, 1500:1520] = 6.0
    big[:, vocab - 2:vocab + 4] = 6.0
    for off in (1, 3, 5):
        z = big.cuda()[:, off:off + vocab]
        _check(z, torch.full((rows,), vocab - 1).cuda(), 7)
        _check(z, torch.full((rows,), 1510).cuda(), 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [700, 50000])
def test_sorted_rows(dtype, vocab):
    """The worst orders for a running list: every element is a new best, or the first ones stay."""
    z = torch.linspace(-20, 20, vocab)
    z = torch.stack([z, z.flip(0)]).to(dtype).cuda()
    _check(z, torch.tensor([vocab - 3, vocab - 3]).cuda(), 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [515, 50001])
def test_masked_rows(dtype, vocab):
    """Rows with few entries left, one, none; masks of the type's lowest value; masked tokens."""
    low = torch.finfo(dtype).min
    z = _logits(12, vocab, torch.float32, 3)
    z[0] = -INF
    z[1, :] = -INF
    z[1, 400] = 2.0
    z[2, 5:] = -INF
    z[3] = low
    z[4, 1:] = low
    z[5, ::2] = -INF
    z[6] = low
    z[6, 100:] = -INF
    z[7, :-1] = -INF
    z[8] = torch.where(torch.arange(vocab) % 3 == 0, low, -INF)
    z[9, :300] = -INF
    z[10] = -60000.0
    z[11, ::3] = low
    tokens = torch.tensor([3, 400, 0, 9, 0, 1, 99, vocab - 1, 0, 10, 7, 0]).cuda()
    _check(z.to(dtype).cuda(), tokens, 32)
    _check(z.to(dtype).cuda(), torch.full((12,), 14).cuda(), 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [300, 50001])
def test_great_magnitudes(dtype, vocab):
    """Logits of any magnitude: where one step of fp32 is more than the exponential's range, and masks
    of finite values (whole threads, or rows, of nothing else)."""
    sizes = [1e5, 1e7, 2e7, 6e7, 7e7, 1e9, 1e10, 1e12, 1e20, 1e30, 1e37]
    z = torch.cat([_logits(len(sizes), vocab, torch.float32, 8) * torch.tensor(sizes)[:, None],
                   _logits(len(sizes), vocab, torch.float32, 9), _logits(len(sizes), vocab, torch.float32, 10),
                   -torch.tensor(sizes)[:, None] + _logits(len(sizes), vocab, torch.float32, 11)])
    for i, size in enumerate(sizes):
        z[len(sizes) + i, 20:] = -size          # one row's masks
        z[2 * len(sizes) + i, :-20] = -size
        z[2 * len(sizes) + i, -10:] = -INF
    tokens = torch.arange(len(z)) * 5 % vocab
    _check(z.to(dtype).cuda(), tokens.cuda(), 9)
    _check(z.to(dtype).cuda(), z.argmax(1).cuda(), 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 50001])
def test_nan_and_infinite_rows(dtype, vocab):
    z = _logits(8, vocab, torch.float32, 4)
    z[0, 17] = NAN
    z[1, 250] = INF
    z[2, 3], z[2, 200] = INF, NAN
    z[3, 100:110] = NAN
    z[4] = NAN
    z[5] = INF
    z[6] = torch.finfo(dtype).max
    z[7, 11] = torch.finfo(dtype).max
    for tokens in ([17, 0, 5, 105, 8, 9, 10, 11], [4, 250, 3, 2, 0, 0, 0, 12]):
        _check(z.to(dtype).cuda(), torch.tensor(tokens).cuda(), 12)


def test_tokens_outside_the_vocabulary():
    z = _logits(4, 1000, torch.float32, 5).cuda()
    _check(z, torch.tensor([-1, 1000, 2 ** 40, -2 ** 40]).cuda(), 2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_padded_and_unaligned_rows(dtype, offset):
    """Rows of a padded head, further apart than the vocabulary and from any element on; what lies
    between them is not read as part of a row."""
    big = torch.full((9, 4133), 1e4).to(dtype)
    z = _logits(9, 4100, dtype, 6)
    big[:, offset:offset + 4100] = z
    big = big.cuda()
    _check(big[:, offset:offset + 4100], torch.arange(9).cuda() * 400, 9)
    _check(big[4:5, offset:offset + 4100], torch.tensor([4099]).cuda(), 9)


def test_rows_past_2_to_the_31_elements():
    """Row offsets beyond 32 bits."""
    rows, ld = 3, 1 << 30
    buf = torch.empty(((rows - 1) * ld + 1001,), dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (rows, 1001), (ld, 1))
    z.copy_(_logits(rows, 1001, torch.bfloat16, 8))
    _check(z, torch.tensor([5, 6, 7]).cuda(), 5)


def test_entropy_of_known_rows():
    z = torch.stack([torch.zeros(4096), torch.full((4096,), -INF)])
    z[1, :2] = 5.0
    got = fi.token_logprobs(z.cuda(), torch.tensor([0, 1]).cuda())
    assert abs(got.entropy[0].item() - math.log(4096)) < 1e-5
    assert abs(got.entropy[1].item() - math.log(2)) < 1e-6
    assert got.top_ids.shape == (2, 0) and got.top_logprobs.shape == (2, 0)


def test_no_rows():
    got = fi.token_logprobs(torch.empty((0, 10), device="cuda"), torch.empty((0,), dtype=torch.int64, device="cuda"), 3)
    assert [tuple(t.shape) for t in got] == [(0,), (0,), (0,), (0, 3), (0, 3)]


@pytest.mark.parametrize("rows,vocab", [(1, 152064), (40, 20001), (900, 3001)])
def test_repeats_bit_for_bit_on_streams_and_in_graphs(rows, vocab):
    z = _logits(rows, vocab, torch.bfloat16, 9).cuda()
    tokens = (torch.arange(rows) * 37 % vocab).cuda()
    ref = fi.token_logprobs(z, tokens, topk=20)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [fi.token_logprobs(z, tokens, topk=20) for _ in range(3)]
    with torch.cuda.stream(s):
        got += [fi.token_logprobs(z, tokens, topk=20) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = fi.token_logprobs(z, tokens, topk=20)
    for _ in range(2):
        for t in held:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    for r in got + [held]:
        assert all(torch.equal(x, y) for x, y in zip(r, ref))
