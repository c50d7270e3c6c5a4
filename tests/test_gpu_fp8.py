"""8-bit codes with a scale per block of 128, and their products, on the GPU."""
import os
import subprocess
import sys

import pytest
import torch

import bf16_activations_nvfp4_b200 as fi
from tests import _fp8

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _bits(q):
    return q.cpu().view(torch.uint8)


def _assert_codes(x, square):
    rows = 128 if square else 1
    q, s = (fi.pack_weights_fp8 if square else fi.quantize_fp8)(x.cuda())
    oq, os_ = _fp8.quantize(x, rows)
    assert q.dtype == _fp8.E4M3 and s.dtype == torch.float32
    nan = torch.isnan(os_)
    assert torch.equal(torch.isnan(s.cpu()), nan)
    assert torch.equal(s.cpu()[~nan], os_[~nan])
    qn = torch.isnan(oq.float())
    assert torch.equal(torch.isnan(q.cpu().float()), qn)
    assert torch.equal(_bits(q)[~qn], _bits(oq)[~qn])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 48), (1, 128), (7, 144), (33, 2704), (130, 384), (257, 1024),
                                    (1200, 4096)])
@pytest.mark.parametrize("square", [False, True])
def test_codes_and_scales_are_the_definitions(dtype, rows, k, square):
    x = _fp8.normal(rows, k, rows + k, outliers=True)
    x = x * torch.exp(3 * _fp8.normal(rows, 1, 5)).clamp(1e-4, 1e4)  # rows of many sizes
    _assert_codes(x.to(dtype), square)


@pytest.mark.parametrize("square", [False, True])
def test_codes_of_special_values(square):
    """Zero blocks and signed zeros, midpoints between codes, subnormal scales, the largest
    values, infinities and NaN, each in a block of its own."""
    x = torch.zeros(14 * 128, 256)
    r = 128  # a row block apart, so that no two share a weight block
    x[1 * r, 5] = -0.0
    x[2 * r, :16] = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10, 0.0,
                                  -0.0, 432, 416, -432, 2.0 ** -9, 1.5 * 2.0 ** -9])
    x[3 * r, :128] = 1.4 * 2.0 ** -140
    x[4 * r, :4] = torch.tensor([1.0, 2.0, 3.0, -2.5]) * 2.0 ** -148
    x[5 * r, :3] = torch.tensor([3.4e38, -3.4e38, 1e38])
    x[6 * r, :3] = torch.tensor([float("inf"), 1.0, -2.0])
    x[7 * r, 130] = float("nan")
    x[7 * r, :2] = torch.tensor([1.0, -1.0])
    x[8 * r, 255] = float("-inf")
    x[9 * r, :3] = torch.tensor([1e-30, 1e-38, 1e-45])
    x[10 * r, :128] = torch.linspace(-1, 1, 128)
    _assert_codes(x, square)


def test_codes_near_every_border():
    """Values at and one fp32 step around the midpoints between neighbouring codes, for scales of
    many mantissas: the quotient decides, as one IEEE division gives it."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(_fp8.E4M3).float()
    mid = (codes[1:] + codes[:-1]) / 2
    g = torch.Generator().manual_seed(3)
    rows = []
    for _ in range(400):
        s = (1 + torch.rand(1, generator=g)) * 2.0 ** int(torch.randint(-20, 20, (1,), generator=g))
        v = torch.cat([mid[1:] * s, mid[:1] * s])[:127]
        v = torch.nextafter(v, v * torch.randint(0, 3, v.shape, generator=g))
        rows.append(torch.cat([v[:126], (448 * s).repeat(2)]))
    _assert_codes(torch.stack(rows), False)


def test_codes_into_given_tensors():
    x = _fp8.normal(20, 272, 1).to(torch.bfloat16).cuda()
    q = torch.zeros((22, 272), dtype=_fp8.E4M3, device="cuda")
    s = torch.full((22, 3), 7.0, device="cuda")
    a, b = fi.quantize_fp8(x, out=(q[:20], s[:20]))
    assert a.data_ptr() == q.data_ptr() and b.data_ptr() == s.data_ptr()
    oq, os_ = _fp8.quantize(x, 1)
    assert torch.equal(_bits(q[:20]), _bits(oq)) and torch.equal(s[:20].cpu(), os_)
    assert bool((q[20:].float() == 0).all()) and bool((s[20:] == 7).all())


def test_empty_codes():
    for fn in (fi.quantize_fp8, fi.pack_weights_fp8):
        q, s = fn(torch.empty((0, 64), device="cuda"))
        assert q.shape == (0, 64) and s.shape == (0, 1)


# ------------------------------------------------------------------------------ products

def _whole(r, c, rows, seed):
    """Codes of small whole numbers and scales of powers of two: every sum is exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-4, 5, (r, c), generator=g).float().to(_fp8.E4M3)
    s = 2.0 ** torch.randint(-3, 3, (-(-r // rows), -(-c // 128)), generator=g).float()
    return q, s


SIZES_NK = [(1, 16), (127, 128), (128, 144), (129, 272), (300, 2704), (512, 4096), (2000, 1040)]
SIZES_M = [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("m", SIZES_M)
@pytest.mark.parametrize("n,k", SIZES_NK)
def test_whole_numbers_are_exact(m, n, k):
    a, w = _whole(m, k, 1, m + k), _whole(n, k, 128, n + k)
    ref, _ = _fp8.product(a, w)
    buf = torch.full((m + 2, n), 7.0, device="cuda")
    out = fi.mm_fp8(*_fp8.cuda(a), *_fp8.cuda(w), out=buf[1:m + 1])
    assert torch.equal(out.cpu().double(), ref)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("m,n,k", [(2500, 5000, 400), (3000, 2501, 128), (257, 20000, 16), (65, 39001, 272),
                                   (96, 10304, 2704)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tiles(m, n, k, dtype):
    """More output tiles than the GPU holds at once, with ragged edges, in every type; rows around
    the output stay as they were."""
    a, w = _whole(m, k, 1, 1), _whole(n, k, 128, 2)
    ref, _ = _fp8.product(a, w)
    buf = torch.full((m + 2, n), 7.0, device="cuda", dtype=dtype)
    fi.mm_fp8(*_fp8.cuda(a), *_fp8.cuda(w), out=buf[1:m + 1])
    _fp8.check(buf[1:m + 1], ref, torch.zeros_like(ref))
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("m,n,k", [(2500, 3000, 400), (1300, 2501, 144)])
def test_many_gated_tiles(m, n, k):
    a, g, u = _whole(m, k, 1, 1), _whole(n, k, 128, 2), _whole(n, k, 128, 3)
    g = (g[0], g[1] * 2.0 ** -8)
    (gr, gm), (ur, um) = _fp8.product(a, g), _fp8.product(a, u)
    ref, tol = _fp8.gated(gr, 0 * gm, ur, 0 * um, k)
    _fp8.check(fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u)), ref, tol)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 2048), (3, 1000, 2688), (16, 640, 7168), (31, 513, 5120), (77, 1030, 2704),
                                   (200, 384, 1024), (300, 500, 1040), (1100, 900, 656), (2048, 1024, 1024)])
def test_products(dtype, m, n, k):
    a = _fp8.quantize(_fp8.normal(m, k, 1, outliers=True), 1)
    w = _fp8.quantize(_fp8.normal(n, k, 2, 0.02), 128)
    out = fi.mm_fp8(*_fp8.cuda(a), *_fp8.cuda(w), out_dtype=dtype)
    assert out.dtype == dtype and out.shape == (m, n)
    _fp8.check_product(out, *_fp8.product(a, w), k)


@pytest.mark.parametrize("m", SIZES_M)
@pytest.mark.parametrize("n,k", [(1, 16), (127, 128), (129, 272), (300, 2704), (512, 4096)])
def test_gated_products(m, n, k):
    a, g, u = _whole(m, k, 1, m + k), _whole(n, k, 128, n + k), _whole(n, k, 128, n + k + 1)
    g = (g[0], g[1] * 2.0 ** -8)  # gates on both sides of where the activation bends
    (gr, gm), (ur, um) = _fp8.product(a, g), _fp8.product(a, u)
    ref, tol = _fp8.gated(gr, 0 * gm, ur, 0 * um, k)  # exact sums: only the activation's error
    for dtype in DTYPES:
        buf = torch.full((m + 2, n), 7.0, device="cuda", dtype=dtype)
        fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u), out=buf[1:m + 1])
        _fp8.check(buf[1:m + 1], ref, tol)
        assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("m,n,k", [(1, 640, 5120), (40, 1000, 2704), (500, 640, 1024)])
def test_gated_products_of_quantised_values(m, n, k):
    a = _fp8.quantize(_fp8.normal(m, k, 1, outliers=True), 1)
    g = _fp8.quantize(_fp8.normal(n, k, 2, 0.02), 128)
    u = _fp8.quantize(_fp8.normal(n, k, 3, 0.02), 128)
    (gr, gm), (ur, um) = _fp8.product(a, g), _fp8.product(a, u)
    ref, tol = _fp8.gated(gr, gm, ur, um, k)
    out = fi.mm_fp8_gated(*_fp8.cuda(a), *_fp8.cuda(g), *_fp8.cuda(u), out_dtype=torch.float32)
    _fp8.check(out, ref, tol)


def test_halves_of_a_fused_weight():
    n, k = 256, 528
    w = _fp8.cuda(_fp8.quantize(_fp8.normal(2 * n, k, 2, 0.02), 128))
    a = _fp8.cuda(_fp8.quantize(_fp8.normal(9, k, 1), 1))
    out = fi.mm_fp8_gated(*a, w[0][:n], w[1][:n // 128], w[0][n:], w[1][n // 128:], out_dtype=torch.float32)
    both = fi.mm_fp8(*a, *w, out_dtype=torch.float32).double()
    ref = torch.nn.functional.silu(both[:, :n]) * both[:, n:]
    # the same sums in another order of splits at most: a few units of 2^-24 around cancellation
    assert bool(((out.double() - ref).abs() <= 1e-5 * ref.abs() + 1e-6).all())


def test_a_row_of_nan_and_an_empty_row_stay_alone():
    m, n, k = 40, 300, 1024
    x = _fp8.normal(m, k, 4)
    x[3, 200] = float("nan")
    x[7] = 0
    a, w = fi.quantize_fp8(x.cuda()), _fp8.cuda(_fp8.quantize(_fp8.normal(n, k, 2, 0.02), 128))
    out = fi.mm_fp8(*a, *w)
    gat = fi.mm_fp8_gated(*a, *w, *w)
    for o in (out, gat):
        assert bool(torch.isnan(o[3]).all()) and bool((o[7] == 0).all())
        assert int(torch.isnan(o).any(1).sum()) == 1


@pytest.mark.parametrize("out_dtype", [torch.float16])
def test_f16_overflows_to_infinity(out_dtype):
    a = (torch.full((2, 128), 448.0).to(_fp8.E4M3).cuda(), torch.ones((2, 1), device="cuda"))
    w = (torch.full((5, 128), 448.0).to(_fp8.E4M3).cuda(), torch.ones((1, 1), device="cuda"))
    assert bool(torch.isinf(fi.mm_fp8(*a, *w, out_dtype=out_dtype)).all())


def test_empty_products():
    def codes(r, c, rows):
        return (torch.zeros((r, c), dtype=torch.uint8, device="cuda").view(_fp8.E4M3),
                torch.zeros((-(-r // rows), -(-c // 128)), device="cuda"))
    assert fi.mm_fp8(*codes(0, 64, 1), *codes(5, 64, 128)).shape == (0, 5)
    assert fi.mm_fp8(*codes(3, 64, 1), *codes(0, 64, 128)).shape == (3, 0)
    out = torch.full((3, 5), 7.0, device="cuda")
    assert bool((fi.mm_fp8(*codes(3, 0, 1), *codes(5, 0, 128), out=out) == 0).all())
    out.fill_(7)
    assert bool((fi.mm_fp8_gated(*codes(3, 0, 1), *codes(5, 0, 128), *codes(5, 0, 128), out=out) == 0).all())


@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (16, 4096, 1024), (100, 512, 2048), (700, 512, 1024),
                                   (1500, 5000, 512)])
def test_repeats_bit_for_bit_on_streams_and_in_graphs(m, n, k):
    a = _fp8.cuda(_fp8.quantize(_fp8.normal(m, k, 1, outliers=True), 1))
    w = _fp8.cuda(_fp8.quantize(_fp8.normal(n, k, 2, 0.02), 128))
    u = _fp8.cuda(_fp8.quantize(_fp8.normal(n, k, 3, 0.02), 128))
    mm, gat = fi.mm_fp8(*a, *w), fi.mm_fp8_gated(*a, *w, *u)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):  # two streams at once, each with both products
        with torch.cuda.stream(streams[i % 2]):
            got.append((fi.mm_fp8(*a, *w), fi.mm_fp8_gated(*a, *w, *u)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, mm) and torch.equal(y, gat)
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn: they share nothing
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = fi.mm_fp8(*a, *w), fi.mm_fp8_gated(*a, *w, *u)
        graphs.append((g, o))
    for g, o in graphs + graphs:
        for t in o:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], mm) and torch.equal(o[1], gat)


def test_a_product_reads_what_the_call_before_it_wrote():
    """Weights, activations and scales written by the calls just before, again and again on one
    stream: nothing may be read early."""
    n, k = 1024, 2048
    ws = [_fp8.normal(n, k, s, 0.02).cuda() for s in range(3)]
    xs = [_fp8.normal(8, k, 10 + s).cuda() for s in range(3)]
    ref = []
    for x, w in zip(xs, ws):
        a, b = fi.quantize_fp8(x), fi.pack_weights_fp8(w)
        torch.cuda.synchronize()
        ref.append(fi.mm_fp8(*a, *b))
        torch.cuda.synchronize()
    a, b = fi.quantize_fp8(xs[0]), fi.pack_weights_fp8(ws[0])
    outs = []
    for i in range(30):
        fi.pack_weights_fp8(ws[i % 3], out=b)
        fi.quantize_fp8(xs[i % 3], out=a)
        outs.append(fi.mm_fp8(*a, *b))
    for i, o in enumerate(outs):
        assert torch.equal(o, ref[i % 3]), i


@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (80, 20480, 1024), (200, 512, 1024), (600, 1024, 1024),
                                   (1024, 8192, 1024)])
@pytest.mark.parametrize("gate", [False, True])
def test_stalled_producer_reports_timeout_and_recovers(m, n, k, gate):
    a = _fp8.cuda(_fp8.quantize(_fp8.normal(m, k, 1), 1))
    w = _fp8.cuda(_fp8.quantize(_fp8.normal(n, k, 2, 0.02), 128))

    def call():
        return fi.mm_fp8_gated(*a, *w, *w) if gate else fi.mm_fp8(*a, *w)

    ref = call()
    torch.cuda.synchronize()
    assert fi.get_device_error() == 0
    fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, 20_000_000)
    fi.debug_set(fi.DEBUG_STALL_PRODUCER, 1)
    try:
        call()
        torch.cuda.synchronize()
        assert fi.get_device_error() != 0
        assert fi.get_device_error() == 0
    finally:
        fi.debug_set(fi.DEBUG_STALL_PRODUCER, 0)
        fi.debug_set(fi.DEBUG_WAIT_TIMEOUT_NS, 1_000_000_000)
    assert torch.equal(call(), ref)
    assert fi.get_device_error() == 0


def test_feed_forward_and_head_in_a_row():
    """The calls as a server makes them: activations to codes, the gated half, codes again, the
    down projection, codes, the head in fp32, and the answer; each step against 64 bits on the
    inputs that it was given."""
    m, hidden, wide, vocab = 5, 512, 1408, 3001
    x = _fp8.normal(m, hidden, 1).to(torch.bfloat16).cuda()
    g, u = (fi.pack_weights_fp8(_fp8.normal(wide, hidden, s, 0.05).cuda()) for s in (2, 3))
    d = fi.pack_weights_fp8(_fp8.normal(hidden, wide, 4, 0.05).cuda())
    head = fi.pack_weights_fp8(_fp8.normal(vocab, hidden, 5, 0.5).cuda())
    a = fi.quantize_fp8(x)
    h = fi.mm_fp8_gated(*a, *g, *u)
    b = fi.quantize_fp8(h)
    y = fi.mm_fp8(*b, *d)
    c = fi.quantize_fp8(y)
    logits = fi.mm_fp8(*c, *head, out_dtype=torch.float32)
    tokens = logits.argmax(1)
    lp = fi.token_logprobs(logits, tokens, topk=3)

    def host(p):
        return tuple(t.cpu() for t in p)

    (gr, gm), (ur, um) = _fp8.product(host(a), host(g)), _fp8.product(host(a), host(u))
    ref, tol = _fp8.gated(gr, gm, ur, um, hidden)
    _fp8.check(h, ref, tol)
    assert torch.equal(_bits(b[0]), _bits(_fp8.quantize(h, 1)[0]))
    _fp8.check_product(y, *_fp8.product(host(b), host(d)), wide)
    _fp8.check_product(logits, *_fp8.product(host(c), host(head)), hidden)
    z = torch.log_softmax(logits.cpu().double(), 1)
    assert bool((lp.rank == 0).all()) and torch.equal(lp.top_ids[:, 0], tokens)
    assert bool((lp.logprob.cpu().double() - z.gather(1, tokens.cpu()[:, None])[:, 0]).abs().max() < 1e-5)
    assert bool((lp.top_logprobs.cpu().double() - z.topk(3, 1).values).abs().max() < 1e-5)


@pytest.mark.parametrize("rows", [1, 5, 70])
def test_head_and_answer_of_both_weight_formats(rows):
    """lm_head_logprobs is the head product and the answer to its logits, for 8-bit and 4-bit heads."""
    vocab, k = 1003, 512
    x = _fp8.normal(rows, k, 1).to(torch.bfloat16).cuda()
    w = _fp8.normal(vocab, k, 2, 0.05).cuda()
    tokens = (torch.arange(rows) * 13 % vocab).cuda()
    w8, w4 = fi.pack_weights_fp8(w), fi.pack_weights(w)
    for weight, logits in ((w8, fi.mm_fp8(*fi.quantize_fp8(x), *w8, out_dtype=torch.float32)), (w4, fi.mm_bf16_fp4(x, *w4))):
        got, ref = fi.lm_head_logprobs(x, weight, tokens, topk=4), fi.token_logprobs(logits, tokens, topk=4)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        z = torch.log_softmax(logits.double(), 1)
        assert bool((got.logprob.double() - z.gather(1, tokens[:, None])[:, 0]).abs().max() < 1e-5)
        assert torch.equal(got.top_ids[:, 0], logits.float().argmax(1))
    with pytest.raises(ValueError):
        fi.lm_head_logprobs(x, (w,), tokens)


def test_first_calls_inside_a_capture():
    """A process whose first call of each operator is captured: what a call sets up once does not
    break the capture, and the replay gives what the plain calls give afterwards."""
    code = """
import torch
import bf16_activations_nvfp4_b200 as fi
x = torch.randn(40, 512, device="cuda").bfloat16()
big = torch.randn(2000, 512, device="cuda").bfloat16()
w = torch.randn(3000, 512, device="cuda")
t = torch.zeros(40, dtype=torch.int64, device="cuda")
def calls():
    p, a, b = fi.pack_weights_fp8(w), fi.quantize_fp8(x), fi.quantize_fp8(big)
    y = fi.mm_fp8(*a, *p, out_dtype=torch.float32)
    return [y, fi.mm_fp8(*b, *p), fi.mm_fp8_gated(*a, *p, *p), fi.mm_fp8_gated(*b, *p, *p), *fi.token_logprobs(y, t, 5)]
torch.cuda.synchronize()
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    held = calls()
g.replay()
torch.cuda.synchronize()
for a, b in zip(held, calls()):
    assert torch.equal(a, b)
assert fi.get_device_error() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("m", [1, 16, 17, 32, 64])
@pytest.mark.parametrize("n,k", [(40000, 2048), (4096, 4096), (1000, 14336)])
def test_gated_waves_one_after_another(m, n, k):
    """Many CTAs, two on an SM, and calls that follow one another without a pause: an epilogue that falls
    behind its tensor core still sees every block."""
    a = fi.quantize_fp8(_fp8.normal(m, k, 1).cuda())
    w = fi.pack_weights_fp8(_fp8.normal(n, k, 2, 0.02).cuda())
    ref = fi.mm_fp8_gated(*a, *w, *w, out_dtype=torch.float32)
    g, gm = _fp8.product(a, w)
    _fp8.check(ref, *(t.cpu() for t in _fp8.gated(g, gm, g, gm, k)))
    got = [fi.mm_fp8_gated(*a, *w, *w, out_dtype=torch.float32) for _ in range(40)]
    torch.cuda.synchronize()
    assert fi.get_device_error() == 0
    assert all(torch.equal(x, ref) for x in got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k,gate", [(1000, 2506, 256, False), (1000, 2501, 256, False), (1030, 2500, 144, True),
                                        (700, 3001, 128, True)])
def test_outputs_of_any_pitch_and_start(dtype, m, n, k, gate):
    """Many rows whose outputs start off a 16-byte boundary, and off a word; what is beside them stays."""
    a, w, u = _whole(m, k, 1, 1), _whole(n, k, 128, 2), _whole(n, k, 128, 3)
    w = (w[0], w[1] * 2.0 ** -8) if gate else w
    (gr, gm), (ur, um) = _fp8.product(a, w), _fp8.product(a, u)
    ref, tol = _fp8.gated(gr, 0 * gm, ur, 0 * um, k) if gate else (gr, 0 * gm)
    a, w, u = _fp8.cuda(a), _fp8.cuda(w), _fp8.cuda(u)
    for off in (0, 1, 2, 3, 4):
        buf = torch.full((m * n + 16,), 7.0, device="cuda", dtype=dtype)
        out = buf[off:off + m * n].view(m, n)
        fi.mm_fp8_gated(*a, *w, *u, out=out) if gate else fi.mm_fp8(*a, *w, out=out)
        _fp8.check(out, ref, tol)
        assert bool((buf[:off] == 7).all()) and bool((buf[off + m * n:] == 7).all())
