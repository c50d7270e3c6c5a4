"""The block-scaled 8-bit products and the token log probabilities, as cases to be timed and checked.

`run` computes them with elementary torch operations, or through the package's entry points where `own` is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decode step's activations (32 sequences) into the down projection of 4096 x 14336
        {"name": "quantize decode m=32", "op": "quantize", "m": 32, "k": 14336, "dtype": "bf16"},
        # a prompt of 8192 tokens; rows of 21 groups of 128
        {"name": "quantize prompt m=8192", "op": "quantize", "m": 8192, "k": 2688, "dtype": "bf16"},
        # weight preparation: the smallest weight of the library's tests, and a feed-forward weight in bf16
        {"name": "pack 512x2048", "op": "pack", "n": 512, "k": 2048, "dtype": "f32"},
        {"name": "pack 14336x4096", "op": "pack", "n": 14336, "k": 4096, "dtype": "bf16"},
        # single-token decode: the weight is streamed once
        {"name": "mm m=1 4096x14336", "op": "mm", "m": 1, "n": 4096, "k": 14336, "out": "bf16"},
        # a ragged batch with an output width and a k that no tile divides
        {"name": "mm m=77 10300x2704", "op": "mm", "m": 77, "n": 10300, "k": 2704, "out": "f16"},
        # a prompt of 8192 tokens through a down projection: bound by the tensor cores
        {"name": "mm m=8192 4096x14336", "op": "mm", "m": 8192, "n": 4096, "k": 14336, "out": "bf16"},
        # the lm_head of 64 sequences, logits kept in 32 bits
        {"name": "mm m=64 152064x5120 f32", "op": "mm", "m": 64, "n": 152064, "k": 5120, "out": "f32"},
        # the gate/up half of a feed-forward block (34816 x 5120 fused): a decode batch and a prompt
        {"name": "gated m=16 17408x5120", "op": "gated", "m": 16, "n": 17408, "k": 5120, "out": "bf16"},
        {"name": "gated m=4096 17408x5120", "op": "gated", "m": 4096, "n": 17408, "k": 5120, "out": "bf16"},
        # one sampled token of one sequence, with the 20 alternatives that a server may return
        {"name": "logprobs 1x152064", "op": "logprobs", "rows": 1, "vocab": 152064, "topk": 20, "dtype": "f32"},
        # prompt log probabilities: a row for each of 2047 prompt tokens
        {"name": "logprobs 2047x152064", "op": "logprobs", "rows": 2047, "vocab": 152064, "topk": 5, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "pack", "mm", "mm", "gated", "logprobs"])
    if op == "quantize":
        return {"op": op, "m": _log(rng, 1, 8192), "k": 16 * _log(rng, 4, 1088), "dtype": rng.choice(list(DTYPES))}
    if op == "pack":
        return {"op": op, "n": _log(rng, 100, 14336), "k": 16 * _log(rng, 8, 896), "dtype": rng.choice(list(DTYPES))}
    if op in ("mm", "gated"):
        while True:
            c = {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 34816), "k": 16 * _log(rng, 8, 1088),
                 "out": rng.choice(list(DTYPES))}
            if c["m"] * c["n"] * c["k"] * (2 if op == "gated" else 1) <= 8192 * 4096 * 14336:
                return c
    while True:
        c = {"op": op, "rows": _log(rng, 1, 4096), "vocab": _log(rng, 1000, 260000), "topk": rng.randint(0, 32),
             "dtype": rng.choice(list(DTYPES))}
        if c["rows"] * c["vocab"] <= 2047 * 152064:
            return c


# ------------------------------------------------------------------------------ the plain forms

def _blocks(x, rows):
    """x [r, c] in 32 bits, padded with zeros to whole blocks of rows x 128: [r', rows, c', 128]."""
    r, c = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -c % 128, 0, -r % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _quantize(x, rows):
    """Codes and scales of blocks of rows x 128: s = amax / 448, q = E4M3(x / s), 0 where s is 0."""
    r, c = x.shape
    b = _blocks(x, rows)
    s = b.abs().amax((1, 3))
    s = s / torch.full_like(s, E4M3_MAX)  # by a tensor: a division, where a number would be a product with its inverse
    d = s[:, None, :, None]
    q = torch.where(d == 0, torch.zeros((), device=x.device), b / d).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.reshape(b.shape[0] * rows, -1)[:r, :c].to(torch.float8_e4m3fn)
    return q, s


def _values(q, s, rows):
    """The values that codes and scales stand for, in 32 bits."""
    r, c = q.shape
    return (_blocks(q, rows) * s[:, None, :, None]).reshape(s.shape[0] * rows, -1)[:r, :c]


def _logprobs(logits, tokens, topk):
    z = logits.float()
    rows, vocab = z.shape
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    # -inf stands for a masked entry: it adds nothing (and not -inf times 0)
    entropy = torch.log(total) - (torch.where(e == 0, torch.zeros((), device=z.device), z - top) * e).sum(1, keepdim=True) / total
    lse = top + torch.log(total)
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)  # integers that sort as the values do
    ids = torch.arange(vocab, device=z.device)
    key = (order << 32) | (0xFFFFFFFF - ids)  # value first, then the lower index
    mine = key.gather(1, tokens[:, None])
    rank = (key > mine).sum(1)
    best = torch.topk(key, min(topk, vocab), 1).values
    at = 0xFFFFFFFF - (best & 0xFFFFFFFF)
    return {"logprob": (z.gather(1, tokens[:, None]) - lse)[:, 0], "entropy": entropy[:, 0], "rank": rank,
            "top_logprobs": z.gather(1, at) - lse, "top_ids": at}


# ------------------------------------------------------------------------------------ the cases

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1009 + 7)

    def normal(r, c, scale=1.0):
        return torch.randn((r, c), generator=g, device="cuda") * scale

    def activations(m, k, dtype):  # normal, 1% of the entries 50 times as large
        a = normal(m, k)
        return torch.where(torch.rand((m, k), generator=g, device="cuda") < 0.01, a * 50, a).to(dtype)

    op = case["op"]
    if op == "quantize":
        return {"case": case, "x": activations(case["m"], case["k"], DTYPES[case["dtype"]])}
    if op == "pack":
        return {"case": case, "x": normal(case["n"], case["k"], 0.02).to(DTYPES[case["dtype"]])}
    if op in ("mm", "gated"):
        s = {"case": case, "a": _quantize(activations(case["m"], case["k"], torch.bfloat16), 1)}
        for name in ("w",) if op == "mm" else ("g", "u"):
            s[name] = _quantize(normal(case["n"], case["k"], 0.02), 128)
        return s
    rows, vocab = case["rows"], case["vocab"]
    z = normal(rows, vocab, 3.0)
    z[torch.rand((rows, vocab), generator=g, device="cuda") < 0.002] = -math.inf  # tokens that the server bans
    tokens = torch.multinomial(torch.softmax(z, 1)[:, :1 << 20], 1, generator=g)[:, 0]  # sampled from the row
    return {"case": case, "logits": z.to(DTYPES[case["dtype"]]), "tokens": tokens}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import bf16_activations_nvfp4_b200 as fi
        if op == "quantize":
            return fi.quantize_fp8(state["x"])
        if op == "pack":
            return fi.pack_weights_fp8(state["x"])
        if op == "mm":
            return fi.mm_fp8(*state["a"], *state["w"], out_dtype=DTYPES[case["out"]])
        if op == "gated":
            return fi.mm_fp8_gated(*state["a"], *state["g"], *state["u"], out_dtype=DTYPES[case["out"]])
        return fi.token_logprobs(state["logits"], state["tokens"], topk=case["topk"])._asdict()
    if op == "quantize":
        return _quantize(state["x"], 1)
    if op == "pack":
        return _quantize(state["x"], 128)
    if op == "logprobs":
        return _logprobs(state["logits"], state["tokens"], case["topk"])
    a = _values(*state["a"], 1)
    if op == "mm":
        return (a @ _values(*state["w"], 128).T).to(DTYPES[case["out"]])
    gate = a @ _values(*state["g"], 128).T
    return (gate / (1 + torch.exp(-gate)) * (a @ _values(*state["u"], 128).T)).to(DTYPES[case["out"]])


def work(case):
    op = case["op"]
    if op in ("quantize", "pack"):
        rows, k, tall = (case["m"], case["k"], 1) if op == "quantize" else (case["n"], case["k"], 128)
        return {"bytes": rows * k * (SIZE[case["dtype"]] + 1) + 4 * -(-rows // tall) * -(-k // 128), "flops": 3 * rows * k}
    if op in ("mm", "gated"):
        m, n, k, w = case["m"], case["n"], case["k"], 2 if op == "gated" else 1
        kb = -(-k // 128)
        return {"bytes": m * k + w * n * k + 4 * kb * (m + w * -(-n // 128)) + SIZE[case["out"]] * m * n,
                "flops": 2 * w * m * n * k}
    rows, vocab = case["rows"], case["vocab"]
    return {"bytes": rows * vocab * SIZE[case["dtype"]] + rows * (8 + 4 + 4 + 8 + 12 * min(case["topk"], vocab)),
            "flops": 7 * rows * vocab}


# ------------------------------------------------------------------- the definitions in 64 bits

def _e4m3(x):
    """The nearest E4M3 value (ties to the even one) of 64-bit values: steps of 2^(e-3), e at least -6, at most 448."""
    e = torch.frexp(x)[1].sub(1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantize(x, rows):
    """Strip by strip: the scale and each quotient are rounded once to 32 bits, as the format says, then the code."""
    r, c = x.shape
    q = torch.zeros((r, c), dtype=torch.float64, device=x.device)
    s = torch.zeros((-(-r // rows), -(-c // 128)), dtype=torch.float64, device=x.device)
    for j in range(s.shape[1]):
        v = x[:, 128 * j:128 * j + 128].double()
        group = torch.arange(r, device=x.device) // rows
        amax = torch.zeros(s.shape[0], dtype=torch.float64, device=x.device)
        amax.scatter_reduce_(0, group, v.abs().amax(1), "amax")
        s[:, j] = (amax / E4M3_MAX).float().double()
        d = s[:, j][group][:, None]
        q[:, 128 * j:128 * j + 128] = torch.where(d > 0, _e4m3((v / d.clamp(min=1e-300)).float().double()), 0.0)
    return q, s


def _exact_product(a, w):
    """Block by block of 128 k."""
    (aq, sa), (wq, sw) = a, w
    n, k = wq.shape
    out = torch.zeros((aq.shape[0], n), dtype=torch.float64, device=aq.device)
    for j in range(-(-k // 128)):
        b = slice(128 * j, 128 * j + 128)
        right = wq[:, b].double() * sw[:, j].double().repeat_interleave(128)[:n, None]
        out.addmm_(aq[:, b].double() * sa[:, j].double()[:, None], right.T)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("quantize", "pack"):
        return _exact_quantize(s["x"], 1 if op == "quantize" else 128)
    if op == "mm":
        return _exact_product(s["a"], s["w"])
    if op == "gated":
        gate = _exact_product(s["a"], s["g"])
        return gate * torch.sigmoid(gate) * _exact_product(s["a"], s["u"])
    rows, vocab = s["logits"].shape
    k = min(case["topk"], vocab)
    lp, ent = [], []
    best = []
    for i in range(0, rows, 64):  # a few rows at a time: 64-bit copies are large
        z = s["logits"][i:i + 64].double()
        y = torch.log_softmax(z, 1)
        lp.append(y.gather(1, s["tokens"][i:i + 64, None])[:, 0])
        ent.append(-torch.where(torch.isinf(y), 0.0, y * y.exp()).sum(1))
        best.append(torch.topk(y, k, 1).values)
    return {"logprob": torch.cat(lp), "entropy": torch.cat(ent), "rank": None, "top_logprobs": torch.cat(best),
            "top_ids": None}
