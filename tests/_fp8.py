"""Plain forms of the 8-bit products and the token log probabilities for the tests: codes and
scales by the definition's steps on the CPU, sums in 64 bits."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def blocks(x, rows):
    """x [r, c] padded with zeros to whole blocks of rows x 128."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def quantize(x, rows):
    """(codes, scales) of blocks of rows x 128, in fp32 on the CPU (whose division is IEEE's)."""
    r, c = x.shape
    b = blocks(x.cpu().float(), rows).numpy()
    with np.errstate(all="ignore"):
        s = (np.abs(b).max((1, 3)) / np.float32(448)).astype(np.float32)
        d = s[:, None, :, None]
        q = torch.from_numpy(np.where(d == 0, np.float32(0), b / np.where(d == 0, np.float32(1), d)))
    q = q.clamp(-448, 448).reshape(b.shape[0] * rows, -1)[:r, :c].to(E4M3)
    return q, torch.from_numpy(s)


def values(q, s, rows):
    """What codes and scales stand for, in 64 bits."""
    r, c = q.shape
    b = blocks(q.float().double(), rows) * s.double()[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:r, :c]


def product(a, w):
    """(sum, sum of magnitudes) in 64 bits of the products of (codes, scales) a and w."""
    x, y = values(*a, 1), values(*w, 128)
    return x @ y.T, x.abs() @ y.abs().T


def sum_error(k):
    """Bound on the error of a product's fp32 sums, relative to the sum of magnitudes. Within a
    block the tensor core adds 128 exact products, each addition off by at most one unit in the
    last place (2^-23, as it may truncate) of a partial sum; each of the ceil(k / 128) blocks adds
    the rounding of its scales' product and of its addition (2^-24 each), and the joining of up to
    8 splits 7 more."""
    return 128 * 2.0 ** -23 + (2 * -(-k // 128) + 7) * 2.0 ** -24


def check(out, ref, tol, what=""):
    """One rounding of a value within `tol` of `ref`. An f16 output is infinite, with the value's
    sign, where that value may be 65520 or more (half a step above the largest f16 rounds up), and
    has to be where it cannot be less."""
    out = out.cpu()
    t = tol + HALF_STEP[out.dtype] * (ref.abs() + tol) + TINY[out.dtype]
    fine = (out.double() - ref).abs() <= t
    if out.dtype == torch.float16:
        fine = torch.where(ref.abs() + tol >= 65520, (out == torch.sign(ref) * torch.inf) | fine, fine)
        fine = torch.where(ref.abs() - tol >= 65520, out == torch.sign(ref) * torch.inf, fine)
    assert bool(fine.all()), f"{what} {out.dtype}: {int((~fine).sum())} of {fine.numel()} outside, first " \
                             f"{out[~fine][0].item()!r} for {ref[~fine][0].item()!r} +- {t[~fine][0].item():.3g} at " \
                             f"{(~fine).nonzero()[0].tolist()}"


def check_product(out, ref, magnitude, k, what=""):
    """The fp32 sums' error, then one rounding to the output type."""
    check(out, ref, sum_error(k) * magnitude, what)


def gated(g, gm, u, um, k):
    """(silu(g) * u, the bound on its error before the last rounding). The activation's slope is
    below 1.1; its exponential is off by at most 2 + 1.173 |g| units (2^-23) and its quotient by
    2, the sum and the two products by one rounding each."""
    s = g * torch.sigmoid(g)
    eg, eu = sum_error(k) * gm, sum_error(k) * um
    rel = (2 + 1.173 * g.abs() + 2 + 2) * 2.0 ** -23
    tol = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + rel * (s * u).abs() + 2.0 ** -126 * u.abs()
    return s * u, tol


def normal(r, c, seed, scale=1.0, outliers=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((r, c), generator=g) * scale
    if outliers:
        x = torch.where(torch.rand((r, c), generator=g) < 0.01, x * 50, x)
    return x


def cuda(pair):
    return tuple(t.cuda() for t in pair)
