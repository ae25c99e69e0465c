"""Plain 64-bit forms of the rotary, norm, paged-append and 8-bit-cache decode
operators, on the CPU, and the error bounds their tests use.

Half a rounding step relative to the value: bf16 2^-8, fp16 2^-11, fp32 2^-24,
e4m3 2^-4."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# Half the spacing of the subnormals, for results next to zero.
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def frequencies(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def turns_to_radians(turns):
    """The table's entries (int64, units of 2^-64 turn) as radians."""
    return torch.tensor([(int(t) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns], dtype=torch.float64)


def rotate(x, pos, freq, interleaved=False, magnitude=1.0):
    """x float64 [..., D]; pos broadcasts over x's leading dimensions.  Returns
    (y, a): the rotated rows, and for every element magnitude * (|a| + |b|) of
    its pair (|x| outside the rotated part), the scale of fp32 errors."""
    h = len(freq)
    i = torch.arange(h)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    angle = pos.double()[..., None] * freq
    y, size = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    y[..., first] = magnitude * (a * angle.cos() - b * angle.sin())
    y[..., second] = magnitude * (b * angle.cos() + a * angle.sin())
    size[..., first] = size[..., second] = magnitude * (a.abs() + b.abs())
    return y, size


def norm(x, w, eps):
    r = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    return r if w is None else r * w.double()


# A rotated element in fp32: the angle's float (2^-25 half turns = 1.6 * 2^-24
# radians), sine and cosine (2 ulp, 2^-23, and their product with the magnitude),
# two products and a sum: under 2^-21 of magnitude * (|a| + |b|).
ROTATION_ERROR = 2.0 ** -21


def norm_error(D):
    """Relative error of x * rsqrt(mean) * w in fp32: D/8 + 4 sequential additions of
    squares (halved by the root) and a handful of roundings."""
    return (D / 8 + 16) * 2.0 ** -24


def check_rows(got, want, size, error, what=""):
    """got: 16- or 32-bit rows; want, size: float64; error: fp32 error relative to size."""
    h = HALF_STEP[got.dtype]
    tol = h * want.abs() + (1 + h) * error * size + TINY[got.dtype]
    g = got.detach().cpu().double()
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float(((g - want).abs() / tol).max()):.2f} of the bound"


def slots(cu, lens):
    """(token, request, slot) of every token of every request."""
    for b in range(len(lens)):
        for j in range(cu[b], cu[b + 1]):
            yield j, b, int(lens[b]) - (cu[b + 1] - j)


E4M3_MAX = 448.0


def pow2_scale(amax: float, limit: float) -> float:
    """The smallest power of two s >= 2^-100 with amax <= limit * s (exact: the
    arguments are floats, the products exact in double)."""
    s = 2.0 ** -100
    while amax > limit * s:
        s *= 2.0
    return s


def k_limit(magnitude: float, rot: int, D: int) -> float:
    """448 / b of rotated keys: b = sqrt(2) * magnitude, at least 1 if part of the head passes."""
    if rot == 0:
        return E4M3_MAX
    b = math.sqrt(2.0) * float(torch.tensor(magnitude, dtype=torch.float32))
    return float(torch.tensor(E4M3_MAX / (max(b, 1.0) if rot < D else b), dtype=torch.float32))


def gather(cache, table, b, n):
    """K and V of request b's first n slots: [2, Hkv, n, D] in the cache's type."""
    page = cache.shape[3]
    ids = table[b, : -(-n // page)].long()
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[ids].permute(1, 2, 0, 3, 4).reshape(2, cache.shape[2], len(ids) * page, -1)[:, :, :n]
    return x.contiguous().view(cache.dtype)


def gather_scales(scales, table, b, n, page):
    """[2, Hkv, n] of request b's first n slots."""
    ids = table[b, : -(-n // page)].long()
    return scales[ids].permute(1, 2, 0).repeat_interleave(page, dim=2)[:, :, :n].double()


def decode_e4m3(q, cache, scales, table, lens, scale=None):
    """(o, lse, spread, dx) in float64: spread = sum p vs |v| / sum p for every output
    element; dx = the bound of a score's fp32 error for every head."""
    B, Hq, _, D = q.shape
    Hkv, page = cache.shape[2], cache.shape[3]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    spread = torch.zeros(B, Hq, D, dtype=torch.float64)
    dx = torch.zeros(B, Hq, dtype=torch.float64)
    most = torch.zeros(B, Hq, 1, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        kv = gather(cache, table, b, n).double() * gather_scales(scales, table, b, n, page)[..., None]
        kv = kv.repeat_interleave(Hq // Hkv, dim=1)
        x = torch.einsum("hd,hnd->hn", q[b, :, 0].double(), kv[0]) * scale
        size = torch.einsum("hd,hnd->hn", q[b, :, 0].double().abs(), kv[0].abs()) * abs(scale)
        lse[b] = torch.logsumexp(x, dim=-1)
        p = torch.exp(x - lse[b][:, None])
        o[b] = torch.einsum("hn,hnd->hd", p, kv[1])
        spread[b] = torch.einsum("hn,hnd->hd", p, kv[1].abs())
        # D/16 products of 16 terms added to an fp32 sum, each step within 2^-22 of the
        # terms' sizes (the tensor core may truncate), and three fp32 products.
        dx[b] = size.amax(dim=-1) * (D / 16 + 6) * 2.0 ** -22
        most[b] = (p * gather_scales(scales, table, b, n, page)[1].repeat_interleave(Hq // Hkv, dim=0)).amax(
            dim=-1, keepdim=True)
        most[b] *= n * 448.0
    return o, lse, spread, dx, most


def check_decode(o, lse, ref, keys, what=""):
    """Weights are fp16 (2^-11 each, 2^-25 of the largest weight below fp16's normal
    range), exponentials 2^-21 and the scores' dx; sums of `keys` positive terms over
    four lanes and the warps' pieces."""
    want, wl, spread, dx, most = ref
    h = HALF_STEP[o.dtype]
    sums = (keys / 4 + 64) * 2.0 ** -24
    rel = 2.0 ** -11 + 2.0 ** -20 + 2 * dx[..., None] + 2 * sums
    tol = h * want.abs() + (1 + h) * (rel * spread + 2.0 ** -25 * most) + TINY[o.dtype]
    got = o.detach().cpu().double()[:, :, 0]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: o: {int(bad.sum())} off, worst {float(((got - want).abs() / tol).max()):.2f} of the bound"
    if lse is not None:
        l = lse.detach().cpu().double()
        empty = torch.isinf(wl)
        assert torch.equal(torch.isneginf(l), empty), what
        ltol = dx + sums + 2.0 ** -20 + wl.abs() * 2.0 ** -22
        bad = ~((l - wl).abs() <= ltol) & ~empty
        assert not bad.any(), f"{what}: lse off by {float((l - wl).abs()[~empty].max()):.2e}"


def random_codes(shape, gen):
    return (torch.randn(shape, generator=gen) * 96.0).clamp(-448, 448).to(torch.float8_e4m3fn)


def random_table(lens, page, gen, spare=3):
    """Distinct blocks in a random order, -1 past each request's last page."""
    per = [-(-int(n) // page) for n in lens]
    pool = torch.randperm(sum(per) + spare, generator=gen).tolist()
    table = torch.full((len(per), max(1, max(per))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(pool[at:at + n], dtype=torch.int32)
        at += n
    return table, len(pool)
