"""What the decode over the 8-bit cache makes of a key's weight: results that are small
differences of large sums, and results that come from light keys alone, because the heavy
ones' values are zero.  Nothing here is relative to the largest weight: the bound is
relative to sum p vs |v|, the weighted values that are there."""
import math

import pytest
import torch

import kv_ref
from gpu_util import attn, check_status
from test_gpu_decode_e4m3 import _run, _wide

pytestmark = pytest.mark.gpu


def _check(a, pr, scale, weight, keys, what):
    """weight: the relative error of a key's weight as the products see it."""
    want, wl, spread, dx, _ = kv_ref.decode_e4m3(*pr, scale=scale)
    h = kv_ref.HALF_STEP[pr[0].dtype]
    # As in kv_ref.check_decode: scores, exponentials (2^-20, and 2^-24 of exponents up to
    # 128), and sums of `keys` positive terms.
    rel = weight + 2.0 ** -20 + 2.0 ** -17 + 2 * dx[..., None] + 2 * (keys / 4 + 64) * 2.0 ** -24
    tol = h * want.abs() + (1 + h) * rel * spread + kv_ref.TINY[pr[0].dtype]
    for p, name in ((pr, "own table"), (_wide(pr), "wide table")):
        o, lse = _run(a, p, scale=scale)
        check_status(a)
        got = o.cpu().double()[:, :, 0]
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), (f"{what}, {name}: {int(bad.sum())} off, worst "
                               f"{float(((got - want).abs() / tol).max()):.2f} of the bound")
        assert ((lse.cpu().double() - wl).abs() <= dx + 2.0 ** -17 + wl.abs() * 2.0 ** -22).all(), what


def _empty(n, Hq, Hkv, D, page, dtype):
    """One request of n keys, scales of 1, scores of 0 and values of 0."""
    table, blocks = kv_ref.random_table(torch.tensor([n]), page, torch.Generator().manual_seed(n))
    q = torch.zeros(1, Hq, 1, D, dtype=dtype)
    cache = torch.zeros(blocks, 2, Hkv, page, D)
    return q, cache, torch.ones(blocks, 2, Hkv), table, torch.tensor([n], dtype=torch.int32)


def _rows(pr, which, values):
    """Writes K (0) or V (1) rows [n, D] of every KV head."""
    _, cache, _, table, _ = pr
    page, j = cache.shape[3], torch.arange(len(values))
    cache[table[0, j // page].long(), which, :, j % page] = values[:, None].expand(-1, cache.shape[2], -1)


def _codes(pr):
    q, cache, scales, table, lens = pr
    codes = cache.to(torch.float8_e4m3fn)
    assert torch.equal(codes.float(), cache)  # the tests' values are codes
    return q, codes, scales, table, lens


@pytest.mark.parametrize("Hq,D,page,dtype", [(4, 128, 16, "f16"), (16, 128, 16, "bf16"), (3, 64, 24, "f16"),
                                             (20, 64, 32, "bf16"), (12, 128, 5, "f16")])
def test_small_differences_of_large_sums(Hq, D, page, dtype):
    """As many keys of weight 1 and value 3 as of weight p and value -4, p next to 3/4: the
    result, about 4 (3/4 - p) / (1 + p), is of the size of an 11-bit weight's rounding."""
    a = attn()
    n = 96
    for t in (0.5, -0.4, 1.5, 0.9):  # p = 3/4 + t * 2^-12: between two fp16 values
        pr = _empty(n, Hq, 1, D, page, {"bf16": torch.bfloat16, "f16": torch.float16}[dtype])
        odd = torch.randperm(n, generator=torch.Generator().manual_seed(3)) % 2
        k = torch.zeros(n, D)
        k[:, 7] = odd.float()
        _rows(pr, 0, k)
        _rows(pr, 1, (3.0 - 7.0 * odd.float())[:, None].expand(n, D))
        pr[0][:, :, 0, 7] = -1.0
        scale = float(torch.tensor(-math.log(0.75 + t * 2.0 ** -12), dtype=torch.float32))
        # Two fp16 terms, half a step of the second: 2^-12 * 2^-12.
        _check(a, _codes(pr), scale, 2.0 ** -24, n, f"p = 3/4 + {t} * 2^-12")


@pytest.mark.parametrize("n,place,Hq", [(8000, 0, 4), (8000, 4321, 16), (70000, 69999, 4), (70000, 33333, 1)])
def test_many_light_keys_behind_one_with_no_value(n, place, Hq):
    """One key takes nearly all the weight and has values of zero; what is left is `gap` nats
    lighter a key, under every 16-bit number next to 1 from 17.4 on, but for its own sum."""
    a = attn()
    for gap, dtype in ((17.0, torch.float16), (17.4, torch.float16), (18.0, torch.bfloat16), (24.0, torch.bfloat16),
                       (40.0, torch.bfloat16)):
        pr = _empty(n, Hq, 1, 128, 16, dtype)
        k, v = torch.zeros(n, 128), torch.ones(n, 128)
        k[place, 3] = 16.0
        v[:, 1::2] = torch.tensor([0.5, 2.0]).repeat(n // 2)[:, None]
        v[place] = 0.0
        _rows(pr, 0, k)
        _rows(pr, 1, v)
        pr[0][:, :, 0, 3] = 1.0
        _check(a, _codes(pr), gap / 16.0, 2.0 ** -14, n, f"{gap} nats")


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (16, 1, 64, 16), (5, 5, 64, 24), (32, 2, 128, 7)])
def test_weights_far_apart_in_one_tile(Hq, Hkv, D, page):
    """Scores up to 60 nats apart, in any order, and scales 2^-12 to 1 of V: the values of all
    keys above a level are zero, another level for every column."""
    a = attn()
    n = 500
    g = torch.Generator().manual_seed(61)
    pr = _empty(n, Hq, Hkv, D, page, torch.bfloat16)
    level = torch.randint(0, 61, (n,), generator=g)
    k = torch.zeros(n, D)
    k[:, 0], k[:, 1] = level // 8 * 8, level % 8  # scores as sums of codes
    v = torch.randint(1, 9, (n, D), generator=g).float()
    for d in range(D):
        v[level > 60 * d / D, d] = 0.0
    _rows(pr, 0, k)
    _rows(pr, 1, v)
    pr[0][:, :, 0, :2] = 1.0
    pr[0][:, ::3, 0, :2] = 0.5
    pr[2][:, 1] = torch.exp2(-torch.randint(0, 13, pr[2][:, 1].shape, generator=g).float())
    _check(a, _codes(pr), 1.0, 2.0 ** -14, n, "levels")


@pytest.mark.parametrize("exponent", [-118, -100, 100, 118])
def test_values_at_the_ends_of_the_scales(exponent):
    """V scales at which the factor from the weighted sum to the result is hardly a normal float."""
    a = attn()
    for Hq, D, n in ((8, 128, 500), (16, 64, 77), (3, 128, 3000)):
        pr = _empty(n, Hq, 1, D, 16, torch.bfloat16)
        g = torch.Generator().manual_seed(81)
        q, codes, scales, table, lens = _codes(pr)
        q.copy_(torch.randn(q.shape, generator=g))
        codes = kv_ref.random_codes(codes.shape, g)
        scales[:, 0], scales[:, 1] = 2.0 ** -7, 2.0 ** exponent
        _check(a, (q, codes, scales, table, lens), 1.0 / math.sqrt(D), 2.0 ** -14, n, f"2^{exponent}")
