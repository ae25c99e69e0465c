"""Accumulated attention weights over contexts whose length times the group passes 32 bits."""
import math

import pytest
import torch

import kv4_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,n,length", [(100, 3, 22_000_003), (48, 1, 45_000_001)])
def test_many_heads_over_millions_of_keys(Hq, n, length):
    """Tiles that are not whole columns of 32, and keys far before what their tokens see up to:
    sampled keys against the 64-bit form, and no key without a weight."""
    a = attn()
    D, page = 64, 256
    g = torch.Generator(device="cuda").manual_seed(211)
    pages = -(-length // page)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    cache = torch.randint(0, 256, (pages, 2, 1, page, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((pages, 2, 1, page, D // 16), 0.25, device="cuda").to(torch.float8_e4m3fn)
    q = torch.randn(n, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    lse = 17.0 + torch.rand(Hq, n, generator=g, device="cuda")
    weights = torch.zeros(pages, 1, page, device="cuda")
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [length]))
    a.attn_weights_paged_e2m1(q, lse, cache, scales, table, cu, lens, weights)
    check_status(a)
    w = weights[table[0].long()].flatten()
    assert bool((w[:length] > 0).all()) and bool((w[length:] == 0).all())
    keys = torch.cat((torch.arange(600), torch.arange(length - 600, length),
                      torch.randint(0, length, (4000,), generator=torch.Generator().manual_seed(212))))
    at = table[0].cpu().long()[keys // page], keys % page
    k = kv4_ref.values(kv4_ref.unpack(cache[:, 0, 0][at[0].cuda(), at[1].cuda()].cpu())) * 0.25
    qd, z = q.cpu().double(), lse.cpu().double().t()
    x = torch.einsum("nhd,kd->nhk", qd, k) / math.sqrt(D)
    size = torch.einsum("nhd,kd->nhk", qd.abs(), k.abs()) / math.sqrt(D)
    seen = keys <= length - n + torch.arange(n)[:, None]
    p = torch.exp(x - z[..., None]) * seen[:, None]
    rel = size * kv4_ref.score_error(D) + (x.abs() + z[..., None].abs() + 1.0) * 2.0 ** -21
    want = p.sum(dim=(0, 1))
    tol = (p * rel).sum(dim=(0, 1)) + want * (n * Hq / 4 + 64) * 2.0 ** -24
    off = (w[keys.cuda()].cpu().double() - want).abs() / tol
    assert float(off.max()) <= 1, float(off.max())
