"""Decode over the 4-bit cache, with the keys' weights, at the most keys that a table may have."""
import math

import pytest
import torch

from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu


def test_weights_of_two_thousand_million_keys():
    """32767 pages of 65536 keys, all of them one of 64 blocks: every key has the same score, so a
    place gets its block's count over the number of keys (their sum in fp32 within 2^-15, the
    exponentials' arguments within 2^-16)."""
    a = attn()
    D, page, pages, blocks = 64, 65536, 32767, 64
    g = torch.Generator().manual_seed(231)
    table = torch.randint(0, blocks, (1, pages), generator=g).to(torch.int32)
    cache = torch.zeros(blocks, 2, 1, page, D // 2, dtype=torch.uint8, device="cuda")
    cache[:, 1] = 0x22  # V: ones
    scales = torch.ones(blocks, 2, 1, page, D // 16, device="cuda").to(torch.float8_e4m3fn)
    weights = torch.zeros(blocks, 1, page, device="cuda")
    q = torch.randn(1, 1, 1, D, generator=g).to(torch.bfloat16).cuda()
    length = pages * page - 3
    o, lse = a.attn_fwd_decode_paged_e2m1(q, cache, scales, table.cuda(),
                                          torch.tensor([length], dtype=torch.int32, device="cuda"), weights=weights)
    check_status(a)
    assert bool((o == 1).all())
    assert abs(float(lse) - math.log(length)) <= 1e-5
    count = torch.bincount(table[0].long(), minlength=blocks).double()[:, None].expand(blocks, page).clone()
    count[int(table[0, -1]), -3:] -= 1
    off = (weights[:, 0].cpu().double() * length - count).abs() / count
    assert float(off.max()) <= 2.0 ** -14, float(off.max())
