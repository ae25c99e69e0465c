"""The 4-bit cache, weights and eviction with tables far wider than the requests: kept slots, rows
and weights bit for bit, results against the 64-bit form."""
import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status
from test_gpu_evict import _bits

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])
@pytest.mark.parametrize("lens,Hkv", [([400, 90], 2), ([(71 * i) % 300 for i in range(45)], 4)], ids=["clusters", "many"])
def test_evictions_of_wide_tables(lens, Hkv, four):
    """From weights that are the same in all: room for a million keys, for 24576, and as much as it
    takes.  Two requests have clusters in wide tables; forty-five of four heads a CTA a pair."""
    a = attn()
    g = torch.Generator().manual_seed(251)
    lens = torch.tensor(lens, dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens, PAGE, g)
    if four:
        pools = list(kv4_ref.random_pool(blocks, Hkv, PAGE, 64, g))
    else:
        pools = [torch.randn(blocks, 2, Hkv, PAGE, 64, generator=g).to(torch.bfloat16)]
    start = torch.rand(blocks, Hkv, PAGE, generator=g)
    want = kv4_ref.evict([_bits(p) for p in pools], start, table, lens, 100, 30)
    call = a.attn_evict_paged_e2m1 if four else a.attn_evict_paged
    for width in (table.shape[1], 1536, 65536):
        wide = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-5)
        p, w = [x.cuda() for x in pools], start.cuda()
        new, kept = call(*p, w, wide.cuda(), lens.cuda(), 100, 30)
        check_status(a)
        assert torch.equal(new.cpu(), want[2]) and torch.equal(kept.cpu(), want[3])
        assert torch.equal(w.cpu(), want[1])
        for x, y in zip(p, want[0]):
            assert torch.equal(_bits(x.cpu()), y)


@pytest.mark.parametrize("lens", [[400, 90], [(71 * i) % 300 for i in range(45)]], ids=["few", "many"])
def test_decodes_of_wide_tables(lens):
    """Both decode kernels' results and the keys' weights, and the weights of another pass."""
    a = attn()
    g = torch.Generator().manual_seed(252)
    lens = torch.tensor(lens, dtype=torch.int32)
    B = len(lens)
    table, blocks = kv_ref.random_table(lens, PAGE, g)
    cache, scales = kv4_ref.random_pool(blocks, 2, PAGE, 64, g)
    start = torch.rand(blocks, 2, PAGE, generator=g)
    q = torch.randn(B, 4, 1, 64, generator=g).to(torch.bfloat16)
    pool = kv4_ref.held(cache, scales, None)
    ref = kv4_ref.decode(q, pool, table, lens)
    cu = torch.tensor([0] + [int((lens[:b + 1] > 0).sum()) for b in range(B)], dtype=torch.int32)
    some = lens > 0
    lse = ref[1].float().t()[:, some].contiguous()
    share, tol = kv4_ref.column_sums(q[some][:, :, 0], lse, pool, table, cu, lens)
    passes = []
    for width in (table.shape[1], 1536, 65536):
        wide = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-5).cuda()
        w = start.cuda()
        o, l = a.attn_fwd_decode_paged_e2m1(q.cuda(), cache.cuda(), scales.cuda(), wide, lens.cuda(), weights=w)
        check_status(a)
        kv4_ref.check_decode(o, l, ref, int(lens.max()), f"{width} pages")
        kv4_ref.check_weights(w, start, table, lens, ref[4], ref[5], int(lens.max()), f"{width} pages")
        w = start.cuda()
        a.attn_weights_paged_e2m1(q[some][:, :, 0].cuda(), lse.cuda(), cache.cuda(), scales.cuda(), wide, cu.cuda(), lens.cuda(), w)
        kv4_ref.check_weights(w, start, table, lens, share, tol, 4, f"{width} pages")
        passes.append(w)
    assert all(torch.equal(w, passes[0]) for w in passes)
    check_status(a)
