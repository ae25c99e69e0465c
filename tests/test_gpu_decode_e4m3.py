"""Decode over the paged 8-bit cache against its 64-bit form."""
import math

import pytest
import torch

import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _problem(lens, Hq, Hkv, D, page, dtype="bf16", seed=0, scale_range=(-8, -4)):
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens, page, g)
    q = torch.randn(len(lens), Hq, 1, D, generator=g).to(DTYPES[dtype])
    cache = kv_ref.random_codes((blocks, 2, Hkv, page, D), g)
    scales = torch.exp2(torch.randint(*scale_range, (blocks, 2, Hkv), generator=g).float())
    return q, cache, scales, table, lens


def _run(a, pr, **kw):
    return a.attn_fwd_decode_paged_e4m3(*(t.cuda() for t in pr), **kw)


def _wide(pr):
    """The same requests with room in the table for 40000 keys: what the kernel for short
    contexts does not take."""
    q, cache, scales, table, lens = pr
    more = 40000 // cache.shape[3] - table.shape[1]
    return q, cache, scales, torch.nn.functional.pad(table, (0, max(0, more)), value=-7), lens


ways = pytest.mark.parametrize("way", [lambda pr: pr, _wide], ids=["own table", "wide table"])


def _check(a, pr, what="", scale=None):
    ref = kv_ref.decode_e4m3(*pr, scale=scale)
    empty = pr[4] == 0
    for p, name in ((_wide(pr), "wide table"), (pr, "own table")):
        o, lse = _run(a, p, scale=scale)
        check_status(a)
        kv_ref.check_decode(o, lse, ref, int(pr[4].max()), f"{what}, {name}")
        assert (o.cpu()[empty] == 0).all() and torch.isneginf(lse.cpu()[empty]).all()
    return o, lse


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,dtype", [
    ([1], 1, 1, 64, 16, "bf16"),
    ([1, 2, 15, 16, 17, 31, 32, 33], 4, 4, 128, 16, "bf16"),
    ([300, 0, 5], 8, 2, 128, 16, "bf16"),
    ([0, 0, 0], 8, 2, 128, 16, "bf16"),
    ([0, 129, 0, 64], 16, 16, 64, 8, "f16"),
    ([3, 40, 7], 4, 2, 64, 1, "bf16"),
    ([700, 33], 6, 2, 128, 5, "f16"),
    ([700, 256], 8, 1, 128, 256, "bf16"),
    ([1000, 33, 90], 7, 1, 128, 24, "bf16"),        # seven heads, pages that end inside a tile
    ([1000, 9], 9, 1, 64, 32, "bf16"),              # two halves of the product, the second nearly empty
    ([513, 2000], 16, 1, 128, 16, "f16"),
    ([100, 777], 20, 1, 64, 16, "bf16"),            # two head chunks
    ([300], 33, 1, 128, 16, "bf16"),                # three
    ([4096, 1, 2048, 15, 16], 32, 8, 128, 16, "bf16"),
    ([900, 100], 64, 8, 128, 64, "bf16"),
    ([5000], 12, 12, 64, 48, "f16"),
])
def test_matches_the_definition(lens, Hq, Hkv, D, page, dtype):
    a = attn()
    _check(a, _problem(lens, Hq, Hkv, D, page, dtype, seed=41), f"{lens} Hq{Hq} Hkv{Hkv} D{D} P{page}")


@pytest.mark.parametrize("B,Hkv,top", [(97, 4, 200), (1024, 1, 60), (1025, 1, 60), (1500, 2, 20)])
def test_many_short_requests(B, Hkv, top):
    """Many units in one warp's range; beyond 1024 requests the tiles are counted by a kernel
    of their own."""
    a = attn()
    lens = torch.randint(0, top, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    pr = _problem(lens, 2 * Hkv, Hkv, 64, 16, seed=42)
    _check(a, pr, f"{B} requests")
    assert a.last_launch_info()[2] == (1 if B * Hkv < 1100 else 3)
    pr[4][B // 2] = -1
    _run(a, pr)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    _run(a, _wide(pr))
    assert a.last_launch_info()[2] == (2 if B <= 1024 else 3)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT


def test_long_request_over_all_sms():
    a = attn()
    _check(a, _problem([70001], 8, 2, 128, 16, seed=43), "70001 keys")
    _check(a, _problem([40000, 3], 16, 1, 64, 64, seed=44), "40000 keys, 16 heads")


def test_workload_sizes():
    """64 requests of 4096 keys, Hq 32, Hkv 8, D 128."""
    a = attn()
    _check(a, _problem([4096] * 64, 32, 8, 128, 16, seed=45), "64 x 4096")


def test_scales_far_apart():
    """Scales over many powers of two, zero among them: the heavy keys keep their precision."""
    a = attn()
    pr = _problem([500, 90], 8, 2, 128, 16, seed=46)
    g = torch.Generator().manual_seed(47)
    pr[2][:, 0] = torch.exp2(torch.randint(-8, -5, pr[2][:, 0].shape, generator=g).float())
    pr[2][:, 1] = torch.exp2(torch.randint(-100, 40, pr[2][:, 1].shape, generator=g).float())
    _check(a, pr, "V scales from 2^-100 to 2^40")
    pr[2][:, 1] = 2.0 ** -20
    pr[2][::3, 1] = 0.0
    _check(a, pr, "V scales of zero")
    pr[2][:, 1] = 2.0 ** 100
    pr[2][::4, 0] = 0.0
    o, lse = _run(a, pr)  # bf16 holds them
    ref = kv_ref.decode_e4m3(*pr)
    kv_ref.check_decode(o, lse, ref, 500, "large V scales")


def test_scores_far_apart():
    """One key takes all the weight, early or late, and the reference moves often."""
    a = attn()
    pr = _problem([200, 333], 8, 2, 64, 16, seed=48)
    pr[2][:, 0] = torch.exp2(torch.arange(pr[2].shape[0]).float() % 12 - 6)[:, None]
    _check(a, pr, "steep scores", scale=1.0)
    _check(a, pr, "flat scores", scale=1e-6)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 300.0, 1e30])
def test_query_sizes(size):
    """bf16 queries beyond fp16's range, rows of zeros among them."""
    a = attn()
    pr = list(_problem([120, 17], 8, 2, 128, 16, seed=49))
    pr[0] = (pr[0].float() * size).to(torch.bfloat16)
    pr[0][0, 3] = 0
    _check(a, pr, f"queries of {size}", scale=1.0 / size / math.sqrt(128))


def test_general_scales():
    """Scales that are no powers of two."""
    a = attn()
    pr = _problem([333, 64], 4, 4, 64, 16, "f16", seed=50)
    pr[2].copy_(0.001 + 0.02 * torch.rand(pr[2].shape, generator=torch.Generator().manual_seed(51)))
    _check(a, pr, "scales")


@ways
def test_unused_rows_and_blocks_are_never_read(way):
    a = attn()
    pr = way(_problem([5, 33, 16], 8, 2, 128, 16, seed=52))
    want = _run(a, pr)
    q, cache, scales, table, lens = pr
    used = {(int(table[b, t // 16]), t % 16) for b in range(3) for t in range(int(lens[b]))}
    raw = cache.view(torch.uint8)
    for blk in range(cache.shape[0]):
        for r in range(16):
            if (blk, r) not in used:
                raw[blk, :, :, r] = 0x7F  # NaN
        if not any((blk, r) in used for r in range(16)):
            scales[blk] = math.nan
    got = _run(a, pr)
    check_status(a)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@ways
def test_nan_in_a_used_row_reaches_its_head_only(way):
    a = attn()
    pr = way(_problem([40, 40], 4, 2, 64, 16, seed=53))
    pr[1].view(torch.uint8)[int(pr[3][0, 1]), 1, 1, 3, 9] = 0x7F
    o, lse = _run(a, pr)
    bad = torch.isnan(o.cpu().float())[:, :, 0]
    assert bad[0, 2:, 9].all() and int(bad.sum()) == 2
    assert torch.isfinite(lse).all()


@ways
def test_bad_block_ids_and_lengths_are_reported(way):
    a = attn()
    for page in (16, 24):
        pr = way(_problem([40, 20], 8, 2, 128, page, seed=54))
        for bad in (pr[1].shape[0], -2, 2 ** 31 - 1):
            t = pr[3].clone()
            t[1, 0] = bad
            _run(a, (pr[0], pr[1], pr[2], t, pr[4]))
            assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        for length in (-1, pr[3].shape[1] * page + 1):
            n = pr[4].clone()
            n[0] = length
            _run(a, (pr[0], pr[1], pr[2], pr[3].clamp(min=0), n))
            assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        _check(a, pr, "afterwards")


@ways
def test_outputs_of_the_caller_and_repeatability(way):
    a = attn()
    pr = [t.cuda() for t in way(_problem([900, 77, 0, 1300], 12, 4, 128, 16, seed=55))]
    out = torch.full((6, 12, 1, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 12), 3.0, device="cuda")
    o, l = a.attn_fwd_decode_paged_e4m3(*pr, out=out[1:5], lse=lse[1:5])
    assert (out[0] == 3).all() and (out[5] == 3).all() and (lse[0] == 3).all() and (lse[5] == 3).all()
    for _ in range(5):
        o2, l2 = a.attn_fwd_decode_paged_e4m3(*pr)
        assert torch.equal(o2, o) and torch.equal(l2, l)
    o3, none = a.attn_fwd_decode_paged_e4m3(*pr, want_lse=False)
    assert none is None and torch.equal(o3, o)


@ways
def test_two_streams_at_once_and_two_graphs(way):
    a = attn()
    first = [t.cuda() for t in way(_problem([2000, 500], 8, 2, 128, 16, seed=56))]
    second = [t.cuda() for t in way(_problem([1500, 900], 8, 2, 128, 16, seed=57))]
    want = [a.attn_fwd_decode_paged_e4m3(*p) for p in (first, second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs = [], []
    for s, p in zip(streams, (first, second)):
        g = torch.cuda.CUDAGraph()
        o, l = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
        with torch.cuda.graph(g, stream=s):
            a.attn_fwd_decode_paged_e4m3(*p, out=o, lse=l)
        graphs.append(g)
        outs.append((o, l))
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    eager = []
    for s, p in zip(streams, (first, second)):
        with torch.cuda.stream(s):
            eager.append(a.attn_fwd_decode_paged_e4m3(*p))
    torch.cuda.synchronize()
    for got in (outs, eager):
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    check_status(a)
