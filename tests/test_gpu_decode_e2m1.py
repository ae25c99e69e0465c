"""Decode over the paged 4-bit cache against its 64-bit form, and the weights it adds up."""
import math

import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _problem(lens, Hq, Hkv, D, page, dtype="bf16", seed=0, factors=True, **kw):
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens, page, g)
    q = torch.randn(len(lens), Hq, 1, D, generator=g).to(DTYPES[dtype])
    cache, scales = kv4_ref.random_pool(blocks, Hkv, page, D, g, **kw)
    f = 0.5 + torch.rand(2, Hkv, generator=g) if factors else None
    weights = torch.rand(blocks, Hkv, page, generator=g)
    return [q, cache, scales, table, lens, f, weights]


def _wide(pr):
    """The same requests with room in the table for 40000 keys: what the kernel for short
    contexts does not take."""
    more = 40000 // pr[1].shape[3] - pr[3].shape[1]
    return pr[:3] + [torch.nn.functional.pad(pr[3], (0, max(0, more)), value=-7)] + pr[4:]


ways = pytest.mark.parametrize("way", [lambda pr: pr, _wide], ids=["own table", "wide table"])


def _run(a, pr, add=True, **kw):
    q, cache, scales, table, lens, f, weights = pr
    w = weights.cuda() if add else None
    o, lse = a.attn_fwd_decode_paged_e2m1(q.cuda(), cache.cuda(), scales.cuda(), table.cuda(), lens.cuda(),
                                          factors=None if f is None else f.cuda(), weights=w, **kw)
    return o, lse, w


def _check(a, pr, what="", scale=None):
    q, cache, scales, table, lens, f, weights = pr
    ref = kv4_ref.decode(q, kv4_ref.held(cache, scales, f), table, lens, scale)
    empty = lens == 0
    keys = int(lens.max())
    for p, name in ((_wide(pr), "wide table"), (pr, "own table")):
        o, lse, w = _run(a, p, scale=scale)
        check_status(a)
        kv4_ref.check_decode(o, lse, ref, keys, f"{what}, {name}")
        assert (o.cpu()[empty] == 0).all() and torch.isneginf(lse.cpu()[empty]).all()
        kv4_ref.check_weights(w, weights, table, lens, ref[4], ref[5], keys, f"{what}, {name}")
        plain = _run(a, p, add=False, scale=scale)
        assert torch.equal(plain[0], o) and torch.equal(plain[1], lse)
        o2, none, w2 = _run(a, p, scale=scale, want_lse=False)
        assert none is None and torch.equal(o2, o) and torch.equal(w2, w)
    return o, lse


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,dtype", [
    ([1], 1, 1, 64, 16, "bf16"),
    ([1, 2, 15, 16, 17, 31, 32, 33], 4, 4, 128, 16, "bf16"),
    ([1, 2, 15, 16, 17, 31, 32, 33], 4, 4, 64, 16, "f16"),
    ([300, 0, 5], 8, 2, 128, 16, "bf16"),
    ([0, 0, 0], 8, 2, 128, 16, "bf16"),
    ([0, 129, 0, 64], 16, 16, 64, 8, "f16"),
    ([3, 40, 7], 4, 2, 64, 1, "bf16"),
    ([700, 33], 6, 2, 128, 5, "f16"),
    ([700, 33], 3, 1, 64, 5, "f16"),
    ([700, 256], 8, 1, 128, 256, "bf16"),
    ([1000, 33, 90], 7, 1, 128, 24, "bf16"),
    ([1000, 9], 9, 1, 64, 32, "bf16"),
    ([513, 2000], 16, 1, 128, 16, "f16"),
    ([100, 777], 20, 1, 64, 16, "bf16"),
    ([300], 33, 1, 128, 16, "bf16"),
    ([4096, 1, 2048, 15, 16], 32, 8, 128, 16, "bf16"),
    ([900, 100], 64, 8, 128, 64, "bf16"),
    ([5000], 12, 12, 64, 48, "f16"),
])
def test_matches_the_definition(lens, Hq, Hkv, D, page, dtype):
    a = attn()
    _check(a, _problem(lens, Hq, Hkv, D, page, dtype, seed=141), f"{lens} Hq{Hq} Hkv{Hkv} D{D} P{page}")


def test_without_factors():
    a = attn()
    _check(a, _problem([333, 64], 4, 4, 64, 16, "f16", seed=142, factors=False), "no factors")


@pytest.mark.parametrize("D", [64, 128])
def test_every_code_at_every_place(D):
    """One key: the result is its row of V, bit for bit (6 bits in bf16 times a power of two)."""
    a = attn()
    pr = _problem([1] * 64, 2, 1, D, 16, seed=143)
    pr[5] = torch.tensor([[1.0], [0.25]])
    o, _, _ = _run(a, pr)
    check_status(a)
    want = kv4_ref.held(pr[1], pr[2], pr[5])
    for b in range(64):
        assert torch.equal(o.cpu()[b, :, 0].double(), want[int(pr[3][b, 0]), 1, 0, :1].expand(2, D))


@pytest.mark.parametrize("B,Hkv,top", [(97, 4, 200), (1024, 1, 60), (1025, 1, 60), (1500, 2, 20)])
def test_many_short_requests(B, Hkv, top):
    a = attn()
    lens = torch.randint(0, top, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    pr = _problem(lens, 2 * Hkv, Hkv, 64, 16, seed=144)
    _check(a, pr, f"{B} requests")
    pr[4][B // 2] = -1
    for p in (pr, _wide(pr)):
        _run(a, p)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT


def test_long_request_over_all_sms():
    a = attn()
    _check(a, _problem([70001], 8, 2, 128, 16, seed=145), "70001 keys")
    _check(a, _problem([40000, 3], 16, 1, 64, 64, seed=146), "40000 keys, 16 heads")


def test_workload_sizes():
    """64 requests of 4096 keys, Hq 32, Hkv 8, D 128."""
    a = attn()
    _check(a, _problem([4096] * 64, 32, 8, 128, 16, seed=147), "64 x 4096")


def test_scales_far_apart():
    """V's scales over all of e4m3, negative and zero ones among them; light keys with large rows."""
    a = attn()
    pr = _problem([500, 90], 8, 2, 128, 16, seed=148)
    g = torch.Generator().manual_seed(149)
    codes = torch.randint(0, 127, pr[2][:, 1].shape, generator=g, dtype=torch.uint8)
    pr[2].view(torch.uint8)[:, 1] = codes
    _check(a, pr, "V scales from 0 to 448")
    pr[2].view(torch.uint8)[:, 1] = codes | 0x80
    pr[2].view(torch.uint8)[::2, 0] |= 0x80
    _check(a, pr, "negative scales")


def test_scores_far_apart():
    """One key takes all the weight, early or late, and the reference moves often."""
    a = attn()
    pr = _problem([200, 333], 8, 2, 64, 16, seed=150)
    n = pr[2].shape[0]
    pr[2].view(torch.uint8)[:, 0] = (torch.exp2(torch.arange(n).float() % 12 - 6)[:, None, None, None] * torch.ones(n, 2, 16, 4)).to(torch.float8_e4m3fn).view(torch.uint8)
    _check(a, pr, "steep scores", scale=1.0)
    _check(a, pr, "flat scores", scale=1e-6)


def test_light_keys_behind_a_heavy_one_without_value():
    """A key whose score is far over the others' has a row of zeros: the result is what the light
    ones add up to, down to 2^-60 of it."""
    a = attn()
    for gap in (10.0, 25.0, 40.0):
        pr = _problem([260], 4, 1, 64, 16, seed=151, factors=False)
        q, cache, scales, table, lens, f, w = pr
        q[:] = 0.0
        q[..., 0] = 1.0
        raw = kv4_ref.unpack(cache)
        raw[..., 0] = 0
        raw[int(table[0, 3]), 0, 0, 5, 0] = 7  # 6 at element 0 of slot 53
        raw[int(table[0, 3]), 1, 0, 5] = 0
        cache.copy_(kv4_ref.pack(raw))
        scales.view(torch.uint8)[int(table[0, 3]), 0, 0, 5] = 0x38  # 1
        _check(a, pr, f"gap {gap}", scale=gap / 6)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 300.0, 1e30])
def test_query_sizes(size):
    a = attn()
    pr = _problem([120, 17], 8, 2, 128, 16, seed=152)
    pr[0] = (pr[0].float() * size).to(torch.bfloat16)
    pr[0][0, 3] = 0
    _check(a, pr, f"queries of {size}", scale=1.0 / size / math.sqrt(128))


def test_factors_far_apart():
    a = attn()
    pr = _problem([90, 300], 4, 2, 128, 24, seed=153)
    pr[5] = torch.tensor([[2.0 ** -90, 3e5], [1e-20, 7e20]])
    pr[0][:, :2] = (pr[0][:, :2].float() * 2.0 ** 90).to(torch.bfloat16)
    pr[0][:, 2:] = (pr[0][:, 2:].float() / 3e5).to(torch.bfloat16)
    _check(a, pr, "factors")


@ways
def test_unused_rows_and_blocks_are_never_read(way):
    a = attn()
    for page in (16, 24):
        pr = way(_problem([5, 33, 16], 8, 2, 128, page, seed=154))
        want = _run(a, pr)
        q, cache, scales, table, lens = pr[:5]
        used = {(int(table[b, t // page]), t % page) for b in range(3) for t in range(int(lens[b]))}
        raw = scales.view(torch.uint8)
        for blk in range(cache.shape[0]):
            for r in range(page):
                if (blk, r) not in used:
                    raw[blk, :, :, r] = 0x7F  # NaN
        got = _run(a, pr)
        check_status(a)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


@ways
def test_requests_that_share_blocks_add_up(way):
    a = attn()
    pr = _problem([300, 290, 700, 4], 8, 2, 128, 16, seed=156)
    for b in (1, 2):
        pr[3][b, :15] = pr[3][0, :15]
    q, cache, scales, table, lens, f, weights = pr
    o, lse, w = _run(a, way(pr))
    check_status(a)
    ref = kv4_ref.decode(q, kv4_ref.held(cache, scales, f), table, lens)
    kv4_ref.check_decode(o, lse, ref, 700)
    kv4_ref.check_weights(w, weights, table, lens, ref[4], ref[5], 700)


@ways
def test_nan_in_a_used_row_reaches_its_head_only(way):
    a = attn()
    pr = way(_problem([40, 40], 4, 2, 64, 16, seed=155))
    pr[2].view(torch.uint8)[int(pr[3][0, 1]), 1, 1, 3, 2] = 0x7F
    o, lse, w = _run(a, pr)
    bad = torch.isnan(o.cpu().float())[:, :, 0]
    assert bad[0, 2:, 32:48].all() and int(bad.sum()) == 32
    assert torch.isfinite(lse).all() and torch.isfinite(w).all()


@ways
def test_bad_block_ids_and_lengths_are_reported(way):
    a = attn()
    for page in (16, 24):
        pr = way(_problem([40, 20], 8, 2, 128, page, seed=156))
        for bad in (pr[1].shape[0], -2, 2 ** 31 - 1):
            t = pr[3].clone()
            t[1, 0] = bad
            o, lse, w = _run(a, pr[:3] + [t] + pr[4:])
            assert a.device_status() == a.ATTN_ERR_BAD_INPUT
            held = torch.zeros(pr[1].shape[0], dtype=torch.bool)
            held[pr[3][pr[3] >= 0].long()] = True
            assert torch.equal(w.cpu()[~held], pr[6][~held])
        for length in (-1, pr[3].shape[1] * page + 1):
            n = pr[4].clone()
            n[0] = length
            _run(a, pr[:3] + [pr[3].clamp(min=0), n] + pr[5:])
            assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        _check(a, pr, "afterwards")


@ways
def test_outputs_of_the_caller_and_repeatability(way):
    a = attn()
    pr = way(_problem([900, 77, 0, 1300], 12, 4, 128, 16, seed=157))
    out = torch.full((6, 12, 1, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 12), 3.0, device="cuda")
    o, l, w = _run(a, pr, out=out[1:5], lse=lse[1:5])
    assert (out[0] == 3).all() and (out[5] == 3).all() and (lse[0] == 3).all() and (lse[5] == 3).all()
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(_run(a, pr), (o, l, w)))


@ways
def test_two_streams_at_once_and_two_graphs(way):
    a = attn()
    problems = [way(_problem(n, 8, 2, 128, 16, seed=s)) for n, s in (([2000, 500], 158), ([1500, 900], 159))]
    want = [_run(a, p) for p in problems]
    dev = [[None if t is None else t.cuda() for t in p] for p in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs = [], []
    for s, p in zip(streams, dev):
        g = torch.cuda.CUDAGraph()
        o, l, w = torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), p[6].clone()
        with torch.cuda.graph(g, stream=s):
            w.copy_(p[6])
            a.attn_fwd_decode_paged_e2m1(*p[:5], factors=p[5], weights=w, out=o, lse=l)
        graphs.append(g)
        outs.append((o, l, w))
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    eager = []
    for s, p in zip(streams, dev):
        with torch.cuda.stream(s):
            w = p[6].clone()
            eager.append((*a.attn_fwd_decode_paged_e2m1(*p[:5], factors=p[5], weights=w), w))
    torch.cuda.synchronize()
    for got in (outs, eager):
        for x, y in zip(got, want):
            assert all(torch.equal(i, j) for i, j in zip(x, y))
    check_status(a)
