"""The 4-bit cache, accumulated weights and eviction beyond 32-bit offsets, with wide tables,
and from two host threads at once."""
import threading

import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE = 16, 8, 128, 16


def _small(tensors, table, lens):
    """The requests' blocks alone: pools of a few blocks on the CPU, and their table."""
    used = [int(b) for row, n in zip(table.tolist(), lens.tolist()) for b in row[: -(-n // PAGE)]]
    at = torch.tensor(used, device="cuda")
    new, k = torch.full_like(table, -1), 0
    for b, n in enumerate(lens.tolist()):
        pages = -(-n // PAGE)
        new[b, :pages] = torch.arange(k, k + pages, dtype=torch.int32)
        k += pages
    small = []
    for t in tensors:
        raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        small.append(raw[at].cpu().view(t.dtype))
    return small, new


@pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])
def test_pool_beyond_four_gibibytes(four):
    """Blocks on both sides of 2^31 and 2^32 bytes (4 bits) or elements (16): appended to,
    decoded, voted on and evicted from."""
    a = attn()
    blocks = 270000 if four else 140000  # 16,384 bytes of codes, or 32,768 elements, a block
    g = torch.Generator().manual_seed(71)
    marks = [blocks - 1, blocks // 2 - 1, blocks // 2, 131072, 0], [131071, blocks - 2, 1, 262145 % blocks, -1]
    if four:
        cache = torch.zeros(blocks, 2, Hkv, PAGE, D // 2, dtype=torch.uint8, device="cuda")
        scales = torch.ones(blocks, 2, Hkv, PAGE, D // 16, device="cuda").to(torch.float8_e4m3fn)
    else:
        cache, scales = torch.zeros(blocks, 2, Hkv, PAGE, D, dtype=torch.bfloat16, device="cuda"), None
    weights = torch.zeros(blocks, Hkv, PAGE, device="cuda")
    lens = torch.tensor([70, 49], dtype=torch.int32)
    table = torch.tensor(marks, dtype=torch.int32)
    cu = torch.tensor([0, 70, 119], dtype=torch.int32)
    x = torch.randn(119, 2 * Hkv, D, generator=g).to(torch.bfloat16)
    args = (table.cuda(), cu.cuda(), lens.cuda())
    k, v = x[:, :Hkv].cuda(), x[:, Hkv:].cuda()
    if four:
        a.attn_append_paged_e2m1(k, v, cache, scales, *args)
    else:
        a.attn_append_paged(k, v, cache, *args)
    check_status(a)

    def held():
        small, small_table = _small([cache] + ([scales] if four else []), table, lens)
        return (kv4_ref.held(small[0], small[1], None) if four else small[0].double()), small_table

    pool, small = held()
    for b in range(2):
        n, t0 = int(lens[b]), int(cu[b])
        want = torch.stack((x[t0:t0 + n, :Hkv], x[t0:t0 + n, Hkv:])).transpose(1, 2)
        if four:
            codes, sc = kv4_ref.quantise(want, torch.ones(1, 1, 1))
            want = kv4_ref.values(codes) * sc.double().repeat_interleave(16, dim=-1)
        assert torch.equal(kv4_ref.rows_of(pool, small, b, n), want.double())
    q = torch.randn(2, Hq, D, generator=g).to(torch.bfloat16)
    one = torch.tensor([0, 1, 2], dtype=torch.int32)
    ref = kv4_ref.decode(q[:, :, None], pool, small, lens)
    lse = ref[1].float().t().contiguous()
    if four:
        o, l = a.attn_fwd_decode_paged_e2m1(q[:, :, None].cuda(), cache, scales, table.cuda(), lens.cuda(), weights=weights)
        kv4_ref.check_decode(o, l, ref, 70, "decode")
        a.attn_weights_paged_e2m1(q.cuda(), lse.cuda(), cache, scales, table.cuda(), one.cuda(), lens.cuda(), weights)
    else:
        for _ in range(2):
            a.attn_weights_paged(q.cuda(), lse.cuda(), cache, table.cuda(), one.cuda(), lens.cuda(), weights)
    check_status(a)
    (small_w,), _ = _small([weights], table, lens)
    kv4_ref.check_weights(small_w, torch.zeros_like(small_w), small, lens, [2 * s for s in ref[4]],
                          [2 * t + 1e-6 * s for t, s in zip(ref[5], ref[4])], 70, "weights")
    assert float(weights.double().sum()) == pytest.approx(float(small_w.double().sum()), rel=1e-9)
    pools = [cache] + ([scales] if four else [])
    before, _ = _small(pools, table, lens)
    want = kv4_ref.evict([p.view(torch.int16) if p.element_size() == 2 else p.view(torch.uint8) for p in before], small_w,
                         small, lens, 20, 5)
    new, kept = (a.attn_evict_paged_e2m1 if four else a.attn_evict_paged)(*pools, weights, table.cuda(), lens.cuda(), 20, 5)
    check_status(a)
    after, _ = _small(pools, table, lens)
    for p, w in zip(after, want[0]):
        assert torch.equal(p.view(torch.int16) if p.element_size() == 2 else p.view(torch.uint8), w)
    assert torch.equal(kept.cpu(), want[3]) and torch.equal(_small([weights], table, lens)[0][0], want[1])


@pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])
def test_tables_far_wider_than_the_requests(four):
    """Room for a million keys and requests of a few hundred: the same bits."""
    a = attn()
    g = torch.Generator().manual_seed(72)
    lens = torch.tensor([400, 90], dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens, PAGE, g)
    wide = torch.nn.functional.pad(table, (0, 65536 - table.shape[1]), value=-5)
    if four:
        pools = list(kv4_ref.random_pool(blocks, 2, PAGE, 64, g))
    else:
        pools = [torch.randn(blocks, 2, 2, PAGE, 64, generator=g).to(torch.bfloat16)]
    start = torch.rand(blocks, 2, PAGE, generator=g)
    q = torch.randn(490, 4, 64, generator=g).to(torch.bfloat16).cuda()
    lse = torch.full((4, 490), 6.0, device="cuda")
    cu = torch.tensor([0, 400, 490], dtype=torch.int32, device="cuda")
    got = []
    for t in (table, wide):
        p, w = [x.cuda() for x in pools], start.cuda()
        (a.attn_weights_paged_e2m1 if four else a.attn_weights_paged)(q, lse, *p, t.cuda(), cu, lens.cuda(), w)
        out = [w.clone()]
        if four:
            one = q[[399, 489]][:, :, None].contiguous()
            out += a.attn_fwd_decode_paged_e2m1(one, *p, t.cuda(), lens.cuda(), weights=w)
        new, kept = (a.attn_evict_paged_e2m1 if four else a.attn_evict_paged)(*p, w, t.cuda(), lens.cuda(), 100, 30)
        got.append(out + [new, kept, w] + p)
        check_status(a)
    for i, (x, y) in enumerate(zip(*got)):
        if four and 1 <= i <= 2 or four and i in (4, 5, 6, 7):
            continue  # the two decode kernels merge in another order, and what follows goes by their weights
        assert torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                           y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y), i


def test_two_host_threads():
    a = attn()
    g = torch.Generator().manual_seed(73)
    lens = torch.tensor([900, 300], dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens, PAGE, g)
    cache, scales = kv4_ref.random_pool(blocks, 2, PAGE, 128, g)
    q = torch.randn(2, 8, 1, 128, generator=g).to(torch.bfloat16).cuda()
    weights = torch.rand(blocks, 2, PAGE, generator=g).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()

    def job(out):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                c, s, w = cache.cuda(), scales.cuda(), weights.clone()
                o, lse = a.attn_fwd_decode_paged_e2m1(q, c, s, table.cuda(), lens.cuda(), weights=w)
                a.attn_weights_paged_e2m1(q[:, :, 0], lse.t(), c, s, table.cuda(), cu, lens.cuda(), w)
                new, kept = a.attn_evict_paged_e2m1(c, s, w, table.cuda(), lens.cuda(), 200, 40)
                out.append([t.cpu() for t in (o, lse, w, kept, c)])

    results = [[], []]
    threads = [threading.Thread(target=job, args=(r,)) for r in results]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(results[0]) == len(results[1]) == 20
    for r in results[0] + results[1]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[0][0]))
    check_status(a)
