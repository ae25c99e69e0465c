"""The rotary, append and 8-bit-cache calls beyond 32-bit offsets, with far more
requests than tokens, and from two host threads at once."""
import threading

import pytest
import torch

import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE = 16, 8, 128, 16


def _small(cache, scales, table, lens):
    """The requests' blocks alone: a pool of a few blocks on the CPU, and its table."""
    used = [int(b) for row, n in zip(table.tolist(), lens.tolist()) for b in row[: -(-n // PAGE)]]
    at = torch.tensor(used, device="cuda")
    raw = cache.view(torch.uint8)[at].view(cache.dtype) if scales is not None else cache[at]
    new = torch.full_like(table, -1)
    k = 0
    for b, n in enumerate(lens.tolist()):
        pages = -(-n // PAGE)
        new[b, :pages] = torch.arange(k, k + pages, dtype=torch.int32)
        k += pages
    return raw.cpu(), None if scales is None else scales[at].cpu(), new


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_pool_beyond_four_gibibytes(e4m3):
    """140,000 blocks of 32,768 elements: offsets past 2^32 elements, blocks on both sides of
    2^31 and 2^32."""
    a = attn()
    blocks = 140000
    g = torch.Generator().manual_seed(71)
    cache = torch.zeros(blocks, 2, Hkv, PAGE, D, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    cache = cache.view(torch.float8_e4m3fn) if e4m3 else cache
    scales = torch.ones(blocks, 2, Hkv, device="cuda") if e4m3 else None
    lens = torch.tensor([70, 33], dtype=torch.int32)
    table = torch.tensor([[139999, 65535, 65536, 131072, 0], [131071, 139998, 1, -1, -1]], dtype=torch.int32)
    total = int(lens.sum())
    qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    cu = torch.tensor([0, 70, 103], dtype=torch.int32)
    turns, _ = a.rope_turns(D)
    rotation, freq = a.Rotation(turns.cuda()), kv_ref.turns_to_radians(turns.tolist())
    x = qkv.cuda()
    args = (table.cuda(), cu.cuda(), lens.cuda())
    if e4m3:
        q, _ = a.attn_append_paged_e4m3(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, scales, *args, rotation=rotation,
                                        q=x[:, :Hq])
    else:
        q, _ = a.attn_append_paged(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, *args, rotation=rotation, q=x[:, :Hq])
    check_status(a)
    held, sc, small = _small(cache, scales, table, lens)
    for b in range(2):
        n, t0 = int(lens[b]), int(cu[b])
        pos = torch.arange(n)[:, None]
        k, size = kv_ref.rotate(qkv[t0:t0 + n, Hq:Hq + Hkv].double(), pos, freq)
        v = qkv[t0:t0 + n, Hq + Hkv:].double()
        kv = kv_ref.gather(held, small, b, n).transpose(1, 2)
        if e4m3:
            s = kv_ref.gather_scales(sc, small, b, n, PAGE).transpose(1, 2)[..., None]
            want, err = torch.stack((k, v)) / s, torch.stack((kv_ref.ROTATION_ERROR * size, torch.zeros_like(v))) / s
            assert ((kv.double() - want).abs() <= (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) + 1.1 * err).all()
        else:
            kv_ref.check_rows(kv[0], k, size, kv_ref.ROTATION_ERROR, "K")
            assert torch.equal(kv[1].double(), v)
    # Nothing was written past the last slot of the last pages.
    assert not held.view(torch.uint8)[4][:, :, 6:].any() and not held.view(torch.uint8)[7][:, :, 1:].any()
    last = q[[69, 102]].unsqueeze(2).contiguous()
    if e4m3:
        o, lse = a.attn_fwd_decode_paged_e4m3(last, cache, scales, table.cuda(), lens.cuda())
        check_status(a)
        kv_ref.check_decode(o, lse, kv_ref.decode_e4m3(last.cpu(), held, sc, small, lens), 70, "decode")


def test_rope_beyond_two_to_the_31_elements():
    a = attn()
    T, H = 140001, 128
    x = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(72)
    for i in range(0, T, 20000):
        x[i:i + 20000] = torch.randn(x[i:i + 20000].shape, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns, _ = a.rope_turns(D)
    freq = kv_ref.turns_to_radians(turns.tolist())
    y, _ = a.attn_rope(x, None, pos, a.Rotation(turns.cuda()))
    check_status(a)
    rows = torch.tensor([0, 1, 65535, 65536, 131071, 131072, 139999, 140000])
    want, size = kv_ref.rotate(x[rows.cuda()].cpu().double(), rows[:, None], freq)
    kv_ref.check_rows(y[rows.cuda()], want, size, kv_ref.ROTATION_ERROR, "sampled rows")


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_many_requests_and_few_tokens(e4m3):
    """5000 requests of which three have a new token: the search passes over runs of equal
    offsets, and a bad length at the far end is reported."""
    a = attn()
    B, some = 5000, [0, 2999, 4999]
    new = torch.zeros(B, dtype=torch.int32)
    new[some] = 1
    cu = torch.cat((torch.zeros(1, dtype=torch.int32), new.cumsum(0).to(torch.int32)))
    lens = new.clone()
    table = torch.arange(B, dtype=torch.int32)[:, None].contiguous()
    g = torch.Generator().manual_seed(73)
    kv = torch.randn(3, 4, 64, generator=g).to(torch.float16)
    cache = torch.zeros(B, 2, 2, PAGE, 64, dtype=torch.uint8 if e4m3 else torch.float16, device="cuda")
    x = kv.cuda()

    def call(lens):
        if e4m3:
            a.attn_append_paged_e4m3(x[:, :2], x[:, 2:], cache.view(torch.float8_e4m3fn),
                                     torch.ones(B, 2, 2, device="cuda"), table.cuda(), cu.cuda(), lens.cuda())
        else:
            a.attn_append_paged(x[:, :2], x[:, 2:], cache, table.cuda(), cu.cuda(), lens.cuda())

    call(lens)
    check_status(a)
    filled = cache.view(torch.uint8).flatten(1).any(dim=1).cpu().nonzero()[:, 0].tolist()
    assert filled == some
    if not e4m3:
        for j, b in enumerate(some):
            assert torch.equal(cache[b, 0, :, 0].cpu(), kv[j, :2]) and torch.equal(cache[b, 1, :, 0].cpu(), kv[j, 2:])
    lens[4998] = PAGE + 1
    call(lens)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT


def test_two_host_threads():
    """Each thread on a stream of its own, its calls after one another; every round gives the
    same bits."""
    a = attn()
    g = torch.Generator().manual_seed(74)
    turns, _ = a.rope_turns(D)
    rotation = a.Rotation(turns.cuda())
    problems = []
    for n in (50, 300):
        lens = torch.tensor([n, 7], dtype=torch.int32)
        table, blocks = kv_ref.random_table(lens, PAGE, g)
        x = torch.randn(n + 7, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
        cu = torch.tensor([0, n, n + 7], dtype=torch.int32).cuda()
        problems.append((x, cu, lens.cuda(), table.cuda(), blocks))

    def work(p):
        x, cu, lens, table, blocks = p
        cache = torch.zeros(blocks, 2, Hkv, PAGE, D, device="cuda").to(torch.float8_e4m3fn)
        scales = torch.ones(blocks, 2, Hkv, device="cuda")
        q, k = a.attn_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], None, None, torch.arange(
            x.shape[0], dtype=torch.int32, device="cuda"), rotation)
        a.attn_append_paged_e4m3(k, x[:, Hq + Hkv:], cache, scales, table, cu, lens)
        o, lse = a.attn_fwd_decode_paged_e4m3(q[:2].unsqueeze(2).contiguous(), cache, scales, table, lens)
        return q, cache.view(torch.uint8), scales, o, lse

    want = [work(p) for p in problems]
    torch.cuda.synchronize()
    wrong = []

    def loop(p, w):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = work(p)
                stream.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, w)):
                    wrong.append(p)

    threads = [threading.Thread(target=loop, args=(p, w)) for p, w in zip(problems, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    check_status(a)
