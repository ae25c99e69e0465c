"""Appending keys and values to the paged caches (16-bit, and 8-bit with block
scales) against their 64-bit forms, bit for bit where nothing is computed."""
import math

import pytest
import torch

import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Problem:
    """B requests with new[b] tokens after past[b] cached ones."""

    def __init__(self, a, new, past, Hq=6, Hkv=2, D=128, page=16, dtype="bf16", rot=None, inter=False,
                 magnitude=1.0, e4m3=False, seed=0, tail=0, scale_range=(-9, -5)):
        g = torch.Generator().manual_seed(seed)
        self.a, self.D, self.Hq, self.Hkv, self.page, self.e4m3 = a, D, Hq, Hkv, page, e4m3
        self.dtype, self.inter, self.magnitude = DTYPES[dtype], inter, magnitude
        self.new, self.past = list(new), list(past)
        self.lens = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32)
        self.cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
        self.total = int(self.cu[-1]) + tail
        self.qkv = torch.randn(self.total, Hq + 2 * Hkv, D, generator=g).to(self.dtype)
        self.table, blocks = kv_ref.random_table(self.lens, page, g)
        shape = (blocks, 2, Hkv, page, D)
        if e4m3:
            self.cache = kv_ref.random_codes(shape, g)
            self.scales = torch.exp2(torch.randint(*scale_range, (blocks, 2, Hkv), generator=g).float())
        else:
            self.cache, self.scales = torch.randn(shape, generator=g).to(self.dtype), None
        rot = D if rot is None else rot
        turns = a.rope_turns(rot)[0] if rot else torch.empty(0, dtype=torch.int64)
        self.freq = kv_ref.turns_to_radians(turns.tolist())
        self.rotation = a.Rotation(turns.cuda(), inter, magnitude)

    @property
    def q(self):
        return self.qkv[:, :self.Hq]

    @property
    def k(self):
        return self.qkv[:, self.Hq:self.Hq + self.Hkv]

    @property
    def v(self):
        return self.qkv[:, self.Hq + self.Hkv:]

    def run(self, with_q=True, with_k=True, positions=None, rotate=True, table=None, lens=None, cu=None):
        a, dev = self.a, self.qkv.cuda()
        Hq, Hkv = self.Hq, self.Hkv
        q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
        mark = torch.full((self.total, Hq, self.D), 7.0, dtype=self.dtype, device="cuda")
        kout = torch.full((self.total, Hkv, self.D), 7.0, dtype=self.dtype, device="cuda")
        self.dev_cache = self.cache.cuda()
        kw = dict(rotation=self.rotation if rotate else None, positions=None if positions is None else positions.cuda(),
                  q=q if with_q else None, out_q=mark if with_q else None, out_k=kout if with_k else None)
        args = ((self.table if table is None else table).cuda(), (self.cu if cu is None else cu).cuda(),
                (self.lens if lens is None else lens).cuda())
        if self.e4m3:
            self.dev_scales = self.scales.cuda()
            oq, ok = a.attn_append_paged_e4m3(k, v, self.dev_cache, self.dev_scales, *args, **kw)
        else:
            oq, ok = a.attn_append_paged(k, v, self.dev_cache, *args, **kw)
        assert (oq is mark) == with_q and (ok is kout) == with_k
        return (oq.cpu() if with_q else None), (ok.cpu() if with_k else None)

    def check(self, oq, ok, positions=None, rotate=True, skip=()):
        """Everything the call may have written, and that nothing else was."""
        cache = self.dev_cache.cpu()
        raw_now, raw_before = (c.view(torch.uint8) if self.e4m3 else c for c in (cache, self.cache))
        seen = torch.zeros(self.cache.shape[0], self.page, dtype=torch.bool)
        tokens = torch.zeros(self.total, dtype=torch.bool)
        pos = torch.zeros(self.total, dtype=torch.int64)
        at = {}
        for j, b, slot in kv_ref.slots(self.cu.tolist(), self.lens):
            if b in skip:
                continue
            blk, row = int(self.table[b, slot // self.page]), slot % self.page
            seen[blk, row] = tokens[j] = True
            pos[j] = slot if positions is None else int(positions[j])
            at[j] = (blk, row)
        freq = self.freq if rotate else self.freq[:0]
        kr, ks = kv_ref.rotate(self.k.double(), pos[:, None], freq, self.inter, self.magnitude)
        qr, qs = kv_ref.rotate(self.q.double(), pos[:, None], freq, self.inter, self.magnitude)
        for out, want, size in ((oq, qr, qs), (ok, kr, ks)):
            if out is not None:
                kv_ref.check_rows(out[tokens], want[tokens], size[tokens], kv_ref.ROTATION_ERROR)
                assert (out[~tokens] == 7).all()  # tokens of no request
        old_rows = self.check_scales(cache, skip, rotate) if self.e4m3 else torch.zeros_like(seen)
        untouched = ~seen & ~old_rows
        assert torch.equal(raw_now.transpose(1, 3)[untouched], raw_before.transpose(1, 3)[untouched])
        if not at:
            return
        js = torch.tensor(sorted(at))
        blk = torch.tensor([at[int(j)][0] for j in js])
        row = torch.tensor([at[int(j)][1] for j in js])
        if not self.e4m3:
            kv_ref.check_rows(cache[blk, 0, :, row], kr[js], ks[js], kv_ref.ROTATION_ERROR, "K rows")
            assert torch.equal(cache[blk, 1, :, row].view(torch.int16), self.v[js].view(torch.int16))
            return
        s = self.dev_scales.cpu().double()[blk]
        got = raw_now[blk, :, :, row].view(torch.float8_e4m3fn).double()
        for j, (x, size, error) in enumerate(((kr[js], ks[js], kv_ref.ROTATION_ERROR),
                                              (self.v[js].double(), self.v[js].double().abs(), 0.0))):
            u = x / s[:, j][..., None]
            # Half a step of e4m3 (2^-4, 2^-10 among its subnormals) around the fp32 value.
            tol = 2.0 ** -4 * u.abs() + 1.1 * error * size / s[:, j][..., None]
            tol = torch.maximum(tol, torch.full_like(tol, 2.0 ** -10) + 1.1 * error * size / s[:, j][..., None])
            assert ((got[:, j] - u).abs() <= tol).all(), f"codes of {'KV'[j]}"

    def check_scales(self, cache, skip, rotate):
        """Scales are exact; older rows of a grown block are its codes divided and rounded."""
        now, limits = self.dev_scales.cpu(), (kv_ref.k_limit(self.magnitude, 2 * len(self.freq) if rotate else 0, self.D), 448.0)
        want, old_rows = self.scales.clone(), torch.zeros(self.cache.shape[0], self.page, dtype=torch.bool)
        cu, lens = self.cu.tolist(), self.lens.tolist()
        for b in range(len(lens)):
            if b in skip or cu[b] == cu[b + 1]:
                continue
            start = lens[b] - (cu[b + 1] - cu[b])
            for page in range(start // self.page, -(-lens[b] // self.page)):
                lo, hi = max(start, page * self.page), min(lens[b], (page + 1) * self.page)
                blk = int(self.table[b, page])
                held = lo - page * self.page
                toks = slice(cu[b] + lo - start, cu[b] + hi - start)
                for j, x in enumerate((self.k[toks], self.v[toks])):
                    f = x.float().abs()
                    most = torch.where(torch.isfinite(f), f, torch.zeros_like(f)).amax(dim=(0, 2))
                    for h in range(self.Hkv):
                        s = kv_ref.pow2_scale(float(most[h]), limits[j])
                        if held:
                            s = max(s, float(self.scales[blk, j, h]))
                            ratio = float(self.scales[blk, j, h]) / s
                            old = self.cache[blk, j, h, :held].float() * ratio
                            assert torch.equal(cache[blk, j, h, :held].float(),
                                               old.to(torch.float8_e4m3fn).float()), "older rows"
                        want[blk, j, h] = s
                old_rows[blk, :held] = True
        assert torch.equal(now, want), "scales"
        return old_rows


CASES = [
    dict(new=[1], past=[0]),
    dict(new=[1, 1, 1], past=[15, 16, 17]),                       # the last row of a page, the first, the second
    dict(new=[40, 1, 0, 17], past=[0, 3, 9, 30]),                 # a request without new tokens
    dict(new=[5, 33], past=[0, 70], page=1),
    dict(new=[50, 8, 29], past=[3, 0, 61], page=5, D=64),
    dict(new=[200, 31], past=[11, 40], page=64),
    dict(new=[300], past=[130], page=256, D=64, Hkv=1),
    dict(new=[23, 19], past=[5, 7], page=24, Hq=12, Hkv=12),
    dict(new=[19, 64], past=[0, 33], dtype="f16", inter=True, rot=64),
    dict(new=[19, 20], past=[0, 33], dtype="f16", rot=20, D=64),
    dict(new=[9, 14], past=[2, 3], rot=36, magnitude=1.25, Hkv=5),
    dict(new=[9, 14], past=[2, 3], rot=6, magnitude=0.5),           # what passes is larger than what turns
    dict(new=[9, 14], past=[2, 3], magnitude=0.5),
    dict(new=[9, 14], past=[2, 3], rot=0),
    dict(new=[700, 400], past=[0, 100], Hq=32, Hkv=8),
    dict(new=[4, 5], past=[20, 30], tail=6),                      # rows behind the last request
    dict(new=[1] * 150, past=[(7 * i) % 40 for i in range(150)]),  # many requests: two probes of the search
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_append(case, e4m3):
    a = attn()
    pr = Problem(a, **case, e4m3=e4m3, seed=31)
    oq, ok = pr.run()
    check_status(a)
    pr.check(oq, ok)
    # The queries alone change nothing else, and none at all works.
    before = pr.dev_cache.clone()
    pr.run(with_q=False, with_k=False)
    check_status(a)
    assert torch.equal(pr.dev_cache.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_positions_of_the_caller_and_no_rotation(e4m3):
    a = attn()
    pr = Problem(a, new=[20, 3], past=[5, 12], e4m3=e4m3, seed=32)
    positions = torch.randint(-100, 100000, (23,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    pr.check(*pr.run(positions=positions), positions=positions)
    oq, ok = pr.run(rotate=False)
    pr.check(oq, ok, rotate=False)
    assert torch.equal(oq, pr.q) and torch.equal(ok, pr.k)  # copies
    check_status(a)


def test_token_by_token_equals_one_call():
    """The 16-bit cache does not depend on how the tokens arrive."""
    a = attn()
    pr = Problem(a, new=[37], past=[0], seed=33)
    pr.run()
    whole = pr.dev_cache.clone()
    dev, cache = pr.qkv.cuda(), pr.cache.cuda()
    at = 0
    for n in (1, 15, 1, 1, 18, 1):
        t = dev[at:at + n]
        at += n
        a.attn_append_paged(t[:, 6:8], t[:, 8:], cache, pr.table.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                            torch.tensor([at], dtype=torch.int32).cuda(), rotation=pr.rotation)
    check_status(a)
    assert torch.equal(whole, cache)


def test_e4m3_scale_grows_token_by_token():
    """Rows of growing size, one at a time: the scale follows, and what is held stays within
    half a step of e4m3 at the last scale plus the divisions among its subnormals."""
    a = attn()
    D, page, Hkv = 64, 16, 2
    g = torch.Generator().manual_seed(34)
    x = torch.randn(page, 2 * Hkv, D, generator=g) * torch.exp2(torch.arange(page).float() - 8)[:, None, None]
    x = x.to(torch.bfloat16)
    cache = torch.zeros(1, 2, Hkv, page, D, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((1, 2, Hkv), 1.0, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(page):
        row = x[i:i + 1].cuda()
        a.attn_append_paged_e4m3(row[:, :Hkv], row[:, Hkv:], cache, scales, table, one,
                                 torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
        most = x[:i + 1].float().abs().amax(dim=(0, 2))
        want = torch.tensor([kv_ref.pow2_scale(float(m), 448.0) for m in most]).reshape(2, Hkv)
        assert torch.equal(scales.cpu()[0], want), i
    check_status(a)
    held = (cache.cpu().float() * scales.cpu()[..., None, None])[0].permute(2, 0, 1, 3).reshape(page, 2 * Hkv, D)
    step = scales.cpu()[0].reshape(1, 2 * Hkv, 1) * 2.0 ** -9
    # One rounding of the row (2^-4), then one of half a subnormal step for every growth (each
    # halves what came before): under a whole step in all.
    assert ((held - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + step).all()


def test_e4m3_codes_of_odd_values():
    """Zero rows, infinities and NaN, the type's extremes, values next to a scale's border."""
    a = attn()
    for dtype in ("bf16", "f16"):
        pr = Problem(a, new=[4, 3, 2], past=[0, 5, 0], Hkv=3, D=64, rot=0, dtype=dtype, e4m3=True, seed=35)
        big = torch.finfo(pr.dtype).max
        kv = pr.qkv[:, pr.Hq:]
        kv[:4, 0] = 0.0                        # an empty block
        kv[:4, 1] = 448.0                      # exactly a scale of 1
        kv[0, 2, 0] = big
        kv[1, 3, 3] = math.inf
        kv[2, 3, 4] = -math.inf
        kv[3, 3, 5] = math.nan
        kv[4:7, 4] = torch.finfo(pr.dtype).tiny / 4
        kv[7:9, 0] = math.nan                  # nothing finite
        kv[7:9, 5] = 450.0                     # just over 448
        oq, ok = pr.run(rotate=False)
        check_status(a)
        pr.check_scales(pr.dev_cache.cpu(), (), False)
        s, c = pr.dev_scales.cpu(), pr.dev_cache.cpu().float()
        blk = [int(pr.table[b, 0]) for b in range(3)]
        assert s[blk[0], 0, 0] == 2.0 ** -100 and (c[blk[0], 0, 0, :4] == 0).all()
        assert s[blk[0], 0, 1] == 1.0 and (c[blk[0], 0, 1, :4] == 448).all()
        assert c[blk[0], 1, 0, 1, 3] == 448 and c[blk[0], 1, 0, 2, 4] == -448
        assert math.isnan(c[blk[0], 1, 0, 3, 5])
        assert torch.isnan(c[blk[2], 0, 0, :2]).all() and s[blk[2], 0, 0] == 2.0 ** -100
        assert s[blk[2], 1, 2] == 2.0


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_bad_requests_and_blocks_are_left_out(e4m3):
    a = attn()
    pr = Problem(a, new=[20, 9, 6], past=[3, 2, 40], e4m3=e4m3, seed=36)
    for b, length in ((1, 8), (1, -1), (0, pr.table.shape[1] * 16 + 1)):  # under the new tokens, over the table
        lens = pr.lens.clone()
        lens[b] = length
        oq, ok = pr.run(lens=lens)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        pr.check(oq, ok, skip=(b,))
    cu = pr.cu.clone()
    cu[2] = cu[3] + 4  # past the tokens: requests 1 and 2 are not valid
    oq, ok = pr.run(cu=cu)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    pr.check(oq, ok, skip=(1, 2))
    cu = pr.cu.clone()
    cu[0] = -3
    oq, ok = pr.run(cu=cu)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    pr.check(oq, ok, skip=(0,))
    for bad in (-1, pr.cache.shape[0], 2 ** 31 - 1):
        table = pr.table.clone()
        table[0, 0] = bad
        pr.run(table=table)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        # Only that page is missing.
        want = Problem(a, new=[20, 9, 6], past=[3, 2, 40], e4m3=e4m3, seed=36)
        want.run()
        blk = int(pr.table[0, 0])
        keep = torch.arange(pr.cache.shape[0]) != blk
        raw = [c.cpu().view(torch.uint8) for c in (pr.dev_cache, want.dev_cache, pr.cache.cuda())]
        assert torch.equal(raw[0][keep], raw[1][keep]) and torch.equal(raw[0][blk], raw[2][blk])
        check_status(a)


def test_no_tokens_launch_nothing():
    a = attn()
    pr = Problem(a, new=[0, 0], past=[3, 0], seed=37)
    pr.run()
    assert a.last_launch_info()[2] == 0
    assert torch.equal(pr.dev_cache.cpu(), pr.cache)


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_graph_replay_and_other_stream(e4m3):
    """One graph over growing lengths, its inputs changed between replays, on a side stream."""
    a = attn()
    pr = Problem(a, new=[1, 1], past=[13, 30], e4m3=e4m3, seed=38, scale_range=(-6, -5))
    eager = Problem(a, new=[1, 1], past=[13, 30], e4m3=e4m3, seed=38, scale_range=(-6, -5))
    pr.table = eager.table = torch.tensor([[0, 1, 4, 5], [2, 3, 6, 7]], dtype=torch.int32)
    shape = (8,) + tuple(pr.cache.shape[1:])
    cache = torch.zeros(shape).to(pr.cache.dtype)
    g_cache, e_cache = cache.cuda(), cache.cuda()
    g_scales, e_scales = (torch.ones(8, 2, 2, device="cuda") for _ in range(2))
    x, lens, table, cu = pr.qkv.cuda(), pr.lens.cuda(), pr.table.cuda(), pr.cu.cuda()

    def step(x, cache, scales, lens, out):
        if e4m3:
            a.attn_append_paged_e4m3(x[:, 6:8], x[:, 8:], cache, scales, table, cu, lens, rotation=pr.rotation,
                                     q=x[:, :6], out_q=out)
        else:
            a.attn_append_paged(x[:, 6:8], x[:, 8:], cache, table, cu, lens, rotation=pr.rotation, q=x[:, :6], out_q=out)

    out, want = torch.empty_like(x[:, :6]), torch.empty_like(x[:, :6])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(x, g_cache, g_scales, lens, out)
    rows = torch.Generator().manual_seed(5)
    with torch.cuda.stream(side):
        for i in range(6):
            fresh = (torch.randn(x.shape, generator=rows) * (i + 1)).to(x.dtype).cuda()
            x.copy_(fresh)
            graph.replay()
            step(fresh, e_cache, e_scales, lens, want)
            side.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(g_cache.view(torch.uint8), e_cache.view(torch.uint8))
            assert torch.equal(g_scales, e_scales)
            lens += 1
    check_status(a)


@pytest.mark.parametrize("D,page,dtype,e4m3", [(128, 16, "bf16", False), (64, 5, "f16", False), (64, 16, "bf16", True),
                                               (128, 24, "f16", True)])
def test_without_a_rotation_rows_are_copied_bit_for_bit(D, page, dtype, e4m3):
    """Every 16-bit pattern, zeros of both signs and NaN of any payload among them."""
    a = attn()
    pr = Problem(a, [90, 3], [7, 0], Hq=5, Hkv=3, D=D, page=page, dtype=dtype, rot=0, e4m3=e4m3, seed=71)
    g = torch.Generator().manual_seed(72)
    pr.qkv = torch.randint(-2 ** 15, 2 ** 15, pr.qkv.shape, generator=g).to(torch.int16).view(pr.dtype)
    pr.qkv[::3, ::2] = -0.0
    for rotate in (False, True):  # no rotation, and one of no elements
        oq, ok = pr.run(rotate=rotate)
        check_status(a)
        assert torch.equal(oq.view(torch.int16), pr.q.view(torch.int16))
        assert torch.equal(ok.view(torch.int16), pr.k.view(torch.int16))
        if e4m3:
            continue
        cache = pr.dev_cache.cpu().view(torch.int16)
        for j, b, slot in kv_ref.slots(pr.cu.tolist(), pr.lens):
            blk, row = int(pr.table[b, slot // page]), slot % page
            assert torch.equal(cache[blk, 0, :, row], pr.k[j].view(torch.int16))
            assert torch.equal(cache[blk, 1, :, row], pr.v[j].view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [[0, 20, 1000, 29, 35], [0, 20, 5, 29, 35], [0, 20, -7, 29, 35], [35, 29, 20, 5, 0],
                                 [0, 2 ** 31 - 1, -2 ** 31, 29, 35]])
def test_offsets_out_of_order_are_reported_and_stay_in_their_pages(bad, e4m3):
    """Any request of the call may miss tokens; blocks of no request, and every slot before a
    token that a valid request could have, stay as they were, and the next call is whole."""
    a = attn()
    pr = Problem(a, new=[20, 3, 6, 6], past=[16, 48, 160, 160], e4m3=e4m3, seed=73)
    oq, ok = pr.run(cu=torch.tensor(bad, dtype=torch.int32))
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    kept = torch.ones(pr.cache.shape[0], dtype=torch.bool)
    for b, n in enumerate(pr.lens.tolist()):
        if 0 <= bad[b] <= bad[b + 1] <= pr.total and bad[b + 1] - bad[b] <= n:
            first = (n - (bad[b + 1] - bad[b])) // pr.page
            kept[pr.table[b, first:-(-n // pr.page)].long()] = False
    now, before = pr.dev_cache.cpu().view(torch.uint8), pr.cache.view(torch.uint8)
    assert torch.equal(now[kept], before[kept]) and int(kept.sum()) > 3
    if e4m3:
        assert torch.equal(pr.dev_scales.cpu()[kept], pr.scales[kept])
    oq, ok = pr.run()
    check_status(a)
    pr.check(oq, ok)
