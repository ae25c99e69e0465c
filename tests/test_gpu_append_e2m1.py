"""Appending to the paged 4-bit cache: codes and scales bit for bit where nothing is
rotated, within the rotation's fp32 error otherwise."""
import math

import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Problem:
    """B requests with new[b] tokens after past[b] cached ones."""

    def __init__(self, a, new, past, Hq=6, Hkv=2, D=128, page=16, dtype="bf16", rot=None, inter=False,
                 magnitude=1.0, factors=True, seed=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.a, self.D, self.Hq, self.Hkv, self.page = a, D, Hq, Hkv, page
        self.dtype, self.inter, self.magnitude = DTYPES[dtype], inter, magnitude
        self.lens = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32)
        self.cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
        self.total = int(self.cu[-1]) + tail
        size = torch.exp(torch.randn(1, Hq + 2 * Hkv, D, generator=g))  # channels of different sizes
        self.qkv = (size * torch.randn(self.total, Hq + 2 * Hkv, D, generator=g)).to(self.dtype)
        self.table, blocks = kv_ref.random_table(self.lens, page, g)
        self.cache, self.scales = kv4_ref.random_pool(blocks, Hkv, page, D, g)
        self.factors = (0.01 + torch.rand(2, Hkv, generator=g)) if factors else None
        rot = D if rot is None else rot
        turns = a.rope_turns(rot)[0] if rot else torch.empty(0, dtype=torch.int64)
        self.freq = kv_ref.turns_to_radians(turns.tolist())
        self.rotation = a.Rotation(turns.cuda(), inter, magnitude)

    def run(self, with_q=True, with_k=True, positions=None, rotate=True, table=None, lens=None, cu=None):
        dev, Hq, Hkv = self.qkv.cuda(), self.Hq, self.Hkv
        mark = torch.full((self.total, Hq, self.D), 7.0, dtype=self.dtype, device="cuda")
        kout = torch.full((self.total, Hkv, self.D), 7.0, dtype=self.dtype, device="cuda")
        self.dev_cache, self.dev_scales = self.cache.cuda(), self.scales.cuda()
        oq, ok = self.a.attn_append_paged_e2m1(
            dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], self.dev_cache, self.dev_scales,
            (self.table if table is None else table).cuda(), (self.cu if cu is None else cu).cuda(),
            (self.lens if lens is None else lens).cuda(), rotation=self.rotation if rotate else None,
            positions=None if positions is None else positions.cuda(), q=dev[:, :Hq] if with_q else None,
            out_q=mark if with_q else None, out_k=kout if with_k else None,
            factors=None if self.factors is None else self.factors.cuda())
        assert (oq is mark) == with_q and (ok is kout) == with_k
        return (oq.cpu() if with_q else None), (ok.cpu() if with_k else None)

    def check(self, oq, ok, positions=None, rotate=True, skip=()):
        """Everything the call may have written, and that nothing else was."""
        Hq, Hkv = self.Hq, self.Hkv
        q, k, v = (t.double() for t in (self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]))
        cache, scales = self.dev_cache.cpu(), self.dev_scales.cpu()
        js, blk, row, pos = [], [], [], torch.zeros(self.total, dtype=torch.int64)
        for j, b, slot in kv_ref.slots(self.cu.tolist(), self.lens):
            if b in skip:
                continue
            js.append(j)
            blk.append(int(self.table[b, slot // self.page]))
            row.append(slot % self.page)
            pos[j] = slot if positions is None else int(positions[j])
        freq = self.freq if rotate else self.freq[:0]
        kr, ks = kv_ref.rotate(k, pos[:, None], freq, self.inter, self.magnitude)
        qr, qs = kv_ref.rotate(q, pos[:, None], freq, self.inter, self.magnitude)
        mine = torch.zeros(self.total, dtype=torch.bool)
        mine[js] = True
        for out, want, size in ((oq, qr, qs), (ok, kr, ks)):
            if out is not None:
                kv_ref.check_rows(out[mine], want[mine], size[mine], kv_ref.ROTATION_ERROR)
                assert (out[~mine] == 7).all()  # tokens of no request
        seen = torch.zeros(cache.shape[0], self.page, dtype=torch.bool)
        seen[blk, row] = True
        for now, before in ((cache, self.cache), (scales.view(torch.uint8), self.scales.view(torch.uint8))):
            assert torch.equal(now.transpose(1, 3)[~seen], before.transpose(1, 3)[~seen])
        if not js:
            return
        factors = torch.ones(2, Hkv) if self.factors is None else self.factors
        codes, sc = kv4_ref.unpack(cache[blk, :, :, row]), scales.float()[blk, :, :, row]
        want, ws = kv4_ref.quantise(self.qkv[js, Hq + Hkv:], factors[1][:, None])
        assert torch.equal(sc[:, 1], ws) and torch.equal(codes[:, 1], want), "V"
        if len(freq) == 0:
            want, ws = kv4_ref.quantise(self.qkv[js, Hq:Hq + Hkv], factors[0][:, None])
            assert torch.equal(sc[:, 0], ws) and torch.equal(codes[:, 0], want), "K"
            return
        # Rounding is monotone: scale and codes lie between those of the ends of the fp32 error.
        x, e = kr[js], kv_ref.ROTATION_ERROR * ks[js]
        f = factors[0][:, None]
        ends = []
        for sign in (-1, 1):
            far = (x.abs() + sign * e).clamp(min=0).unflatten(-1, (-1, 16)).amax(dim=-1) * (1 + sign * 2.0 ** -22)
            ends.append(kv4_ref.scales_of(far.float(), f))
        assert ((ends[0] <= sc[:, 0]) & (sc[:, 0] <= ends[1])).all(), "scales of K"
        by = (1.0 / (sc[:, 0].double() * f.double())).repeat_interleave(16, dim=-1)
        slack = e * by + (x * by).abs() * 2.0 ** -22  # and the reciprocal's and the product's roundings
        got = kv4_ref.values(codes[:, 0])
        low, high = (kv4_ref.values(kv4_ref.e2m1(x * by + s * slack)) for s in (-1, 1))
        assert ((low <= got) & (got <= high)).all(), "codes of K"


CASES = [
    dict(new=[1], past=[0]),
    dict(new=[1, 1, 1], past=[15, 16, 17]),
    dict(new=[40, 1, 0, 17], past=[0, 3, 9, 30], factors=False),
    dict(new=[5, 33], past=[0, 70], page=1),
    dict(new=[50, 8, 29], past=[3, 0, 61], page=5, D=64),
    dict(new=[300], past=[130], page=256, D=64, Hkv=1),
    dict(new=[23, 19], past=[5, 7], page=24, Hq=12, Hkv=12),
    dict(new=[19, 64], past=[0, 33], dtype="f16", inter=True, rot=64),
    dict(new=[19, 20], past=[0, 33], dtype="f16", rot=20, D=64),
    dict(new=[9, 14], past=[2, 3], rot=32, Hkv=5),                  # two chunks turn: pairs of chunks in a lane behind
    dict(new=[9, 14], past=[2, 3], rot=16, Hkv=3),                  # one chunk: a group's halves in one lane
    dict(new=[9, 14], past=[2, 3], rot=48, Hkv=3, D=64),            # three: a group's halves in different places
    dict(new=[9, 14], past=[2, 3], rot=112, magnitude=1.25, Hkv=5),
    dict(new=[9, 14], past=[2, 3], rot=36, magnitude=0.5),
    dict(new=[9, 14], past=[2, 3], rot=0),
    dict(new=[700, 400], past=[0, 100], Hq=32, Hkv=8),
    dict(new=[4, 5], past=[20, 30], tail=6),                        # rows behind the last request
    dict(new=[1] * 150, past=[(7 * i) % 40 for i in range(150)]),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_append(case):
    a = attn()
    pr = Problem(a, **case, seed=131)
    oq, ok = pr.run()
    check_status(a)
    pr.check(oq, ok)
    before = pr.dev_cache.clone(), pr.dev_scales.clone()
    pr.run(with_q=False, with_k=False)
    assert torch.equal(pr.dev_cache, before[0])
    assert torch.equal(pr.dev_scales.view(torch.uint8), before[1].view(torch.uint8))
    oq, ok = pr.run(rotate=False)
    check_status(a)
    pr.check(oq, ok, rotate=False)
    assert torch.equal(oq[:int(pr.cu[-1])], pr.qkv[:int(pr.cu[-1]), :pr.Hq])


def test_positions_of_the_caller():
    a = attn()
    pr = Problem(a, new=[20, 3], past=[5, 12], seed=132)
    positions = torch.randint(-100, 100000, (23,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    pr.check(*pr.run(positions=positions), positions=positions)
    check_status(a)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_every_value_and_every_tie(D, dtype):
    """All finite 16-bit patterns: the borders of codes and scales, subnormals, both zeros."""
    a = attn()
    pr = Problem(a, [512 * 128 // D], [0], Hq=1, Hkv=1, D=D, dtype=dtype, rot=0, seed=133, factors=False)
    pr.qkv = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(pr.dtype).reshape(-1, 1, D)
    pr.qkv = torch.where(torch.isfinite(pr.qkv.float()), pr.qkv, torch.zeros_like(pr.qkv)).repeat(1, 3, 1)
    g = torch.Generator().manual_seed(134)
    pr.qkv[:, 2] = pr.qkv[:, 2].flatten()[torch.randperm(pr.total * D, generator=g)].reshape(-1, D)
    for factors in (None, torch.tensor([[0.37], [1e-4]]), torch.tensor([[2.0 ** 40], [2.0 ** -60]])):
        pr.factors = factors
        pr.check(*pr.run(rotate=False), rotate=False)
        check_status(a)


def test_infinities_and_nan():
    a = attn()
    pr = Problem(a, new=[4], past=[0], Hkv=2, D=64, rot=0, seed=135, factors=False)
    kv = pr.qkv[:, pr.Hq:]
    kv[:] = 3.0
    kv[0, 0, 5] = math.inf
    kv[0, 0, 20] = -math.inf
    kv[1, 1, 33] = math.nan
    kv[1, 1, 34] = math.inf
    kv[2, 2, 16:32] = math.inf
    kv[3, 3] = 0.0
    pr.run()
    check_status(a)
    blk = int(pr.table[0, 0])
    x = kv4_ref.held(pr.dev_cache.cpu(), pr.dev_scales.cpu(), None)[blk]  # [2, Hkv, page, D]
    assert x[0, 0, 0, 5] == 3.0 and x[0, 0, 0, 20] == -3.0 and (x[0, 0, 0, :5] == 3).all()  # 6 scales
    assert torch.isnan(x[0, 1, 1, 32:48]).all() and (x[0, 1, 1, :32] == 3).all() and (x[0, 1, 1, 48:] == 3).all()
    assert (x[1, 0, 2, 16:32] == 6 * 2.0 ** -9).all() and (x[1, 0, 2, :16] == 3).all()  # nothing finite: the least scale
    assert (x[1, 1, 3] == 0).all()


def test_token_by_token_equals_one_call():
    a = attn()
    pr = Problem(a, new=[37], past=[0], seed=136)
    pr.run()
    dev, cache, scales = pr.qkv.cuda(), pr.cache.cuda(), pr.scales.cuda()
    at = 0
    for n in (1, 15, 1, 1, 18, 1):
        t = dev[at:at + n]
        at += n
        a.attn_append_paged_e2m1(t[:, 6:8], t[:, 8:], cache, scales, pr.table.cuda(),
                                 torch.tensor([0, n], dtype=torch.int32).cuda(),
                                 torch.tensor([at], dtype=torch.int32).cuda(), rotation=pr.rotation,
                                 factors=pr.factors.cuda())
    check_status(a)
    assert torch.equal(pr.dev_cache, cache) and torch.equal(pr.dev_scales.view(torch.uint8), scales.view(torch.uint8))


def test_bad_requests_and_blocks_are_left_out():
    a = attn()
    pr = Problem(a, new=[20, 9, 6], past=[3, 2, 40], seed=137)
    for b, length in ((1, 8), (1, -1), (0, pr.table.shape[1] * 16 + 1)):
        lens = pr.lens.clone()
        lens[b] = length
        oq, ok = pr.run(lens=lens)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        pr.check(oq, ok, skip=(b,))
    cu = pr.cu.clone()
    cu[2] = cu[3] + 4
    oq, ok = pr.run(cu=cu)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    pr.check(oq, ok, skip=(1, 2))
    pr.run()
    want = pr.dev_cache.cpu(), pr.dev_scales.cpu().view(torch.uint8)
    for bad in (-1, pr.cache.shape[0], 2 ** 31 - 1):
        table = pr.table.clone()
        table[0, 0] = bad
        pr.run(table=table)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        blk = int(pr.table[0, 0])
        rest = torch.arange(pr.cache.shape[0]) != blk
        for now, full, before in zip((pr.dev_cache.cpu(), pr.dev_scales.cpu().view(torch.uint8)), want,
                                     (pr.cache, pr.scales.view(torch.uint8))):
            assert torch.equal(now[rest], full[rest]) and torch.equal(now[blk], before[blk])


def test_graph_replay_on_a_side_stream():
    a = attn()
    pr = Problem(a, new=[1, 1], past=[13, 30], seed=138)
    table = torch.tensor([[0, 1, 4, 5], [2, 3, 6, 7]], dtype=torch.int32).cuda()
    caches = [torch.zeros(8, 2, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(8, 2, 2, 16, 8, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    x, lens, cu, factors = pr.qkv.cuda(), pr.lens.cuda(), pr.cu.cuda(), pr.factors.cuda()
    outs = [torch.empty_like(x[:, :6]) for _ in range(2)]

    def step(x, i):
        a.attn_append_paged_e2m1(x[:, 6:8], x[:, 8:], caches[i], scales[i], table, cu, lens, rotation=pr.rotation,
                                 q=x[:, :6], out_q=outs[i], factors=factors)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(x, 0)
    rows = torch.Generator().manual_seed(5)
    with torch.cuda.stream(side):
        for i in range(6):
            fresh = (torch.randn(x.shape, generator=rows) * (i + 1)).to(x.dtype).cuda()
            x.copy_(fresh)
            graph.replay()
            step(fresh, 1)
            side.synchronize()
            assert torch.equal(*outs) and torch.equal(*caches)
            assert torch.equal(*(s.view(torch.uint8) for s in scales))
            lens += 1
    check_status(a)


def test_no_tokens_launch_nothing():
    a = attn()
    pr = Problem(a, new=[0, 0], past=[3, 0], seed=139)
    pr.run()
    assert a.last_launch_info()[2] == 0
    assert torch.equal(pr.dev_cache.cpu(), pr.cache)
