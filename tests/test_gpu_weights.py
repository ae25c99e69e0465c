"""Attention weights of packed queries, added up over a paged cache's keys, against their
64-bit form."""
import math

import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Problem:
    """B requests of lens[b] keys, the last new[b] of which are the queries."""

    def __init__(self, lens, new, Hq=8, Hkv=2, D=128, page=16, dtype="bf16", four=False, seed=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
        total = int(self.cu[-1]) + tail
        self.q = torch.randn(total, Hq, D, generator=g).to(DTYPES[dtype])
        seen = torch.cat([torch.arange(n - m, n) + 1.0 for n, m in zip(lens, new)] + [torch.ones(tail)])
        self.lse = seen.log() + 0.5 + 0.1 * torch.randn(Hq, total, generator=g)
        self.table, blocks = kv_ref.random_table(self.lens, page, g)
        self.four, self.factors, self.scales = four, None, None
        if four:
            self.cache, self.scales = kv4_ref.random_pool(blocks, Hkv, page, D, g)
            self.factors = 0.5 + torch.rand(2, Hkv, generator=g)
        else:
            self.cache = torch.randn(blocks, 2, Hkv, page, D, generator=g).to(DTYPES[dtype])
        self.weights = torch.rand(blocks, Hkv, page, generator=g)

    def pool(self):
        return kv4_ref.held(self.cache, self.scales, self.factors) if self.four else self.cache

    def run(self, a, scale=None, q=None, lse=None, table=None, cu=None, lens=None):
        w = self.weights.cuda()
        q, lse = (self.q.cuda() if q is None else q), (self.lse.cuda() if lse is None else lse)
        table, cu, lens = (((x if y is None else y).cuda()) for x, y in
                           ((self.table, table), (self.cu, cu), (self.lens, lens)))
        if self.four:
            got = a.attn_weights_paged_e2m1(q, lse, self.cache.cuda(), self.scales.cuda(), table, cu, lens, w,
                                            scale=scale, factors=None if self.factors is None else self.factors.cuda())
        else:
            got = a.attn_weights_paged(q, lse, self.cache.cuda(), table, cu, lens, w, scale=scale)
        assert got is w
        return w

    def check(self, w, scale=None, skip=(), what=""):
        lens = self.lens.clone()
        share, tol = kv4_ref.column_sums(self.q, self.lse, self.pool(), self.table, self.cu, lens, scale)
        for b in skip:
            share[b], tol[b] = share[b] * 0, tol[b] * 0
        kv4_ref.check_weights(w, self.weights, self.table, lens, share, tol,
                              int(torch.diff(self.cu).max()) * self.q.shape[1], what)


fours = pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])

CASES = [
    dict(lens=[1], new=[1], Hq=1, Hkv=1, D=64),
    dict(lens=[1, 2, 15, 16, 17, 31, 32, 33], new=[1, 1, 1, 1, 1, 1, 1, 1], Hq=4, Hkv=4),
    dict(lens=[300, 0, 5], new=[7, 0, 5]),
    dict(lens=[300, 40], new=[0, 0]),
    dict(lens=[129, 64, 128, 127], new=[129, 64, 1, 2], Hq=16, Hkv=16, D=64, page=8, dtype="f16"),
    dict(lens=[3, 40, 7], new=[3, 33, 1], Hq=4, D=64, page=1),
    dict(lens=[700, 33], new=[100, 33], Hq=6, page=5, dtype="f16"),
    dict(lens=[500, 90], new=[70, 17], Hq=7, Hkv=1, page=24),
    dict(lens=[300], new=[9], Hq=33, Hkv=1),
    dict(lens=[700, 256], new=[64, 256], Hq=8, Hkv=1, page=256, D=64),
    dict(lens=[2048, 31, 900], new=[1, 1, 64], Hq=32, Hkv=8),
    dict(lens=[5000], new=[33], Hq=12, Hkv=12, D=64, page=48, dtype="f16"),
    dict(lens=[260, 70], new=[40, 3], tail=9),   # rows behind the last request
    dict(lens=[(37 * i) % 90 + 1 for i in range(150)], new=[min((37 * i) % 90 + 1, i % 5) for i in range(150)], Hq=2),
    dict(lens=[1100], new=[1100], Hq=4, Hkv=2),  # a whole prompt
    dict(lens=[600, 100], new=[2, 5], Hq=130, Hkv=1, D=64),  # more heads than a tile has rows
    dict(lens=[2000, 700, 2600], new=[1400, 30, 513], Hq=2, Hkv=1, D=64),  # ranges of queries
    dict(lens=[1029], new=[1029], Hq=3, Hkv=1, D=64, page=5, dtype="f16"),
    dict(lens=[33, 500, 0, 700, 257, 64], new=[1, 1, 0, 1, 1, 1], Hq=32, Hkv=2, D=64),  # a step of 16 heads to a KV head
    dict(lens=[900] + [40] * 30, new=[31] + [0] * 30, Hq=4, Hkv=4),   # eight rows to a request, and all in one
    dict(lens=[5000, 4100, 1, 3], new=[2, 2, 1, 3], Hq=8, Hkv=2, page=1),
    dict(lens=[(53 * i) % 700 for i in range(60)], new=[min(1, (53 * i) % 700) for i in range(60)], Hq=7, Hkv=7, page=24),
]


@fours
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_the_definition(case, four):
    a = attn()
    pr = Problem(**case, four=four, seed=161)
    w = pr.run(a)
    check_status(a)
    pr.check(w, what=str(case))
    assert torch.equal(pr.run(a), w)  # the same bits again
    pr.check(pr.run(a, scale=0.01), scale=0.01)


def test_without_factors():
    a = attn()
    pr = Problem([100, 40], [3, 40], four=True, seed=162)
    pr.factors = None
    pr.check(pr.run(a))


@fours
def test_wide_table(four):
    a = attn()
    pr = Problem([300, 70], [65, 1], four=four, seed=163)
    w = pr.run(a)
    assert torch.equal(pr.run(a, table=torch.nn.functional.pad(pr.table, (0, 4000), value=-3)), w)
    check_status(a)


@fours
def test_strides_of_queries_and_lse(four):
    """A slice of a fused projection, heads before tokens, and lse as a decode returns it."""
    a = attn()
    pr = Problem([90, 40], [12, 40], Hq=8, Hkv=4, four=four, seed=164)
    w = pr.run(a)
    fused = torch.randn(52, 20, 128).to(torch.bfloat16).cuda()
    fused[:, 3:11] = pr.q.cuda()
    assert torch.equal(pr.run(a, q=fused[:, 3:11]), w)
    assert torch.equal(pr.run(a, q=pr.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)), w)
    assert torch.equal(pr.run(a, lse=pr.lse.cuda().t().contiguous().t()), w)
    pr.q = pr.q[:1].expand(52, 8, 128)  # one query for all tokens, and one for all heads too
    pr.check(pr.run(a, q=pr.q[:1].cuda().expand(52, 8, 128)), what="a token's stride of 0")
    pr.q = pr.q[:, :1].expand(52, 8, 128)
    pr.check(pr.run(a, q=pr.q[:1, :1].cuda().expand(52, 8, 128)), what="strides of 0")
    pr.check(pr.run(a, q=pr.q[:, :1].contiguous().cuda().expand(52, 8, 128)), what="a head's stride of 0")
    check_status(a)


@fours
def test_steep_scores_and_rows_that_saw_nothing(four):
    a = attn()
    pr = Problem([200, 77], [50, 9], four=four, seed=165)
    pr.lse += 40.0
    pr.lse[:, 3] = -math.inf
    pr.lse[2] = math.inf
    w = pr.run(a, scale=1.0)
    check_status(a)
    assert torch.isfinite(w).all()
    share, tol = kv4_ref.column_sums(pr.q, pr.lse, pr.pool(), pr.table, pr.cu, pr.lens, 1.0)
    tol = [t.nan_to_num(0.0) for t in tol]
    kv4_ref.check_weights(w, pr.weights, pr.table, pr.lens, share, tol, 8 * 50)


@fours
def test_unused_rows_and_blocks_are_never_read(four):
    """NaN rows and infinite ones past a request's end."""
    a = attn()
    for D, page in ((128, 16), (64, 24)):
        pr = Problem([5, 33, 16], [3, 30, 1], D=D, page=page, four=four, seed=166)
        want = pr.run(a)
        used = {(int(pr.table[b, t // page]), t % page) for b in range(3) for t in range(int(pr.lens[b]))}
        for blk in range(pr.cache.shape[0]):
            for r in range(page):
                if (blk, r) not in used:
                    if four:
                        pr.scales.view(torch.uint8)[blk, :, :, r] = 0x7F
                    else:
                        pr.cache[blk, :, :, r] = math.nan if r % 2 else math.inf
        assert torch.equal(pr.run(a), want)
        check_status(a)


def test_an_infinite_key_is_masked_for_the_queries_before_it():
    """Values that a causal mask hides reach nothing: key 30's own query and later ones see it."""
    a = attn()
    pr = Problem([40], [40], Hq=2, Hkv=1, seed=167)
    pr.cache[int(pr.table[0, 1]), 0, 0, 14, 5] = math.nan
    w = pr.run(a).cpu()
    at = [(int(pr.table[0, s // 16]), 0, s % 16) for s in range(40)]
    assert math.isnan(w[at[30]]) and all(math.isfinite(w[at[s]]) for s in range(40) if s != 30)
    pr.q[31:, :] = 0.0  # and no other row's padding
    pr.cache[int(pr.table[0, 1]), 0, 0, 14, 5] = math.inf
    w = pr.run(a).cpu()
    assert all(math.isfinite(w[at[s]]) for s in range(40) if s != 30)


@fours
def test_bad_requests_and_blocks(four):
    a = attn()
    pr = Problem([60, 40, 30], [20, 9, 30], four=four, seed=168)
    for b, length in ((1, 8), (1, -1), (0, pr.table.shape[1] * 16 + 1)):
        lens = pr.lens.clone()
        lens[b] = length
        w = pr.run(a, lens=lens)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        pr.check(w, skip=(b,))
    for bad in ([0, 20, 1000, 59], [-3, 20, 29, 59], [0, 20, 5, 59]):
        pr.run(a, cu=torch.tensor(bad, dtype=torch.int32))
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    want = pr.run(a).cpu()
    for bad in (-1, pr.cache.shape[0], 2 ** 31 - 1):
        table = pr.table.clone()
        table[0, 0] = bad
        w = pr.run(a, table=table).cpu()
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        blk = int(pr.table[0, 0])
        rest = torch.arange(w.shape[0]) != blk
        assert torch.equal(w[rest], want[rest]) and torch.equal(w[blk], pr.weights[blk])
    check_status(a)


@fours
@pytest.mark.parametrize("Hq,new", [(8, 20), (8, 1), (2, 600), (130, 3)], ids=["prompts", "step", "ranges", "fallback"])
def test_requests_that_share_blocks_add_up(Hq, new, four):
    a = attn()
    pr = Problem([700, 650, 900], [new, new, new], Hq=Hq, Hkv=1, D=64, four=four, seed=183)
    for b in (1, 2):
        pr.table[b, :30] = pr.table[0, :30]  # the same first 480 keys
    w = pr.run(a)
    check_status(a)
    pr.check(w)


def test_no_tokens_launch_nothing():
    a = attn()
    pr = Problem([5, 3], [0, 0], seed=169)
    assert torch.equal(pr.run(a).cpu(), pr.weights)
    assert a.last_launch_info()[2] == 0


@fours
def test_graph_on_a_side_stream(four):
    a = attn()
    pr = Problem([700, 90], [1, 65], four=four, seed=170)
    want = pr.run(a)
    dev = [t.cuda() for t in (pr.q, pr.lse, pr.cache, pr.table, pr.cu, pr.lens, pr.weights)]
    q, lse, cache, table, cu, lens, before = dev
    scales, factors = (pr.scales.cuda(), pr.factors.cuda()) if four else (None, None)
    w = before.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w.copy_(before)
        if four:
            a.attn_weights_paged_e2m1(q, lse, cache, scales, table, cu, lens, w, factors=factors)
        else:
            a.attn_weights_paged(q, lse, cache, table, cu, lens, w)
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert torch.equal(w, want)
    check_status(a)


@fours
def test_two_streams_at_once_with_ranges(four):
    """Prompts whose queries are cut into ranges, captured and eager, on two streams: each call's
    sums pass through a workspace of its own."""
    a = attn()
    problems = [Problem([1500, 40], [1500, 3], Hq=4, D=64, four=four, seed=s) for s in (191, 192)]
    want = [pr.run(a) for pr in problems]
    torch.cuda.synchronize()
    streams, graphs, held = [torch.cuda.Stream(), torch.cuda.Stream()], [], []

    def call(pr, dev, w):
        q, lse, cache, table, cu, lens, scales, factors = dev
        if four:
            a.attn_weights_paged_e2m1(q, lse, cache, scales, table, cu, lens, w, factors=factors)
        else:
            a.attn_weights_paged(q, lse, cache, table, cu, lens, w)

    for s, pr in zip(streams, problems):
        dev = [None if t is None else t.cuda() for t in (pr.q, pr.lse, pr.cache, pr.table, pr.cu, pr.lens, pr.scales, pr.factors)]
        before, w = pr.weights.cuda(), pr.weights.cuda()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            w.copy_(before)
            call(pr, dev, w)
        graphs.append(g)
        held.append((dev, before, w))
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    eager = []
    for s, pr, (dev, before, w) in zip(streams, problems, held):
        with torch.cuda.stream(s):
            e = before.clone()
            call(pr, dev, e)
            eager.append(e)
    torch.cuda.synchronize()
    for w, e, (_, _, g) in zip(want, eager, held):
        assert torch.equal(e, w) and torch.equal(g, w)
    check_status(a)


@fours
def test_a_step_of_many_requests_some_long(four):
    """More runs of keys to a request than blocks for it; and a table far wider than any request."""
    a = attn()
    lens = [(13 * i) % 40 for i in range(400)]
    lens[7], lens[399] = 2500, 2049
    pr = Problem(lens, [min(1, n) for n in lens], Hq=8, Hkv=8, D=64, page=64, four=four, seed=184)
    w = pr.run(a)
    check_status(a)
    pr.check(w)
    assert torch.equal(pr.run(a, table=torch.nn.functional.pad(pr.table, (0, 3000), value=-3)), w)
    check_status(a)


@fours
def test_many_requests(four):
    """5000 requests of which few have queries, found 32 at a time."""
    a = attn()
    B = 5000
    lens = [1 + (i * 7) % 40 for i in range(B)]
    new = [0] * B
    for i in (0, 31, 32, 2999, 4999):
        new[i] = min(3, lens[i])
    pr = Problem(lens, new, Hq=2, Hkv=1, D=64, four=four, seed=193)
    pr.check(pr.run(a))
    check_status(a)
    pr.lens[4998] = -1
    pr.run(a)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT


@fours
def test_a_request_that_is_not_valid_between_long_ones(four):
    a = attn()
    pr = Problem([800, 700, 900], [600, 600, 600], Hq=2, Hkv=1, D=64, four=four, seed=194)
    lens = pr.lens.clone()
    lens[1] = 599
    pr.check(pr.run(a, lens=lens), skip=(1,))
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
