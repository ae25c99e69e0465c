"""Eviction by accumulated weight against a slot-by-slot form, bit for bit."""
import math

import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu


class Problem:
    def __init__(self, lens, Hkv=2, D=128, page=16, dtype=torch.bfloat16, four=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.table, blocks = kv_ref.random_table(self.lens, page, g)
        if four:
            self.pools = list(kv4_ref.random_pool(blocks, Hkv, page, D, g))
        else:
            self.pools = [torch.randint(-2 ** 15, 2 ** 15, (blocks, 2, Hkv, page, D), generator=g).to(torch.int16).view(dtype)]
        self.weights = torch.exp(3 * torch.randn(blocks, Hkv, page, generator=g))
        self.weights *= torch.rand(blocks, Hkv, page, generator=g) > 0.2  # ties at 0
        self.four = four

    def run(self, a, keep, recent, table=None, lens=None, **kw):
        pools, w = [p.cuda() for p in self.pools], self.weights.cuda()
        t, n = (self.table if table is None else table).cuda(), (self.lens if lens is None else lens).cuda()
        call = a.attn_evict_paged_e2m1 if self.four else a.attn_evict_paged
        new, kept = call(*pools, w, t, n, keep, recent, **kw)
        return pools, w, new, kept

    def check(self, a, keep, recent):
        got = self.run(a, keep, recent)
        check_status(a)
        want = kv4_ref.evict([_bits(p) for p in self.pools], self.weights, self.table, self.lens, keep, recent)
        for x, y in zip(got[0], want[0]):
            assert torch.equal(_bits(x.cpu()), y), "rows"
        assert torch.equal(got[2].cpu(), want[2]) and torch.equal(got[3].cpu(), want[3])
        assert torch.equal(got[1].cpu().view(torch.int32), want[1].view(torch.int32)), "weights"
        again = self.run(a, keep, recent, want_kept=False)
        assert again[3] is None and torch.equal(again[1].view(torch.int32), got[1].view(torch.int32))
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(again[0], got[0]))


def _bits(t):
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.uint8)


fours = pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])


@fours
@pytest.mark.parametrize("lens,keep,recent,kw", [
    ([1], 1, 0, {}),
    ([2], 1, 0, {}),
    ([2], 1, 1, {}),
    ([17, 0, 16, 15, 33], 16, 4, {}),
    ([100, 37], 36, 36, {}),                                  # the last 36 and nothing else
    ([100, 37], 36, 0, {}),
    ([100, 5], 99, 7, dict(D=64)),                            # one goes
    ([300, 40, 299], 50, 10, dict(page=5, Hkv=3)),
    ([90, 70], 33, 1, dict(page=1, D=64, dtype=torch.float16)),
    ([520, 513, 511], 200, 3, dict(page=24, Hkv=1)),
    ([1000], 700, 100, dict(page=256, D=64)),
    ([60, 61], 400, 20, {}),                                  # nobody is that long
    ([30, 20], 10 ** 5, 20, {}),
    ([9000, 8193], 4100, 512, dict(Hkv=1)),
    ([30000, 24577, 24576], 2000, 300, dict(Hkv=1, D=64, page=64)),  # more than are held in shared memory, and as many
    ([70] * 40, 20, 5, dict(Hkv=8)),
])
def test_matches_slot_by_slot(lens, keep, recent, kw, four):
    a = attn()
    Problem(lens, **kw, four=four, seed=171).check(a, keep, recent)


@fours
@pytest.mark.parametrize("kind", ["equal", "zeros of both signs", "nan", "infinities", "negative", "close", "one digit"])
def test_weights_of_all_kinds(kind, four):
    a = attn()
    pr = Problem([400, 130], four=four, page=16, seed=172)
    g = torch.Generator().manual_seed(173)
    w = pr.weights
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zeros of both signs":
        w[:] = torch.where(torch.rand(w.shape, generator=g) > 0.5, 0.0, -0.0)
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g) > 0.3] = math.nan
        w.view(torch.int32)[:, 0, ::3] |= -2 ** 31
    elif kind == "infinities":
        w[torch.rand(w.shape, generator=g) > 0.5] = math.inf
        w[torch.rand(w.shape, generator=g) > 0.7] = -math.inf
    elif kind == "negative":
        w *= -1
    elif kind == "close":
        w.view(torch.int32)[:] = torch.randint(0x3f800000, 0x3f800040, w.shape, generator=g, dtype=torch.int32)
    else:
        w.view(torch.int32)[:] = torch.randint(0, 4, w.shape, generator=g, dtype=torch.int32) << 21
    for keep, recent in ((100, 10), (129, 0), (77, 77)):
        pr.check(a, keep, recent)


@fours
@pytest.mark.parametrize("lens,keep,recent,kw", [
    ([2049], 1000, 100, dict(Hkv=1)),
    ([2175, 2177], 2048, 2048, dict(Hkv=1, D=64, page=1)),
    ([5000, 0, 1300], 1290, 0, dict(Hkv=1, page=5, D=64)),
    ([16385], 16384, 5, dict(Hkv=1, page=64)),
    ([17000], 8200, 8199, dict(Hkv=1, page=1, dtype=torch.float16)),
    ([20000, 300, 9001], 5000, 1, dict(Hkv=2, page=24)),
    ([16000], 15000, 3, dict(Hkv=3, D=64)),
    ([200001], 3000, 700, dict(Hkv=1, D=64, page=256)),
])
def test_few_long_ones(lens, keep, recent, kw, four):
    a = attn()
    Problem(lens, **kw, four=four, seed=178).check(a, keep, recent)


@fours
@pytest.mark.parametrize("kind", ["equal", "nan in one place", "a thousand of a digit", "last few", "one digit"])
def test_few_long_ones_of_all_kinds(kind, four):
    a = attn()
    pr = Problem([20000], Hkv=1, four=four, page=16, seed=179)
    g = torch.Generator().manual_seed(180)
    w = pr.weights
    at = lambda slot: (int(pr.table[0, slot // 16]), 0, slot % 16)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "nan in one place":
        w[at(13001)] = math.nan
    elif kind == "a thousand of a digit":  # and those close by, so that the second digit decides
        w[:] = 4 * torch.rand(w.shape, generator=g)
        for i in range(1100):
            w[at(18 * i)] = 1.0 + i * 2.0 ** -14
    elif kind == "last few":
        w[:] = 0
        for slot in range(15000, 15050):
            w[at(slot)] = slot % 7
    else:
        w.view(torch.int32)[:] = torch.randint(0, 4, w.shape, generator=g, dtype=torch.int32) << 21
    for keep, recent in ((10000, 10), (15000, 0), (6000, 5990), (19999, 1)):
        pr.check(a, keep, recent)


@fours
@pytest.mark.parametrize("lens,keep,recent", [([300, 77, 129], 65, 3), ([5000], 2001, 100)])
def test_weights_at_any_place(lens, keep, recent, four):
    """Weights that four floats at a time could not be read from."""
    a = attn()
    pr = Problem(lens, Hkv=1, D=64, four=four, seed=185)
    pools, t, n = [p.cuda() for p in pr.pools], pr.table.cuda(), pr.lens.cuda()
    w = torch.empty(pr.weights.numel() + 1, device="cuda")[1:].view(pr.weights.shape)
    w.copy_(pr.weights)
    call = a.attn_evict_paged_e2m1 if four else a.attn_evict_paged
    new, kept = call(*pools, w, t, n, keep, recent)
    check_status(a)
    want = pr.run(a, keep, recent)
    assert torch.equal(w.view(torch.int32), want[1].view(torch.int32))
    assert torch.equal(new, want[2]) and torch.equal(kept, want[3])
    assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(pools, want[0]))


@fours
def test_bad_blocks_of_a_long_one(four):
    a = attn()
    pr = Problem([9000], Hkv=1, four=four, seed=181)
    for bad in (-1, pr.weights.shape[0]):
        table = pr.table.clone()
        table[0, 100] = table[0, 400] = bad
        got = pr.run(a, 4000, 50, table=table)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        kept = got[3].cpu()[0, 0].long()
        assert int(got[2][0]) == 4000 and torch.equal(kept[-50:], torch.arange(8950, 9000))
        assert bool((kept[1:] > kept[:-1]).all())
        slots = torch.arange(9000)
        w = pr.weights[table[0].clamp(0, pr.weights.shape[0] - 1).long()[slots // 16], 0, slots % 16].clone()
        w[(slots // 16 == 100) | (slots // 16 == 400)] = math.nan
        w = w.tolist()
        heaviest = sorted(range(8950), key=lambda i: (math.isnan(w[i]), 0.0 if math.isnan(w[i]) else -w[i], i))[:3950]
        assert kept[:-50].tolist() == sorted(heaviest)
    check_status(a)


@fours
def test_two_graphs_at_once_of_long_ones(four):
    """Captured on two streams without a list of what is kept (a workspace each), replayed side by side."""
    a = attn()
    runs = []
    for seed, lens, Hkv in ((186, [9000], 2), (187, [6000, 30, 4500], 1)):
        pr = Problem(lens, Hkv=Hkv, D=64, four=four, seed=seed)
        want = pr.run(a, 2500, 70)
        pools, w, t, n = [p.cuda() for p in pr.pools], pr.weights.cuda(), pr.table.cuda(), pr.lens.cuda()
        start = [p.clone() for p in pools], w.clone()
        new = torch.empty(len(lens), dtype=torch.int32, device="cuda")
        call = a.attn_evict_paged_e2m1 if four else a.attn_evict_paged
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for p, s in zip(pools, start[0]):
                p.copy_(s)
            w.copy_(start[1])
            call(*pools, w, t, n, 2500, 70, new_lens=new, want_kept=False)
        runs.append((graph, side, pools, w, new, want, start, t, n))
    for _ in range(5):
        for graph, side, *_ in runs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    check_status(a)
    for _, _, pools, w, new, want, *_ in runs:
        assert torch.equal(new, want[2]) and torch.equal(w.view(torch.int32), want[1].view(torch.int32))
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(pools, want[0]))


@fours
def test_evicted_again_and_again(four):
    """Each eviction's result is the next one's input; pages past the kept keys are free."""
    a = attn()
    pr = Problem([500, 260, 31], four=four, seed=174)
    for keep, recent in ((250, 40), (90, 40), (89, 0), (16, 8)):
        pools, w, new, _ = pr.run(a, keep, recent)
        pr.check(a, keep, recent)
        pr.pools, pr.weights, pr.lens = [p.cpu() for p in pools], w.cpu(), new.cpu()
        pr.table = pr.table[:, :max(1, -(-int(pr.lens.max()) // 16))].contiguous()
    check_status(a)


@fours
def test_bad_lengths_and_blocks(four):
    a = attn()
    pr = Problem([60, 40], four=four, seed=175)
    for length in (-1, pr.table.shape[1] * 16 + 1):
        lens = pr.lens.clone()
        lens[1] = length
        got = pr.run(a, 20, 5, lens=lens, table=pr.table.clamp(min=0))
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        assert int(got[2][0]) == 20
    for bad in (-1, pr.weights.shape[0], 2 ** 31 - 1):
        table = pr.table.clone()
        table[0, 1] = bad
        got = pr.run(a, 20, 5, table=table)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        mine = torch.zeros(pr.weights.shape[0], dtype=torch.bool)
        mine[pr.table[pr.table >= 0].long()] = True
        mine[int(pr.table[0, 1])] = False
        for x, y in zip(got[0], pr.pools):
            assert torch.equal(_bits(x.cpu())[~mine], _bits(y)[~mine])
        # The other request is whole.
        want = kv4_ref.evict([_bits(p) for p in pr.pools], pr.weights, pr.table, pr.lens, 20, 5)
        own = pr.table[1, :3].long()
        assert all(torch.equal(_bits(x.cpu())[own], y[own]) for x, y in zip(got[0], want[0]))
        assert torch.equal(got[3].cpu()[1], want[3][1])
    check_status(a)


def test_refusals():
    a = attn()
    pr = Problem([60, 40], seed=176)
    cache, w, t, n = pr.pools[0].cuda(), pr.weights.cuda(), pr.table.cuda(), pr.lens.cuda()
    for keep, recent in ((0, 0), (5, 6), (5, -1), (2 ** 31, 0)):
        with pytest.raises(ValueError):
            a.attn_evict_paged(cache, w, t, n, keep, recent)
    with pytest.raises(a.AttnError, match="seq_lens"):
        a.attn_evict_paged(cache, w, t, n, 5, 1, new_lens=n)
    with pytest.raises(ValueError, match="weights"):
        a.attn_evict_paged(cache, w[:, :1], t, n, 5, 1)
    with pytest.raises(ValueError, match="kept"):
        a.attn_evict_paged(cache, w, t, n, 5, 1, kept=torch.empty(2, 2, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="bf16 or fp16"):
        a.attn_evict_paged(cache.view(torch.uint8), w, t, n, 5, 1)
    with pytest.raises(ValueError, match="scales"):
        a.attn_evict_paged_e2m1(cache.view(torch.uint8)[..., :64].contiguous(), None, w, t, n, 5, 1)


@fours
def test_outputs_of_the_caller_and_graph(four):
    a = attn()
    pr = Problem([700, 90, 300], Hkv=4, four=four, seed=177)
    want = pr.run(a, 64, 20)
    pools, w = [p.cuda() for p in pr.pools], pr.weights.cuda()
    t, n = pr.table.cuda(), pr.lens.cuda()
    start = [p.clone() for p in pools], w.clone()
    new = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    kept = torch.full((3, 4, 64), 9, dtype=torch.int32, device="cuda")
    call = a.attn_evict_paged_e2m1 if four else a.attn_evict_paged
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for p, s in zip(pools, start[0]):
            p.copy_(s)
        w.copy_(start[1])
        got = call(*pools, w, t, n, 64, 20, new_lens=new, kept=kept)
    assert got[0] is new or got[0].data_ptr() == new.data_ptr()
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert torch.equal(new, want[2]) and torch.equal(kept, want[3])
        assert torch.equal(w.view(torch.int32), want[1].view(torch.int32))
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(pools, want[0]))
    check_status(a)
