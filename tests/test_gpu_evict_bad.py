"""Eviction with lengths and block ids that are out of range: nothing that they name changes."""
import pytest
import torch

import kv4_ref
from gpu_util import attn, check_status
from test_gpu_evict import Problem, _bits

pytestmark = pytest.mark.gpu

fours = pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])


@fours
@pytest.mark.parametrize("lens,keep,kw", [([320, 320, 200], 50, dict(D=64)), ([9600, 9600], 4000, dict(Hkv=1, D=64))],
                         ids=["short", "clusters"])
def test_a_length_out_of_range_leaves_the_request_out(lens, keep, kw, four):
    """Its table is full of blocks of its own."""
    a = attn()
    pr = Problem(lens, **kw, four=four, seed=241)
    want = kv4_ref.evict([_bits(p) for p in pr.pools], pr.weights, pr.table, pr.lens, keep, 7)
    own = pr.table[1].long()
    for length in (lens[1] + 1, 2 ** 31 - 1, -1, -2 ** 31):
        n = pr.lens.clone()
        n[1] = length
        pools, w, new, kept = pr.run(a, keep, 7, lens=n)
        assert a.device_status() == a.ATTN_ERR_BAD_INPUT
        assert int(new[1]) == 0 and bool((kept[1] == -1).all())
        others = torch.ones(pr.weights.shape[0], dtype=torch.bool)
        others[own] = False
        for x, y, before in zip(pools, want[0], pr.pools):
            assert torch.equal(_bits(x.cpu())[own], _bits(before)[own])
            assert torch.equal(_bits(x.cpu())[others], y[others])
        assert torch.equal(w.cpu()[own], pr.weights[own]) and torch.equal(w.cpu()[others], want[1][others])
        for b in range(len(lens)):
            if b != 1:
                assert int(new[b]) == int(want[2][b]) and torch.equal(kept[b].cpu(), want[3][b])
    check_status(a)


@fours
@pytest.mark.parametrize("lens,keep,recent,bad", [
    ([320, 90], 100, 40, (2, 18, 19)),       # of the kept ones by their order, and of the last
    ([9600, 300], 4000, 300, (100, 598)),    # by clusters
], ids=["short", "clusters"])
def test_weights_stay_where_their_rows_stay(lens, keep, recent, bad, four):
    a = attn()
    pr = Problem(lens, Hkv=1, D=64, four=four, seed=242)
    table = pr.table.clone()
    for page, value in zip(bad, (-1, pr.weights.shape[0], 2 ** 31 - 1)):
        table[0, page] = value
    pools, w, new, kept = pr.run(a, keep, recent, table=table)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    assert int(new[0]) == keep
    want, rows = pr.weights.clone(), [_bits(p).clone() for p in pr.pools]
    at = lambda slot: (int(pr.table[0, slot // 16]), slot % 16)
    there = [slot // 16 not in bad for slot in range(lens[0])]
    for slot in range(keep, lens[0]):
        if there[slot]:
            want[at(slot)[0], 0, at(slot)[1]] = 0.0
    stayed = 0
    for i, slot in enumerate(kept[0, 0].tolist()):
        if not (there[slot] and there[i]):
            stayed += 1
            continue
        (to, row), (of, old) = at(i), at(slot)
        want[to, 0, row] = pr.weights[of, 0, old]
        for x, before in zip(rows, pr.pools):
            x[to, :, :, row] = _bits(before)[of, :, :, old]
    assert stayed > 16
    others = kv4_ref.evict([_bits(p) for p in pr.pools], pr.weights, pr.table, pr.lens, keep, recent)
    own = pr.table[1].long()[: -(-lens[1] // 16)]
    want[own] = others[1][own]
    assert torch.equal(w.cpu().view(torch.int32), want.view(torch.int32))
    for x, y, z in zip(pools, rows, others[0]):
        y[own] = z[own]
        assert torch.equal(_bits(x.cpu()), y)
    check_status(a)
