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
