"""Accumulated attention weights of requests whose offsets are out of order and whose queries
are cut into ranges: each has its partial sums within the workspace, or is left out."""
import pytest
import torch

import kv4_ref
from gpu_util import attn, check_status
from test_gpu_weights import Problem

pytestmark = pytest.mark.gpu

fours = pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])


@fours
@pytest.mark.parametrize("total,cu,left_out", [
    (1024, [0, 1024, 0, 1024, 0, 1024], (1, 3, 4)),  # places for two of three
    (600, [0, 600, 0, 600], (1, 2)),
    (600, [0, 500, 0, 512, 0, 600, 20, 25], (1, 3, 5)),  # without ranges: any order
    (1500, [0, 700, 100, 1300, 200, 240, 0, 1500, 1500], (1, 3, 5, 6)),
    (600, [0, 600] * 40 + [0, 5], tuple(i for i in range(81) if i % 2 or 0 < i < 80)),
], ids=["all", "two", "short", "several", "many"])
def test_ranges_of_offsets_out_of_order(total, cu, left_out, four):
    a = attn()
    B = len(cu) - 1
    sizes = [max(0, y - x) for x, y in zip(cu, cu[1:])]
    lens = [max(n, total if b in left_out else 0) + 7 * b for b, n in enumerate(sizes)]
    pr = Problem(lens, sizes, Hq=4, Hkv=2, D=64, four=four, seed=201)
    pr.q, pr.lse = pr.q[:total], pr.lse[:, :total].clamp(min=3.0)
    bad = torch.tensor(cu, dtype=torch.int32)
    want = pr.weights.clone()
    for b in range(B):
        if b in left_out:
            continue
        own = slice(cu[b], cu[b + 1])
        share, tol = kv4_ref.column_sums(pr.q[own], pr.lse[:, own], pr.pool(), pr.table[b:b + 1],
                                         torch.tensor([0, sizes[b]]), pr.lens[b:b + 1])
        kv4_ref.check_weights(one_request(a, pr, b, own), pr.weights * 0, pr.table[b:b + 1], pr.lens[b:b + 1], share, tol, sizes[b] * 4)
    w = pr.run(a, cu=bad)
    assert a.device_status() == a.ATTN_ERR_BAD_INPUT
    # Every request's blocks are its own: those of a request left out are as they were, the others'
    # as if it were alone.
    for b in range(B):
        blocks = pr.table[b].long()[: -(-lens[b] // 16)]
        if b in left_out:
            assert torch.equal(w.cpu()[blocks], want[blocks]), b
        else:
            alone = one_request(a, pr, b, slice(cu[b], cu[b + 1]), pr.weights)
            assert torch.equal(w.cpu()[blocks], alone.cpu()[blocks]), b
    check_status(a)


def one_request(a, pr, b, own, before=None):
    w = (pr.weights * 0 if before is None else before).cuda()
    args = (pr.table[b:b + 1].cuda(), torch.tensor([0, own.stop - own.start], dtype=torch.int32).cuda(), pr.lens[b:b + 1].cuda())
    q, lse = pr.q[own].cuda(), pr.lse[:, own].cuda()
    if pr.four:
        return a.attn_weights_paged_e2m1(q, lse, pr.cache.cuda(), pr.scales.cuda(), *args, w, factors=pr.factors.cuda())
    return a.attn_weights_paged(q, lse, pr.cache.cuda(), *args, w)
