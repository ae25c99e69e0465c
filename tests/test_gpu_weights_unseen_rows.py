"""Query rows whose log-sum-exp is -inf add nothing, whatever is in them: by the kernel that
streams the keys and by the one on tiles alike."""
import math

import pytest
import torch

from gpu_util import attn, check_status
from test_gpu_weights import Problem

pytestmark = pytest.mark.gpu

fours = pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])
# Steps, and groups above a tile's rows, stream; the others go by tiles.
SHAPES = {
    "step": dict(lens=[300, 77, 40], new=[1, 1, 1], Hq=8, Hkv=2),
    "wide": dict(lens=[200, 90], new=[3, 2], Hq=130, Hkv=1, D=64),
    "window": dict(lens=[700, 256, 90], new=[64, 33, 5], Hq=8, Hkv=2),
    "prompt": dict(lens=[1300], new=[1300], Hq=4, Hkv=2, D=64),  # cut into ranges
    "odd": dict(lens=[500, 130], new=[70, 17], Hq=7, Hkv=1, page=24),
}


def marked(pr, low):
    """A third of the rows of lse, and all of a token's."""
    g = torch.Generator().manual_seed(221)
    out = torch.rand(pr.lse.shape, generator=g) < 1 / 3
    out[:, pr.lse.shape[1] // 2] = True
    pr.lse[out] = low
    return out.t()


@fours
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.float32).min], ids=["inf", "lowest"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_that_saw_nothing_may_hold_anything(shape, low, four):
    a = attn()
    pr = Problem(**SHAPES[shape], four=four, seed=222)
    out = marked(pr, low)
    pr.q[out] = 0.0
    want = pr.run(a)
    check_status(a)
    assert torch.isfinite(want).all()
    pr.lse[pr.lse == low] = -math.inf
    pr.check(want)
    for value in (math.nan, math.inf, -math.inf):
        pr.q[out] = value
        assert torch.equal(pr.run(a), want), value
    pr.q[out] = 0.0
    pr.lse[out.t()] = low
    assert torch.equal(pr.run(a), want)
    check_status(a)


@fours
@pytest.mark.parametrize("shape", SHAPES)
def test_a_request_that_saw_nothing_over_keys_that_are_not_numbers(shape, four):
    a = attn()
    pr = Problem(**SHAPES[shape], four=four, seed=223)
    pr.lse[:, : int(pr.cu[1])] = -math.inf
    blocks = pr.table[0].long()[: -(-int(pr.lens[0]) // pr.cache.shape[3])]
    if four:
        pr.scales.view(torch.uint8)[blocks] = 0x7F
    else:
        pr.cache[blocks] = math.inf
    w = pr.run(a).cpu()
    check_status(a)
    assert torch.equal(w[blocks], pr.weights[blocks])
    assert torch.isfinite(w).all()


@fours
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_that_count_are_not_hidden(shape, four):
    """NaN in a row's scores or in its log-sum-exp reaches the keys it sees, by both kernels; +inf
    there leaves them as they were."""
    a = attn()
    pr = Problem(**SHAPES[shape], four=four, seed=224)
    page, n = pr.cache.shape[3], int(pr.lens[0])
    token = int(pr.cu[1]) - 1  # sees all of the first request
    slots = torch.arange(n)
    at = pr.table[0, slots // page].long(), 0, slots % page
    keep = pr.q.clone(), pr.lse.clone()
    pr.q[token, 0] = math.nan
    assert pr.run(a).cpu()[at].isnan().all()
    pr.q, pr.lse[0, token] = keep[0], math.nan
    assert pr.run(a).cpu()[at].isnan().all()
    pr.lse = keep[1]
    pr.lse[:, : int(pr.cu[1])] = math.inf
    assert torch.equal(pr.run(a).cpu()[at], pr.weights[at])
    check_status(a)
