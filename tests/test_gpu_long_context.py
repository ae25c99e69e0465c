"""The 4-bit cache and eviction as a serving program uses them: prompts are appended and
attended over, their last tokens' weights added up, the cache cut back; then tokens are
decoded with their weights added up, and it is cut back again."""
import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE = 8, 2, 128, 16


@pytest.mark.parametrize("four", [False, True], ids=["16bit", "4bit"])
def test_prompt_evict_decode_evict(four):
    a = attn()
    g = torch.Generator().manual_seed(181)
    prompts, steps, window, keep, recent = [150, 40, 330], 24, 16, 64, 20
    B, total = len(prompts), sum(prompts)
    x = torch.randn(total, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    rotation = a.Rotation.make(D)
    table, blocks = kv_ref.random_table([n + steps for n in prompts], PAGE, g)
    table = table.cuda()
    factors = torch.tensor([[0.5, 0.25], [0.125, 0.3]], device="cuda") if four else None
    if four:
        cache = torch.zeros(blocks, 2, Hkv, PAGE, D // 2, dtype=torch.uint8, device="cuda")
        scales = torch.ones(blocks, 2, Hkv, PAGE, D // 16, device="cuda").to(torch.float8_e4m3fn)
    else:
        cache, scales = torch.zeros(blocks, 2, Hkv, PAGE, D, dtype=torch.bfloat16, device="cuda"), None
    weights = torch.zeros(blocks, Hkv, PAGE, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def append(x, cu, lens, **kw):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if four:
            return a.attn_append_paged_e2m1(k, v, cache, scales, table, cu, lens, rotation=rotation, q=q,
                                            factors=factors, **kw)
        return a.attn_append_paged(k, v, cache, table, cu, lens, rotation=rotation, q=q, **kw)

    def pool():
        return kv4_ref.held(cache.cpu(), scales.cpu(), factors.cpu()) if four else cache.cpu().double()

    def evict():
        before = weights.cpu(), [cache.cpu()] + ([scales.cpu()] if four else [])
        bits = [p.view(torch.int16) if p.element_size() == 2 else p.view(torch.uint8) for p in before[1]]
        want = kv4_ref.evict(bits, before[0], table.cpu(), lens.cpu(), keep, recent)
        new, kept = (a.attn_evict_paged_e2m1(cache, scales, weights, table, lens, keep, recent) if four else
                     a.attn_evict_paged(cache, weights, table, lens, keep, recent))
        check_status(a)
        assert torch.equal(new.cpu(), want[2]) and torch.equal(kept.cpu(), want[3]) and torch.equal(weights.cpu(), want[1])
        now = [cache.cpu()] + ([scales.cpu()] if four else [])
        for p, w in zip(now, want[0]):
            assert torch.equal(p.view(torch.int16) if p.element_size() == 2 else p.view(torch.uint8), w)
        return new

    cu, lens = ints([0] + torch.tensor(prompts).cumsum(0).tolist()), ints(prompts)
    kout = torch.empty(total, Hkv, D, dtype=torch.bfloat16, device="cuda")
    q, kr = append(x, cu, lens, out_k=kout)
    o, lse = a.attn_fwd_varlen(q.contiguous(), kr, x[:, Hq + Hkv:].contiguous(), cu, cu, causal=True)
    # The last tokens of each prompt vote.
    last = torch.cat([torch.arange(int(cu[b + 1]) - window, int(cu[b + 1])) for b in range(B)]).cuda()
    votes, vote_lse, vote_cu = q[last], lse[:, last], ints([window * b for b in range(B + 1)])
    if four:
        a.attn_weights_paged_e2m1(votes, vote_lse, cache, scales, table, vote_cu, lens, weights, factors=factors)
    else:
        a.attn_weights_paged(votes, vote_lse, cache, table, vote_cu, lens, weights)
    check_status(a)
    share, tol = kv4_ref.column_sums(votes.cpu(), vote_lse.cpu(), pool(), table.cpu(), vote_cu.cpu(), lens.cpu())
    kv4_ref.check_weights(weights, torch.zeros(weights.shape), table.cpu(), lens.cpu(), share, tol, window * Hq)
    if not four:  # every query's weights over the keys it sees add up to 1
        assert abs(float(weights.double().sum()) - window * Hq * B) < 1e-3 * window * Hq * B
    lens = evict()
    one = ints(list(range(B + 1)))
    for i in range(steps):
        lens = lens + 1
        x = torch.randn(B, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
        q, _ = append(x, one, lens, positions=ints([n + i for n in prompts]))
        q = q.unsqueeze(2).contiguous()
        before = weights.cpu()
        if four:
            o, lse = a.attn_fwd_decode_paged_e2m1(q, cache, scales, table, lens, factors=factors, weights=weights)
        else:
            o, lse = a.attn_fwd_decode_paged(q, cache, table, lens)
            a.attn_weights_paged(q[:, :, 0], lse.t(), cache, table, one, lens, weights)
        check_status(a)
        ref = kv4_ref.decode(q.cpu(), pool(), table.cpu(), lens.cpu())
        if four:
            kv4_ref.check_decode(o, lse, ref, int(lens.max()), f"step {i}")
        kv4_ref.check_weights(weights, before, table.cpu(), lens.cpu(), ref[4],
                              [t + 1e-4 * s for t, s in zip(ref[5], ref[4])], int(lens.max()), f"step {i}")
    assert int(evict().max()) == keep
