"""The operators as a serving step uses them: a prompt is normalised, rotated,
appended and attended over; then tokens are appended one at a time and decoded
against the cache."""
import pytest
import torch

import kv_ref
import oracle
from gpu_util import TOL_LSE_BF16, TOL_O_BF16, attn, check_status, compare

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE = 8, 2, 128, 16


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("with_norm", [False, True], ids=["plain", "norm"])
def test_prompt_then_decode(e4m3, with_norm):
    a = attn()
    g = torch.Generator().manual_seed(61)
    prompts, steps = [37, 5, 64], 18
    B, total = len(prompts), sum(prompts)
    rows = [torch.randn(n + steps, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16) for n in prompts]
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    qw, kw = qw.to(torch.bfloat16), kw.to(torch.bfloat16)
    turns, _ = a.rope_turns(D)
    rotation, freq = a.Rotation(turns.cuda()), kv_ref.turns_to_radians(turns.tolist())
    table, blocks = kv_ref.random_table([n + steps for n in prompts], PAGE, g)
    table = table.cuda()
    shape = (blocks, 2, Hkv, PAGE, D)
    cache = torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    scales = torch.ones(blocks, 2, Hkv, device="cuda")

    # 64-bit history of every request: rotated keys and queries, values.
    def reference(b):
        x = rows[b].double()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if with_norm:
            q, k = kv_ref.norm(q, qw, 1e-6), kv_ref.norm(k, kw, 1e-6)
        pos = torch.arange(len(x))[:, None]
        return kv_ref.rotate(q, pos, freq)[0], kv_ref.rotate(k, pos, freq)[0], v

    refs = [reference(b) for b in range(B)]

    def append(x, cu, lens, out_k=None):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        r = rotation
        if with_norm:  # in place, rotation included: the append copies
            n = torch.diff(cu)
            pos = torch.cat([torch.arange(int(l) - int(c), int(l)) for l, c in zip(lens, n)]).to(torch.int32)
            a.attn_qk_norm_rope(q, k, qw.cuda(), kw.cuda(), pos.cuda(), rotation, out_q=q, out_k=k)
            r = None
        kw_ = dict(rotation=r, q=q, out_k=out_k)
        if e4m3:
            return a.attn_append_paged_e4m3(k, v, cache, scales, table, cu.cuda(), lens.cuda(), **kw_)
        return a.attn_append_paged(k, v, cache, table, cu.cuda(), lens.cuda(), **kw_)

    def check_cache(lens):
        """Every slot within its roundings of the history: one to bf16 where a row is normalised
        or held in 16 bits, one to e4m3 (2^-4), and under a step of e4m3's subnormals (2^-9 of
        the scale) for the roundings of rows that followed a growing scale."""
        held, sc = cache.cpu(), scales.cpu()
        for b in range(B):
            n = int(lens[b])
            kv = kv_ref.gather(held, table.cpu(), b, n).double().transpose(1, 2)
            want = torch.stack((refs[b][1][:n], refs[b][2][:n]))
            fp32 = kv_ref.ROTATION_ERROR + (kv_ref.norm_error(D) if with_norm else 0.0)
            # |a| + |b| of a pair is at most sqrt(2) times its radius, which is at most the sum of its
            # results' sizes.
            pair = want[0].abs() + want[0].roll(D // 2, dims=-1).abs()
            tol = torch.stack((fp32 * 1.5 * pair, torch.zeros_like(pair)))
            if not e4m3:
                tol = tol + 2.0 ** -8 * want.abs()
                tol[1] = 0.0  # values are copied
            else:
                kv = kv * kv_ref.gather_scales(sc, table.cpu(), b, n, PAGE).transpose(1, 2)[..., None]
                first = 2.0 ** -8 if with_norm else 0.0
                tol = tol + (2.0 ** -4 * (1 + first) + first) * want.abs()
                tol = tol + 2.0 ** -9 * kv_ref.gather_scales(sc, table.cpu(), b, n, PAGE).transpose(1, 2)[..., None]
            assert ((kv - want).abs() <= 1.001 * tol).all(), b

    cu = torch.tensor([0] + prompts).cumsum(0).to(torch.int32)
    x = torch.cat([r[:n] for r, n in zip(rows, prompts)]).cuda()
    kout = torch.empty(total, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = x[:, Hq + Hkv:].contiguous()
    q, kr = append(x, cu, torch.tensor(prompts, dtype=torch.int32), kout)
    q = q.contiguous()
    o, lse = a.attn_fwd_varlen(q, kr, v, cu.cuda(), cu.cuda(), causal=True)
    check_status(a)
    want, want_lse = oracle.attention_varlen_f64(q, kr, v, cu, cu, True)
    compare(o, lse, want, want_lse, TOL_O_BF16, TOL_LSE_BF16, "prompt")
    check_cache(prompts)
    one = torch.arange(B + 1, dtype=torch.int32)
    for i in range(steps):
        lens = torch.tensor([n + i + 1 for n in prompts], dtype=torch.int32)
        x = torch.stack([r[n + i] for r, n in zip(rows, prompts)]).cuda()
        q, _ = append(x, one, lens)
        q = q.unsqueeze(2).contiguous()
        if e4m3:
            o, lse = a.attn_fwd_decode_paged_e4m3(q, cache, scales, table, lens.cuda())
            ref = kv_ref.decode_e4m3(q.cpu(), cache.cpu(), scales.cpu(), table.cpu(), lens)
            kv_ref.check_decode(o, lse, ref, int(lens.max()), f"step {i}")
        else:
            o, lse = a.attn_fwd_decode_paged(q, cache, table, lens.cuda())
            want, want_lse = oracle.decode_paged_f64(q, cache, table, lens)
            compare(o[:, :, 0], lse, want, want_lse, TOL_O_BF16, TOL_LSE_BF16, f"step {i}")
        check_status(a)
        check_cache(lens.tolist())
        # The step's query is the history's, rounded once.
        for b in range(B):
            w = refs[b][0][prompts[b] + i]
            size = w.abs() + w.roll(D // 2, dims=-1).abs()
            kv_ref.check_rows(q[b, :, 0], w, 1.5 * size, kv_ref.ROTATION_ERROR + kv_ref.norm_error(D), "query")


@pytest.mark.parametrize("e4m3", [False, True], ids=["16bit", "e4m3"])
def test_decode_step_in_one_graph(e4m3):
    """A whole step captured, with copies and a clearing between the launches and a second stream
    that forks off and joins; replays on new inputs give an eager step's bits, also back to back."""
    a = attn()
    g = torch.Generator().manual_seed(62)
    B, steps = 3, 20
    lens0 = torch.tensor([5, 30, 17], dtype=torch.int32)
    table, blocks = kv_ref.random_table(lens0 + steps, PAGE, g)
    table = table.cuda()
    turns, _ = a.rope_turns(D)
    rotation = a.Rotation(turns.cuda())
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    inputs = [torch.randn(B, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(steps)]
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16

    def state():
        return {"x": torch.zeros_like(inputs[0]), "in": torch.zeros_like(inputs[0]), "lens": lens0.cuda(),
                "cache": torch.zeros(blocks, 2, Hkv, PAGE, D, device="cuda").to(kind),
                "scales": torch.ones(blocks, 2, Hkv, device="cuda"),
                "q": torch.empty(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda"),
                "o": torch.empty(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda"),
                "side": torch.empty(B, Hkv, D, dtype=torch.bfloat16, device="cuda")}

    def step(s, other):
        s["x"].copy_(s["in"])
        s["lens"].add_(1)
        s["o"].zero_()
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            # The same keys rotated apart, at the step's positions.
            a.attn_rope(s["x"][:, Hq:Hq + Hkv], None, s["lens"] - 1, rotation, out_q=s["side"])
        k, v = s["x"][:, Hq:Hq + Hkv], s["x"][:, Hq + Hkv:]
        kw = dict(rotation=rotation, q=s["x"][:, :Hq], out_q=s["q"][:, :, 0])
        if e4m3:
            a.attn_append_paged_e4m3(k, v, s["cache"], s["scales"], table, cu, s["lens"], **kw)
            a.attn_fwd_decode_paged_e4m3(s["q"], s["cache"], s["scales"], table, s["lens"], out=s["o"])
        else:
            a.attn_append_paged(k, v, s["cache"], table, cu, s["lens"], **kw)
            a.attn_fwd_decode_paged(s["q"], s["cache"], table, s["lens"], out=s["o"])
        here.wait_stream(other)
        # In place, after the join.
        a.attn_qk_norm_rope(s["o"][:, :, 0], s["side"], None, None, s["lens"], rotation, out_q=s["o"][:, :, 0],
                            out_k=s["side"])

    eager, captured, other = state(), state(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(captured, torch.cuda.Stream())
    for x in inputs:
        eager["in"].copy_(x)
        captured["in"].copy_(x)
        step(eager, other)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("o", "side", "q", "scales"):
            assert torch.equal(eager[name], captured[name]), name
        assert torch.equal(eager["cache"].view(torch.uint8), captured["cache"].view(torch.uint8))
    check_status(a)
    # Back to back, nothing waiting between.
    for s in (eager, captured):
        s["lens"].copy_(lens0)
    for _ in range(10):
        step(eager, other)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("o", "side", "q", "scales"):
        assert torch.equal(eager[name], captured[name]), name
    check_status(a)
