"""Cases of the rotary, norm, paged-append and 8-bit-cache decode operators.

Every case is one call of a serving program: rotate (and normalise) queries and
keys, append keys and values to the paged cache, or attend over the 8-bit cache.
`run` computes it in its plain form from elementary torch operations, or, where
`own` is set, through the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100


def listed():
    return [
        # One token of one sequence: a decode step's rotation, all launch latency.
        {"name": "rope_step", "op": "rope", "layout": "packed", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "inter": False, "scaling": "none", "far": 8192, "dtype": "bf16"},
        # A batch of training-length sequences in [B, H, T, D], adjacent pairs, half of the head rotated.
        {"name": "rope_batch_part", "op": "rope", "layout": "dense", "B": 8, "T": 1024, "Hq": 12, "Hkv": 12,
         "D": 64, "rot": 32, "inter": True, "scaling": "none", "far": 0, "dtype": "f16"},
        # float32 heads at far positions of a context lengthened by wavelength; an odd token count.
        {"name": "rope_far_f32", "op": "rope", "layout": "packed", "B": 1, "T": 4099, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "inter": False, "scaling": "wavelength", "far": 1000000, "dtype": "f32"},
        # A decode step of 64 requests, q and k sliced out of the fused projection.
        {"name": "norm_rope_step", "op": "norm_rope", "T": 64, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "inter": False, "scaling": "none", "far": 4096, "dtype": "bf16"},
        # A prompt of 8192 tokens, the long workload's length.
        {"name": "norm_rope_prompt", "op": "norm_rope", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "inter": False, "scaling": "wavelength", "far": 0, "dtype": "bf16"},
        # One new token for each of 64 requests against 16-token pages, q rotated with it.
        {"name": "append_step", "op": "append", "cache": "16", "B": 64, "new": 1, "past": 2048, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "rot": 128, "inter": False, "scaling": "none", "dtype": "bf16"},
        # Prompts of different lengths, some continuing a request that has tokens already.
        {"name": "append_prompts", "op": "append", "cache": "16", "B": 9, "new": 1900, "past": 300, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "rot": 128, "inter": False, "scaling": "none", "dtype": "bf16"},
        # The same step into the 8-bit cache: pages are partly filled, some scales grow.
        {"name": "append_e4m3_step", "op": "append", "cache": "e4m3", "B": 64, "new": 1, "past": 2048, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "rot": 128, "inter": False, "scaling": "none", "dtype": "bf16"},
        # And prompts into the 8-bit cache.
        {"name": "append_e4m3_prompts", "op": "append", "cache": "e4m3", "B": 9, "new": 1900, "past": 300, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "rot": 128, "inter": False, "scaling": "none", "dtype": "bf16"},
        # Few ragged requests, one query head per key head, the 64-wide head: the small end of decoding.
        {"name": "decode_e4m3_small", "op": "decode", "B": 3, "len": 777, "spread": 700, "Hq": 12, "Hkv": 12,
         "D": 64, "page": 16, "dtype": "f16"},
        # The decode workload's sizes: 64 requests of about 4096 cached tokens, four query heads a key head.
        {"name": "decode_e4m3", "op": "decode", "B": 64, "len": 4096, "spread": 0, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "dtype": "bf16"},
        # Eight query heads per key head, ragged lengths, larger pages.
        {"name": "decode_e4m3_gqa8", "op": "decode", "B": 32, "len": 3500, "spread": 1200, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "norm_rope", "append", "append", "decode", "decode"))
    D = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 5, 8, 12))
    hq = hkv * rng.choice((1, 2, 3, 4, 7, 8))
    hq = min(hq, hkv * max(1, 64 // hkv))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    rot = rng.choice((D, D, D // 2, D // 4, 2 * rng.randint(2, D // 2)))
    scaling = rng.choice(("none", "linear", "wavelength", "yarn"))
    inter = rng.random() < 0.4
    if op == "rope":
        layout = rng.choice(("packed", "dense"))
        B = 1 if layout == "packed" else rng.randint(1, 8)
        dtype = rng.choice((dtype, "f32"))
        T = _log(rng, 1, 8192 // B // (2 if dtype == "f32" else 1))
        return {"op": op, "layout": layout, "B": B, "T": T, "Hq": hq, "Hkv": hkv, "D": D, "rot": rot, "inter": inter,
                "scaling": scaling, "far": rng.choice((0, 5000, 1000000)), "dtype": dtype}
    if op == "norm_rope":
        dtype = rng.choice((dtype, "f32"))
        return {"op": op, "T": _log(rng, 1, 8192 // (2 if dtype == "f32" else 1)), "Hq": hq, "Hkv": hkv, "D": D, "rot": rot, "inter": inter,
                "scaling": scaling, "far": rng.choice((0, 5000, 1000000)), "dtype": dtype}
    if op == "append":
        B = _log(rng, 1, 96)
        return {"op": op, "cache": rng.choice(("16", "e4m3")), "B": B, "new": _log(rng, 1, 12288 // B),
                "past": rng.choice((0, 40, 700, 1500)), "Hq": hq, "Hkv": hkv, "D": D,
                "page": rng.choice((1, 8, 16, 16, 24, 64)), "rot": rot, "inter": inter, "scaling": scaling,
                "dtype": dtype}
    B = _log(rng, 1, 64)
    length = _log(rng, 1, min(16384, 1048576 // (B * hkv)))
    return {"op": op, "B": B, "len": length, "spread": rng.choice((0, length // 3, length - 1)), "Hq": hq,
            "Hkv": hkv, "D": D, "page": rng.choice((5, 16, 16, 32, 64)), "dtype": dtype}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _frequencies(rot, scaling):
    """Radians per position of each rotated pair and the factor of cos and sin."""
    inv = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [f / 4.0 for f in inv], 1.0
    if scaling == "wavelength":  # long waves are slowed eightfold, short ones kept, the rest between
        out = []
        for f in inv:
            part = (8192 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)
            part = min(1.0, max(0.0, part))
            out.append(f * part + f / 8.0 * (1.0 - part))
        return out, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = max(0, math.floor(pair(32.0))), min(rot - 1, math.ceil(pair(1.0)))
        out = []
        for i, f in enumerate(inv):
            slow = min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo)))
            out.append(f * (1.0 - slow) + f / 16.0 * slow)
        return out, 0.1 * math.log(16.0) + 1.0
    return inv, 1.0


def _rotation(case):
    """What a program keeps of its rotation: the frequencies, and the same as 2^-64 turns per position."""
    freq, magnitude = _frequencies(case["rot"], case["scaling"])
    turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in freq]
    turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    return {"freq": torch.tensor(freq, dtype=torch.float64, device="cuda"),
            "turns": torch.tensor(turns, dtype=torch.int64, device="cuda"),
            "inter": case["inter"], "magnitude": magnitude}


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(lens, most, page, cpu):
    """A block table over a pool that could hold `most` tokens for every request; unused entries are -1."""
    width = max(1, -(-most // page))
    pool, table, at = torch.randperm(len(lens) * width + 3, generator=cpu).tolist(), [], 0
    for n in lens:
        n = -(-n // page)
        table.append(pool[at:at + n] + [-1] * (width - n))
        at += n
    return _int32(table), len(pool)


def _codes(gen, shape):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * 96.0).clamp(
        -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    op, D, Hq, Hkv = case["op"], case["D"], case["Hq"], case["Hkv"]
    if op in ("rope", "norm_rope"):
        T = case["T"]
        s["rotation"] = _rotation(case)
        first = case["far"] - int(torch.randint(0, 64, (1,), generator=cpu)) if case["far"] else 0
        if op == "rope" and case["layout"] == "dense":
            s["q"] = _randn(gen, (case["B"], Hq, T, D), dtype)
            s["k"] = _randn(gen, (case["B"], Hkv, T, D), dtype)
            start = torch.arange(case["B"], device="cuda", dtype=torch.int32)[:, None] * 3
            s["pos"] = (start + torch.arange(T, device="cuda", dtype=torch.int32) + first).contiguous()
        else:
            qkv = _randn(gen, (T, Hq + 2 * Hkv, D), dtype)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
            s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32) + first
        if op == "norm_rope":
            s["qw"] = (1.0 + 0.2 * _randn(gen, (D,), torch.float32)).to(dtype)
            s["kw"] = (1.0 + 0.2 * _randn(gen, (D,), torch.float32)).to(dtype)
        return s
    if op == "append":
        B, page = case["B"], case["page"]
        spread, new = case["new"] // 2, [case["new"]] * B
        for b in range(0, B - 1, 2):  # prompts of different lengths, as many tokens in all
            more = int(torch.randint(-spread, spread + 1, (1,), generator=cpu))
            new[b], new[b + 1] = new[b] + more, new[b + 1] - more
        past = [int(torch.randint(0, case["past"] + 1, (1,), generator=cpu)) for _ in range(B)]
        lens = [n + p for n, p in zip(new, past)]
        s["table"], blocks = _pages(lens, case["new"] + spread + case["past"], page, cpu)
        s["lens"] = _int32(lens)
        s["cu"] = _int32([sum(new[:b]) for b in range(B + 1)])
        qkv = _randn(gen, (sum(new), Hq + 2 * Hkv, D), dtype)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["rotation"] = _rotation(case)
        shape = (blocks, 2, Hkv, page, D)
        if case["cache"] == "e4m3":
            s["cache"] = _codes(gen, shape)
            s["scales"] = torch.exp2(torch.randint(-9, -5, (blocks, 2, Hkv), generator=gen, device="cuda").float())
        else:
            s["cache"] = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
        return s
    B, page = case["B"], case["page"]
    lens = [case["len"] + int(torch.randint(-case["spread"], case["spread"] + 1, (1,), generator=cpu))
            for _ in range(B)]
    if case["spread"] and B > 1:
        lens[-1] = 0  # a request that has no tokens yet
    lens = [max(0, n) for n in lens]
    s["table"], blocks = _pages(lens, case["len"] + case["spread"], page, cpu)
    s["lens"] = _int32(lens)
    s["q"] = _randn(gen, (B, Hq, 1, D), dtype)
    s["cache"] = _codes(gen, (blocks, 2, Hkv, page, D))
    s["scales"] = torch.exp2(torch.randint(-8, -5, (blocks, 2, Hkv), generator=gen, device="cuda").float())
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _rotate(x, pos, rotation):
    """x float32 [..., D], pos broadcasting over x's leading dimensions."""
    h = rotation["freq"].shape[0]
    angle = pos[..., None].double() * rotation["freq"]  # 64 bits: far positions
    c = (angle.cos() * rotation["magnitude"]).float()
    s = (angle.sin() * rotation["magnitude"]).float()
    if rotation["inter"]:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        front = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        front = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((front, x[..., 2 * h:]), dim=-1)


def _norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w.float()


def _power_of_two_at_least(x):
    """The smallest power of two >= x (float64, x >= 0), not below MIN_SCALE."""
    mantissa, exponent = torch.frexp(x)
    exponent = torch.where(mantissa == 0.5, exponent - 1, exponent)
    return torch.ldexp(torch.ones_like(x), exponent).clamp(min=MIN_SCALE).float()


def _slots(s):
    """Request, block and row in the block of every new token."""
    page = s["case"]["page"]
    token = torch.arange(s["k"].shape[0], device="cuda", dtype=torch.int32)
    request = torch.searchsorted(s["cu"][1:], token, right=True)
    slot = s["lens"][request] - s["cu"][1:][request] + token
    return slot, s["table"][request, (slot // page).long()].long(), (slot % page).long()


def _append(s):
    dtype = DTYPES[s["case"]["dtype"]]
    slot, block, row = _slots(s)
    q = _rotate(s["q"].float(), slot[:, None], s["rotation"]).to(dtype)
    k = _rotate(s["k"].float(), slot[:, None], s["rotation"])
    if s["case"]["cache"] == "16":
        s["cache"][block, 0, :, row] = k.to(dtype)
        s["cache"][block, 1, :, row] = s["v"]
        return {"q": q, "cache": s["cache"]}
    page, codes, scales = s["case"]["page"], s["cache"].view(torch.uint8), s["scales"]
    raw = torch.stack((s["k"], s["v"]), dim=1).float().abs().amax(dim=-1)
    largest = torch.zeros_like(scales).flatten(1)
    largest = largest.scatter_reduce(0, block[:, None].expand(-1, largest.shape[1]), raw.flatten(1), "amax")
    largest = largest.view_as(scales)
    limit = torch.tensor([E4M3_MAX / (math.sqrt(2.0) * s["rotation"]["magnitude"]), E4M3_MAX], device="cuda")
    need = _power_of_two_at_least(largest.double() / limit[:, None].double())
    # The first block of a request may hold older rows: its scale only grows, and they follow it.
    start = s["lens"] - (s["cu"][1:] - s["cu"][:-1])
    head = torch.gather(s["table"], 1, (start // page).long()[:, None])[:, 0].long()
    older = torch.arange(page, device="cuda") < (start % page)[:, None]
    before = scales[head]
    after = torch.where(older[:, :1, None], torch.maximum(before, need[head]), need[head])
    need[head] = after
    held = codes[head]
    moved = held.view(torch.float8_e4m3fn).float() * (before / after)[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[head] = torch.where(older[:, None, None, :, None], moved, held)
    scales[block] = need[block]
    rows = torch.stack((k, s["v"].float()), dim=1) / need[block][..., None]
    codes[block, :, :, row] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    return {"q": q, "cache": s["cache"], "scales": scales}


def _decode(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    pages = s["table"].clamp(min=0).long()
    kv = s["cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    kv = kv * s["scales"][pages][..., None, None]  # [B, pages, 2, Hkv, page, D]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, -1, D)
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    scores = q @ kv[0].transpose(-1, -2) / math.sqrt(D)
    unseen = torch.arange(kv.shape[3], device="cuda") >= s["lens"][:, None, None, None]
    scores = scores.masked_fill(unseen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    weights = torch.exp(scores - top.clamp(min=-3e38))
    total = weights.sum(dim=-1, keepdim=True)
    o = (weights @ kv[1]) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0].reshape(B, Hq)
    return {"o": o.to(DTYPES[case["dtype"]]).reshape(B, Hq, 1, D), "lse": lse}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from transformer_attention_fwd_gb300 import attn
        if op == "decode":
            o, lse = attn.attn_fwd_decode_paged_e4m3(state["q"], state["cache"], state["scales"], state["table"],
                                                     state["lens"])
            return {"o": o, "lse": lse}
        r = state["rotation"]
        rotation = attn.Rotation(r["turns"], interleaved=r["inter"], magnitude=r["magnitude"])
        if op == "rope":
            q, k = attn.attn_rope(state["q"], state["k"], state["pos"], rotation)
            return {"q": q, "k": k}
        if op == "norm_rope":
            q, k = attn.attn_qk_norm_rope(state["q"], state["k"], state["qw"], state["kw"], state["pos"], rotation,
                                          eps=1e-6)
            return {"q": q, "k": k}
        if case["cache"] == "16":
            q, _ = attn.attn_append_paged(state["k"], state["v"], state["cache"], state["table"], state["cu"],
                                          state["lens"], rotation=rotation, q=state["q"])
            return {"q": q, "cache": state["cache"]}
        q, _ = attn.attn_append_paged_e4m3(state["k"], state["v"], state["cache"], state["scales"], state["table"],
                                           state["cu"], state["lens"], rotation=rotation, q=state["q"])
        return {"q": q, "cache": state["cache"], "scales": state["scales"]}
    if op == "decode":
        return _decode(state)
    if op == "append":
        return _append(state)
    dtype = DTYPES[case["dtype"]]
    q, k = state["q"].float(), state["k"].float()
    if op == "norm_rope":
        q, k = _norm(q, state["qw"], 1e-6), _norm(k, state["kw"], 1e-6)
    # One position per token: over the heads of [T, H, D] or of [B, H, T, D].
    pos = state["pos"][:, None]
    return {"q": _rotate(q, pos, state["rotation"]).to(dtype), "k": _rotate(k, pos, state["rotation"]).to(dtype)}


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("rope", "norm_rope"):
        tokens = case["T"] * case.get("B", 1)
        values = tokens * (Hq + Hkv) * D
        norm = case["op"] == "norm_rope"
        return {"bytes": 2 * e * values + 4 * tokens + 4 * case["rot"] + (2 * D * e if norm else 0),
                "flops": (7 if norm else 3) * values}
    if case["op"] == "append":
        tokens = case["B"] * case["new"]
        held = 1 if case["cache"] == "e4m3" else 2
        scales = 8 * Hkv * (tokens // case["page"] + case["B"]) if held == 1 else 0
        return {"bytes": tokens * D * (2 * e * Hq + 2 * Hkv * (e + held)) + 4 * (tokens // case["page"] + 3 * case["B"])
                + scales, "flops": 3 * tokens * D * (Hq + Hkv)}
    tokens = case["B"] * case["len"]
    pages = case["B"] * -(-case["len"] // case["page"])
    return {"bytes": tokens * 2 * Hkv * D + pages * (8 * Hkv + 4) + case["B"] * Hq * (2 * D * e + 4),
            "flops": 4 * tokens * Hq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, pos, rotation):
    """x float64 [..., D] with each pair as a complex number times magnitude * e^{i angle}."""
    n = rotation["freq"].shape[0]
    angle = pos.double().unsqueeze(-1) * rotation["freq"]
    by = torch.polar(torch.full_like(angle, rotation["magnitude"]), angle)
    y = x.clone()
    first = slice(0, 2 * n, 2) if rotation["inter"] else slice(0, n)
    second = slice(1, 2 * n, 2) if rotation["inter"] else slice(n, 2 * n)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * by
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(case, s):
    cu, lens, page = s["cu"].tolist(), s["lens"].tolist(), case["page"]
    table = s["table"].tolist()
    pos = torch.cat([torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b]) for b in range(case["B"])]).cuda()
    q = _turned(s["q"].double(), pos[:, None], s["rotation"])
    k = _turned(s["k"].double(), pos[:, None], s["rotation"])
    cache = s["cache"].double()
    held = case["cache"] == "e4m3"
    scales = s["scales"].double() if held else None
    b2 = [math.sqrt(2.0) * s["rotation"]["magnitude"], 1.0]
    for b in range(case["B"]):
        at = lens[b] - (cu[b + 1] - cu[b])
        while at < lens[b]:
            end = min(lens[b], (at // page + 1) * page)
            rows = slice(cu[b + 1] - lens[b] + at, cu[b + 1] - lens[b] + end)
            block, r0 = table[b][at // page], at % page
            for j, (raw, x) in enumerate(((s["k"], k), (s["v"], s["v"].double()))):
                new = x[rows].transpose(0, 1)
                if held:
                    most = raw[rows].double().abs().amax(dim=(0, 2))
                    limit = float(torch.tensor(E4M3_MAX / b2[j], dtype=torch.float32))
                    scale = torch.exp2(torch.ceil(torch.log2(most / limit))).clamp(min=MIN_SCALE)
                    scale = torch.where(most > limit * scale, 2 * scale, scale)
                    if r0:
                        old = scales[block, j].clone()
                        scale = torch.maximum(scale, old)
                        cache[block, j, :, :r0] *= (old / scale)[:, None, None]
                    scales[block, j] = scale
                    new = new / scale[:, None, None]
                cache[block, j, :, r0:r0 + end - at] = new
            at = end
    return {"q": q, "cache": cache, **({"scales": scales} if held else {})}


def _exact_decode(case, s):
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    o = torch.zeros(B, Hq, 1, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        kv = s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
        kv = (kv * s["scales"][ids].double()[..., None, None]).permute(1, 2, 0, 3, 4).reshape(2, Hkv, -1, D)[:, :, :n]
        kv = kv.repeat_interleave(Hq // Hkv, dim=1)
        x = torch.einsum("hd,hnd->hn", s["q"][b, :, 0].double(), kv[0]) / math.sqrt(D)
        lse[b] = torch.logsumexp(x, dim=-1)
        o[b, :, 0] = torch.einsum("hn,hnd->hd", torch.exp(x - lse[b][:, None]), kv[1])
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["op"] == "norm_rope":
            x = x * s[name + "w"].double() / torch.sqrt((x ** 2).sum(dim=-1, keepdim=True) / case["D"] + 1e-6)
        out[name] = _turned(x, s["pos"].unsqueeze(1), s["rotation"])
    return out
