"""Cases of the 4-bit cache and of eviction by accumulated attention weight.

Every case is one call of a serving program: append keys and values to the paged
4-bit cache, attend over it, add up what attention weight each cached key got, or
evict the keys that got least.  `run` computes it in its plain form from elementary
torch operations, or, where `own` is set, through the framework's entry points.

The 4-bit cache holds e2m1 codes (sign, two exponent bits, one mantissa bit), two to a
byte, the even element in the low half, with one e4m3 scale for each 16 elements of a
row and one float factor for each head of K and of V.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX, E4M3_LEAST = 448.0, 2.0 ** -9
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of codes 0 .. 7; 8 .. 15 are negative


def listed():
    return [
        # One new token for each of 64 requests against 16-token pages, its keys rotated already.
        {"name": "append_step", "op": "append", "B": 64, "new": 1, "past": 2048, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "dtype": "bf16"},
        # Prompts of different lengths, some continuing a request that has tokens already.
        {"name": "append_prompts", "op": "append", "B": 9, "new": 1900, "past": 300, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "dtype": "bf16"},
        # Few ragged requests, one query head per key head, the 64-wide head: the small end of decoding.
        {"name": "decode_small", "op": "decode", "B": 3, "len": 777, "spread": 700, "Hq": 12, "Hkv": 12, "D": 64,
         "page": 16, "add": False, "dtype": "f16"},
        # The decode workload's sizes: 64 requests of 4096 cached tokens, four query heads a key head.
        {"name": "decode", "op": "decode", "B": 64, "len": 4096, "spread": 0, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "add": False, "dtype": "bf16"},
        # Eight query heads per key head, ragged lengths, larger pages.
        {"name": "decode_gqa8", "op": "decode", "B": 32, "len": 3500, "spread": 1200, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "add": False, "dtype": "bf16"},
        # The decode workload again, every key's attention weight added up for a later eviction.
        {"name": "decode_add", "op": "decode", "B": 64, "len": 4096, "spread": 0, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "add": True, "dtype": "bf16"},
        # A decode step over the 16-bit cache, its weights added up behind it.
        {"name": "weights_step", "op": "weights", "cache": "16", "B": 32, "new": 1, "len": 4096, "spread": 900,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # What the last 64 tokens of each prompt attend to: the votes an eviction after the prompt goes by.
        {"name": "weights_window", "op": "weights", "cache": "16", "B": 16, "new": 64, "len": 4096, "spread": 1500,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # All tokens of one prompt, over its 4-bit cache.
        {"name": "weights_prompt_4bit", "op": "weights", "cache": "4", "B": 1, "new": 4096, "len": 4096, "spread": 0,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # Two short requests cut back to 512 tokens: latency.
        {"name": "evict_small_4bit", "op": "evict", "cache": "4", "B": 2, "len": 1201, "spread": 300, "keep": 512,
         "recent": 64, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # The decode workload's cache cut back to half, in 16 bits.
        {"name": "evict", "op": "evict", "cache": "16", "B": 64, "len": 4096, "spread": 300, "keep": 2048,
         "recent": 256, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # Longer requests, in 4 bits.
        {"name": "evict_4bit", "op": "evict", "cache": "4", "B": 32, "len": 8192, "spread": 2000, "keep": 4096,
         "recent": 500, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "weights", "weights", "evict", "evict"))
    hkv = rng.choice((1, 2, 4, 5, 8, 12))
    hq = hkv * rng.choice((1, 2, 3, 4, 7, 8))
    hq = min(hq, hkv * max(1, 64 // hkv))
    case = {"op": op, "Hq": hq, "Hkv": hkv, "D": rng.choice((64, 128)), "page": rng.choice((1, 5, 8, 16, 16, 24, 64)),
            "dtype": rng.choice(("bf16", "bf16", "f16"))}
    if op == "append":
        case["B"] = _log(rng, 1, 96)
        return {**case, "new": _log(rng, 1, 12288 // case["B"]), "past": rng.choice((0, 40, 700, 1500))}
    if op == "decode":
        case["B"] = _log(rng, 1, 64)
        length = _log(rng, 1, min(16384, 2097152 // (case["B"] * hkv)))
        return {**case, "len": length, "spread": rng.choice((0, length // 3, length - 1)),
                "add": rng.random() < 0.5}
    cache = rng.choice(("16", "4"))
    if op == "weights":
        case["B"] = _log(rng, 1, 32)
        length = _log(rng, 1, min(16384, 1048576 // (case["B"] * hkv)))
        new = _log(rng, 1, min(length, max(1, 2 ** 28 // (case["B"] * length * hq))))
        return {**case, "cache": cache, "len": length, "spread": rng.choice((0, length // 3, length - 1)), "new": new}
    case["B"] = _log(rng, 1, 64)
    length = _log(rng, 2, min(32768, 2097152 // (case["B"] * hkv)))
    keep = max(1, int(length * rng.uniform(0.1, 0.9)))
    return {**case, "cache": cache, "len": length, "spread": rng.choice((0, length // 3, length - 1)), "keep": keep,
            "recent": rng.choice((0, keep // 8, keep // 2))}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _lengths(case, cpu):
    B, spread = case["B"], case["spread"]
    lens = [max(0, case["len"] + int(torch.randint(-spread, spread + 1, (1,), generator=cpu))) for _ in range(B)]
    if spread and B > 1:
        lens[-1] = 0  # a request that has no tokens yet
    return lens


def _pages(lens, most, page, cpu):
    """A block table over a pool that could hold `most` tokens for every request; unused entries are -1."""
    width = max(1, -(-most // page))
    pool, table, at = torch.randperm(len(lens) * width + 3, generator=cpu).tolist(), [], 0
    for n in lens:
        n = -(-n // page)
        table.append(pool[at:at + n] + [-1] * (width - n))
        at += n
    return _int32(table), len(pool)


def _cache(case, s, blocks, gen, four):
    """The pool: 16-bit rows, or codes, scales and factors that make rows of about the same size."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    if not four:
        s["cache"] = torch.randn((blocks, 2, Hkv, page, D), generator=gen, device="cuda", dtype=DTYPES[case["dtype"]])
        return
    s["cache"] = torch.randint(0, 256, (blocks, 2, Hkv, page, D // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
    scales = torch.rand((blocks, 2, Hkv, page, D // 16), generator=gen, device="cuda")
    s["scales"] = (2.0 + 4.0 * scales).to(torch.float8_e4m3fn)
    s["factors"] = 0.05 + 0.05 * torch.rand((2, Hkv), generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    op, B, D, Hq, Hkv, page = case["op"], case["B"], case["D"], case["Hq"], case["Hkv"], case["page"]
    if op == "append":
        spread, new = case["new"] // 2, [case["new"]] * B
        for b in range(0, B - 1, 2):  # prompts of different lengths, as many tokens in all
            more = int(torch.randint(-spread, spread + 1, (1,), generator=cpu))
            new[b], new[b + 1] = new[b] + more, new[b + 1] - more
        lens = [n + int(torch.randint(0, case["past"] + 1, (1,), generator=cpu)) for n in new]
        s["table"], blocks = _pages(lens, case["new"] + spread + case["past"], page, cpu)
        s["lens"] = _int32(lens)
        s["cu"] = _int32([sum(new[:b]) for b in range(B + 1)])
        kv = torch.randn((sum(new), 2 * Hkv, D), generator=gen, device="cuda", dtype=torch.float32)
        kv *= torch.exp(0.5 * torch.randn((1, 2 * Hkv, D), generator=gen, device="cuda"))  # channels differ in size
        kv = kv.to(dtype)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        _cache(case, s, blocks, gen, True)
        return s
    lens = _lengths(case, cpu)
    s["table"], blocks = _pages(lens, case["len"] + case["spread"], page, cpu)
    s["lens"] = _int32(lens)
    if op == "decode":
        _cache(case, s, blocks, gen, True)
        s["q"] = torch.randn((B, Hq, 1, D), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
        if case["add"]:
            s["weights"] = torch.rand((blocks, Hkv, page), generator=gen, device="cuda")
        return s
    _cache(case, s, blocks, gen, case["cache"] == "4")
    if op == "weights":
        new = [min(case["new"], n) for n in lens]
        cu = [sum(new[:b]) for b in range(B + 1)]
        s["cu"] = _int32(cu)
        s["q"] = torch.randn((cu[-1], Hq, D), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
        # The log-sum-exp of n scores of N(0, 1) is about ln n + 1/2.
        seen = torch.cat([torch.arange(n - m + 1, n + 1) for n, m in zip(lens, new)]).to("cuda", torch.float32)
        s["lse"] = seen.log() + 0.5 + 0.05 * torch.randn((Hq, cu[-1]), generator=gen, device="cuda")
        s["weights"] = torch.rand((blocks, Hkv, page), generator=gen, device="cuda")
        return s
    # Sums of probabilities are spread over orders of magnitude; keys far from every query have none.
    w = torch.exp(2.0 * torch.randn((blocks, Hkv, page), generator=gen, device="cuda")) / max(1, case["len"])
    w *= torch.rand((blocks, Hkv, page), generator=gen, device="cuda") > 0.1
    s["start"], s["weights"] = w, torch.empty_like(w)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _table_rows(s):
    """Block, row in the block and presence of slots 0 .. of every request: [B, slots]."""
    page = s["case"]["page"]
    slot = torch.arange(s["table"].shape[1] * page, device="cuda")
    block = s["table"].clamp(min=0).long().repeat_interleave(page, dim=1)
    return block, (slot % page).expand_as(block), slot < s["lens"][:, None]


def _held(s, side):
    """K (0) or V (1) rows of all pages of every request in 32 bits: [B, Hkv, slots, D]."""
    pages = s["table"].clamp(min=0).long()
    rows = s["cache"][pages, side]
    if s["cache"].dtype == torch.uint8:
        value = torch.tensor(VALUES + tuple(-v for v in VALUES), device="cuda")
        codes = torch.stack((rows & 15, rows >> 4), dim=-1).flatten(-2)
        by = s["scales"].view(torch.uint8)[pages, side].view(torch.float8_e4m3fn).float()
        by = by * s["factors"][side][:, None, None]
        rows = (value[codes.int()].unflatten(-1, (-1, 16)) * by[..., None]).flatten(-2)
    return rows.float().permute(0, 2, 1, 3, 4).flatten(2, 3)


def _codes(x, by):
    """e2m1 codes of x [..., 16] times by [..., 1]: to the nearest, halfway to the even code; two to a byte."""
    half = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda")
    even = torch.tensor((False, True, False, True, False, True, False), device="cuda")
    border = torch.where(even, torch.nextafter(half, torch.zeros_like(half)), half)
    code = torch.bucketize((x * by).abs(), border) + 8 * torch.signbit(x)
    code = code.to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _append(s):
    page = s["case"]["page"]
    token = torch.arange(s["k"].shape[0], device="cuda", dtype=torch.int32)
    request = torch.searchsorted(s["cu"][1:], token, right=True)
    slot = s["lens"][request] - s["cu"][1:][request] + token
    block, row = s["table"][request, (slot // page).long()].long(), (slot % page).long()
    x = torch.stack((s["k"], s["v"]), dim=1).float().unflatten(-1, (-1, 16))  # [T, 2, Hkv, D / 16, 16]
    factor = s["factors"][..., None]
    scale = (x.abs().amax(dim=-1) / (6.0 * factor)).clamp(E4M3_LEAST, E4M3_MAX).to(torch.float8_e4m3fn)
    by = torch.ones_like(factor) / (scale.float() * factor)
    s["cache"][block, :, :, row] = _codes(x, by[..., None])
    s["scales"].view(torch.uint8)[block, :, :, row] = scale.view(torch.uint8)
    return {"cache": s["cache"], "scales": s["scales"]}


def _add(s, share, block, row, here):
    """Adds share [B, Hkv, slots] to the weights of the slots that are there."""
    s["weights"][block[here], :, row[here]] += share.transpose(1, 2)[here]


def _decode(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    block, row, here = _table_rows(s)
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    scores = q @ _held(s, 0).transpose(-1, -2) / math.sqrt(D)
    scores = scores.masked_fill(~here[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    weights = torch.exp(scores - top.clamp(min=-3e38))
    total = weights.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    o = ((weights @ _held(s, 1)) / total).to(DTYPES[case["dtype"]]).reshape(B, Hq, 1, D)
    out = {"o": o, "lse": (top + total.log())[..., 0].reshape(B, Hq)}
    if case["add"]:
        _add(s, (weights / total).sum(dim=2), block, row, here)
        out["weights"] = s["weights"]
    return out


def _weights(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    block, row, here = _table_rows(s)
    first, count = s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(min(case["new"], here.shape[1]), device="cuda")
    there = i < count[:, None]  # [B, new]
    token = (first[:, None] + i).clamp(max=max(0, s["q"].shape[0] - 1)).long()
    q = s["q"].float()[token].reshape(B, -1, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    lse = s["lse"][:, token].reshape(Hkv, Hq // Hkv, B, -1).permute(2, 0, 1, 3)
    scores = q @ _held(s, 0)[:, :, None].transpose(-1, -2) / math.sqrt(D)  # [B, Hkv, group, new, slots]
    last = s["lens"][:, None] - count[:, None] + i  # a token's own slot, and the last that it sees
    seen = there[..., None] & (torch.arange(here.shape[1], device="cuda") <= last[..., None])
    share = torch.exp(scores.sub_(lse[..., None])).masked_fill_(~seen[:, None, None], 0.0).sum(dim=(2, 3))
    _add(s, share, block, row, here)
    return {"weights": s["weights"]}


def _evict(s):
    case = s["case"]
    keep, recent = case["keep"], case["recent"]
    s["weights"].copy_(s["start"])  # what the steps since the last eviction have added up to
    block, row, here = _table_rows(s)
    lens, slots = s["lens"][:, None, None].long(), block.shape[1]
    w = s["weights"][block, :, row].transpose(1, 2)  # [B, Hkv, slots]
    slot = torch.arange(slots, device="cuda")
    w = w.masked_fill((slot >= lens - recent) & (slot < lens), math.inf).masked_fill(slot >= lens, -math.inf)
    held = min(keep, slots)
    kept = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :held].sort(dim=-1)[0]
    i = torch.arange(held, device="cuda")
    kept = torch.where(lens <= keep, i.expand_as(kept), kept)  # [B, Hkv, held]
    b, h, n = torch.nonzero((i < lens) & (lens > keep).expand_as(kept), as_tuple=True)
    source = kept[b, h, n]
    # Everything is read before anything is written.
    names = ("cache", "scales") if "scales" in s else ("cache",)
    rows = [s[name].view(torch.uint8)[block[b, source], :, h, row[b, source]] for name in names]
    moved = s["weights"][block[b, source], h, row[b, source]]
    for name, x in zip(names, rows):
        s[name].view(torch.uint8)[block[b, n], :, h, row[b, n]] = x
    gone = here & (slot >= keep)
    s["weights"][block[gone], :, row[gone]] = 0.0
    s["weights"][block[b, n], h, row[b, n]] = moved
    full = torch.full((*kept.shape[:2], keep), -1, dtype=torch.int32, device="cuda")
    full[..., :held] = torch.where(i < lens, kept, -1)
    return {"lens": s["lens"].clamp(max=keep), "kept": full, "weights": s["weights"],
            **{name: s[name] for name in names}}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from transformer_attention_fwd_gb300 import attn
        if op == "append":
            attn.attn_append_paged_e2m1(s["k"], s["v"], s["cache"], s["scales"], s["table"], s["cu"], s["lens"],
                                        factors=s["factors"])
            return {"cache": s["cache"], "scales": s["scales"]}
        if op == "decode":
            o, lse = attn.attn_fwd_decode_paged_e2m1(s["q"], s["cache"], s["scales"], s["table"], s["lens"],
                                                     factors=s["factors"], weights=s.get("weights"))
            return {"o": o, "lse": lse, **({"weights": s["weights"]} if state["case"]["add"] else {})}
        four = state["case"]["cache"] == "4"
        if op == "weights":
            if four:
                attn.attn_weights_paged_e2m1(s["q"], s["lse"], s["cache"], s["scales"], s["table"], s["cu"],
                                             s["lens"], s["weights"], factors=s["factors"])
            else:
                attn.attn_weights_paged(s["q"], s["lse"], s["cache"], s["table"], s["cu"], s["lens"], s["weights"])
            return {"weights": s["weights"]}
        s["weights"].copy_(s["start"])
        keep, recent = state["case"]["keep"], state["case"]["recent"]
        if four:
            lens, kept = attn.attn_evict_paged_e2m1(s["cache"], s["scales"], s["weights"], s["table"], s["lens"],
                                                    keep, recent)
        else:
            lens, kept = attn.attn_evict_paged(s["cache"], s["weights"], s["table"], s["lens"], keep, recent)
        return {"lens": lens, "kept": kept, "weights": s["weights"], "cache": s["cache"],
                **({"scales": s["scales"]} if four else {})}
    return {"append": _append, "decode": _decode, "weights": _weights, "evict": _evict}[op](s)


def work(case):
    D, Hq, Hkv, B, op = case["D"], case["Hq"], case["Hkv"], case["B"], case["op"]
    row = D // 2 + D // 16 if op in ("append", "decode") or case["cache"] == "4" else 2 * D  # bytes of a K or V row
    if op == "append":
        tokens = B * case["new"]
        return {"bytes": tokens * 2 * Hkv * (2 * D + row) + 4 * (tokens // case["page"] + 3 * B),
                "flops": 4 * tokens * 2 * Hkv * D}
    tokens = B * case["len"]
    pages = 4 * B * -(-case["len"] // case["page"])
    if op == "decode":
        add = 8 * tokens * Hkv if case["add"] else 0
        return {"bytes": tokens * 2 * Hkv * row + pages + B * Hq * (4 * D + 4) + add, "flops": 4 * tokens * Hq * D}
    if op == "weights":
        new = min(case["new"], case["len"])
        pairs = B * (new * case["len"] - new * (new - 1) // 2)
        return {"bytes": tokens * Hkv * (row + 8) + pages + B * new * Hq * (2 * D + 4), "flops": 2 * pairs * Hq * D}
    if case["len"] <= case["keep"]:
        return {"bytes": 8 * B + 4 * B * Hkv * case["keep"], "flops": 0}
    keep = B * Hkv * case["keep"]
    return {"bytes": keep * 2 * 2 * row + 8 * tokens * Hkv + 4 * keep + pages, "flops": tokens * Hkv}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _rows64(case, s, b, side):
    """K or V rows of request b, [Hkv, len, D], code by code."""
    n, page = int(s["lens"][b]), case["page"]
    ids = s["table"][b, :-(-n // page)].long()
    x = s["cache"][ids, side]
    if x.dtype == torch.uint8:
        code = torch.empty((*x.shape[:-1], case["D"]), dtype=torch.int64, device="cuda")
        code[..., 0::2], code[..., 1::2] = x % 16, x // 16
        low = code % 8
        value = torch.where(low < 2, low * 0.5, (1.0 + 0.5 * (low % 2).double()) * 2.0 ** (low // 2 - 1).double())
        value = torch.where(code >= 8, -value, value)
        scale = s["scales"].view(torch.uint8)[ids, side].view(torch.float8_e4m3fn).double()
        x = value * scale.repeat_interleave(16, dim=-1) * s["factors"][side].double()[:, None, None]
    return x.double().transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_append(case, s):
    """The scales and values that would be held if both had all their bits; codes have no such value."""
    scales = s["scales"].double()
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].long()
    for b in range(case["B"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        slot = torch.arange(lens[b] - n, lens[b], device="cuda")
        for side, x in enumerate((s["k"], s["v"])):
            x = x[cu[b]:cu[b + 1]].double().reshape(n, case["Hkv"], -1, 16)
            most = x.abs().max(dim=-1)[0] / (6 * s["factors"][side].double()[:, None])
            most = most.clamp(E4M3_LEAST, E4M3_MAX)
            scales[table[b, slot // case["page"]], side, :, slot % case["page"]] = most
    return {"cache": None, "scales": scales}


def _exact_attention(case, s):
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    decode = case["op"] == "decode"
    add = not decode or case["add"]
    weights = s["weights"].double() if add else None
    o = torch.zeros(B, Hq, 1, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        t0, t1 = (b, b + 1) if decode else (int(s["cu"][b]), int(s["cu"][b + 1]))
        q = s["q"][b].double().transpose(0, 1) if decode else s["q"][t0:t1].double()  # [new, Hq, D]
        slot = torch.arange(n, device="cuda")
        ids = s["table"][b].long()[slot // page]
        k = _rows64(case, s, b, 0)
        v = _rows64(case, s, b, 1) if decode else None
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for part in range(0, t1 - t0, 512):
                x = torch.einsum("thd,nd->htn", q[part:part + 512, heads], k[h]) / math.sqrt(D)
                if decode:
                    z = torch.logsumexp(x, dim=-1, keepdim=True)
                    lse[b, heads] = z[:, 0, 0]
                else:
                    z = s["lse"][heads, t0 + part:t0 + part + x.shape[1], None].double()
                    own_slot = n - (t1 - t0) + part + torch.arange(x.shape[1], device="cuda")
                    x = x.masked_fill(slot > own_slot[:, None], -math.inf)
                p = torch.exp(x - z)
                if decode:
                    o[b, heads, 0] = p[:, 0] @ v[h]
                if add:
                    weights[ids, h, slot % page] += p.sum(dim=(0, 1))
    out = {"o": o, "lse": lse} if decode else {}
    return {**out, **({"weights": weights} if add else {})}


def _exact_evict(case, s):
    """Nothing is computed but the choice: the weights that are left, in 64 bits."""
    page, keep, recent = case["page"], case["keep"], case["recent"]
    weights = s["start"].double()
    for b, n in enumerate(s["lens"].tolist()):
        if n <= keep:
            continue
        slot = torch.arange(n, device="cuda")
        ids, rows = s["table"][b].long()[slot // page], slot % page
        w = s["start"][ids, :, rows].double()  # [n, Hkv]
        order = torch.argsort(-w[:n - recent], dim=0, stable=True)[:keep - recent].sort(dim=0)[0]
        left = torch.zeros_like(w)
        left[:keep - recent] = torch.gather(w, 0, order)
        left[keep - recent:keep] = w[n - recent:]
        weights[ids, :, rows] = left
    return {"lens": None, "kept": None, "weights": weights, "cache": None,
            **({"scales": None} if "scales" in s else {})}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_evict(case, s) if case["op"] == "evict" else _exact_attention(case, s)
