"""Plain forms of the 4-bit cache, of accumulated attention weights and of eviction, on
the CPU: codes and scales in fp32 operation by operation, the rest in 64 bits; and the
error bounds their tests use."""
from __future__ import annotations

import math

import torch

import kv_ref

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BORDERS = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)


def e2m1(y):
    """Codes of y (float64): to the nearest, halfway to the even code; 6 and over to 6."""
    a = y.abs()[..., None]
    up = torch.tensor([False, True, False, True, False, True, False])  # a tie goes up to an even code
    code = ((a > BORDERS) | ((a == BORDERS) & up)).sum(dim=-1)
    return code + 8 * torch.signbit(y)


def values(codes):
    """The magnitudes and signs that codes 0 .. 15 stand for, float64."""
    v = VALUES.double()[codes % 8]
    return torch.where(codes >= 8, -v, v)


def unpack(raw):
    """Codes [..., D] of bytes [..., D / 2]."""
    return torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2).long()


def pack(codes):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def scales_of(most, factor):
    """e4m3 scales (as float32) of groups whose largest magnitude is `most`, fp32 step by step."""
    q = most / (6.0 * factor)
    return q.clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).float()


def quantise(x, factor):
    """(codes [..., D], scales [..., D / 16] float32) of rows x (any float type); factor
    float32, broadcasting over x's leading dimensions with two dimensions of 1 behind."""
    g = x.float().unflatten(-1, (-1, 16))
    finite = torch.where(torch.isfinite(g), g.abs(), torch.zeros_like(g))
    scale = scales_of(finite.amax(dim=-1), factor)
    by = torch.ones_like(scale) / (scale * factor)
    codes = e2m1((g * by[..., None]).double()).flatten(-2)
    return codes, torch.where(torch.isnan(g).any(dim=-1), torch.full_like(scale, math.nan), scale)


def held(cache, scales, factors):
    """Every element of a 4-bit pool: [blocks, 2, Hkv, page, D] float64."""
    x = values(unpack(cache)) * scales.double().repeat_interleave(16, dim=-1)
    return x if factors is None else x * factors.double()[:, :, None, None]


def rows_of(pool, table, b, n):
    """K and V of request b's first n slots: [2, Hkv, n, D]."""
    page = pool.shape[3]
    ids = table[b, : -(-n // page)].long()
    return pool[ids].permute(1, 2, 0, 3, 4).reshape(2, pool.shape[2], len(ids) * page, -1)[:, :, :n]


def random_pool(blocks, Hkv, page, D, gen, low=0.1, high=0.6):
    cache = torch.randint(0, 256, (blocks, 2, Hkv, page, D // 2), generator=gen, dtype=torch.uint8)
    scales = low + (high - low) * torch.rand(blocks, 2, Hkv, page, D // 16, generator=gen)
    return cache, scales.to(torch.float8_e4m3fn)


# The error of a score in fp32: D/16 products of 16 terms added to an fp32 sum, each step
# within 2^-22 of the terms' sizes (the tensor core may truncate), and three fp32 products.
def score_error(D):
    return (D / 16 + 6) * 2.0 ** -22


def decode(q, pool, table, lens, scale=None):
    """(o, lse, spread, dx, share, share_error) in float64 over a pool of rows in float64:
    spread = sum p |v| / sum p; dx bounds a score's fp32 error; share [B][Hkv, n]: the keys'
    weights added over the query heads, share_error its relative bound but for sums."""
    B, Hq, _, D = q.shape
    Hkv = pool.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    spread, dx = torch.zeros_like(o), torch.zeros(B, Hq, dtype=torch.float64)
    share, share_tol = [], []
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            share.append(torch.zeros(Hkv, 0, dtype=torch.float64))
            share_tol.append(torch.zeros(Hkv, 0, dtype=torch.float64))
            continue
        kv = rows_of(pool, table, b, n).repeat_interleave(Hq // Hkv, dim=1)
        x = torch.einsum("hd,hnd->hn", q[b, :, 0].double(), kv[0]) * scale
        size = torch.einsum("hd,hnd->hn", q[b, :, 0].double().abs(), kv[0].abs()) * scale
        lse[b] = torch.logsumexp(x, dim=-1)
        p = torch.exp(x - lse[b][:, None])
        o[b] = torch.einsum("hn,hnd->hd", p, kv[1])
        spread[b] = torch.einsum("hn,hnd->hd", p, kv[1].abs())
        e = size * score_error(D)
        dx[b] = e.amax(dim=-1)
        # A probability: its score's and the log-sum-exp's errors, the latter's two roundings
        # and the difference's (2^-22 of their sizes in all), and the exponential's 2^-21.
        rel = e + dx[b][:, None] + (x.abs() + lse[b].abs()[:, None] + 1.0) * 2.0 ** -21
        share.append(p.reshape(Hkv, -1, n).sum(dim=1))
        share_tol.append((p * rel).reshape(Hkv, -1, n).sum(dim=1))
    return o, lse, spread, dx, share, share_tol


def check_decode(o, lse, ref, keys, what=""):
    """Weights within 2^-14 of themselves, exponentials 2^-20, the scores' dx; sums of `keys`
    positive terms over four lanes and the warps' pieces."""
    want, wl, spread, dx = ref[:4]
    h = kv_ref.HALF_STEP[o.dtype]
    sums = (keys / 4 + 64) * 2.0 ** -24
    rel = 2.0 ** -14 + 2.0 ** -20 + 2 * dx[..., None] + 2 * sums
    tol = h * want.abs() + (1 + h) * rel * spread + kv_ref.TINY[o.dtype]
    got = o.detach().cpu().double()[:, :, 0]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: o: {int(bad.sum())} off, worst {float(((got - want).abs() / tol).max()):.2f} of the bound"
    if lse is not None:
        l = lse.detach().cpu().double()
        empty = torch.isinf(wl)
        assert torch.equal(torch.isneginf(l), empty), what
        ltol = dx + sums + 2.0 ** -20 + wl.abs() * 2.0 ** -22
        bad = ~((l - wl).abs() <= ltol) & ~empty
        assert not bad.any(), f"{what}: lse off by {float((l - wl).abs()[~empty].max()):.2e}"


def check_weights(now, before, table, lens, share, share_tol, keys, what=""):
    """now, before: [blocks, Hkv, page] float32; share added to the requests' slots and nothing
    anywhere else.  A sum's roundings: `keys` terms in lanes of four, and the addition to what
    was there."""
    page = now.shape[2]
    want, tol = before.double().clone(), torch.zeros(before.shape, dtype=torch.float64)
    for b in range(len(lens)):
        n = int(lens[b])
        slot = torch.arange(n)
        blk, row = table[b, slot // page].long(), slot % page
        want[blk, :, row] += share[b].T
        more = share_tol[b].T + share[b].T * (keys / 4 + 64) * 2.0 ** -24
        tol[blk, :, row] += more + (want[blk, :, row].abs() + more) * 2.0 ** -24
    bad = ~((now.detach().cpu().double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: weights: {int(bad.sum())} off, worst {float((now.cpu().double() - want).abs()[bad].max()):.2e}"


def column_sums(q, lse, pool, table, cu, lens, scale=None):
    """(share, share_tol) of every request for packed queries [total, Hq, D], lse [Hq, total]."""
    total, Hq, D = q.shape
    Hkv = pool.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    share, tols = [], []
    for b in range(len(lens)):
        n, t0, t1 = int(lens[b]), int(cu[b]), int(cu[b + 1])
        s, tol = torch.zeros(Hkv, n, dtype=torch.float64), torch.zeros(Hkv, n, dtype=torch.float64)
        if t1 > t0:
            k = rows_of(pool, table, b, n)[0].double()
            last = n - (t1 - t0) + torch.arange(t1 - t0)
            seen = torch.arange(n) <= last[:, None]
            for h in range(Hq):
                x = q[t0:t1, h].double() @ k[h * Hkv // Hq].T * scale
                size = q[t0:t1, h].double().abs() @ k[h * Hkv // Hq].abs().T * scale
                z = lse[h, t0:t1, None].double()
                p = torch.where(seen & ~torch.isneginf(z), torch.exp(x - z), torch.zeros_like(x))
                rel = size * score_error(D) + (x.abs() + z.abs().clamp(max=1e30) + 1.0) * 2.0 ** -21
                s[h * Hkv // Hq] += p.sum(dim=0)
                tol[h * Hkv // Hq] += torch.where(p > 0, p * rel, torch.zeros_like(p)).sum(dim=0)
        share.append(s)
        tols.append(tol)
    return share, tols


def evict(pools, weights, table, lens, keep, recent):
    """Eviction slot by slot: (pools, weights, new_lens, kept) after it."""
    pools, weights = [p.clone() for p in pools], weights.clone()
    page, Hkv = weights.shape[2], weights.shape[1]
    kept = torch.full((len(lens), Hkv, keep), -1, dtype=torch.int32)
    for b, n in enumerate(int(x) for x in lens):
        if n <= keep:
            kept[b, :, :n] = torch.arange(n, dtype=torch.int32)
            continue
        at = [(int(table[b, s // page]), s % page) for s in range(n)]
        for h in range(Hkv):
            w = [float(weights[blk, h, row]) for blk, row in at]
            order = sorted(range(n - recent), key=lambda s: (0 if not math.isnan(w[s]) else 1, -w[s] if not math.isnan(w[s]) else 0.0, s))
            stay = sorted(order[:keep - recent]) + list(range(n - recent, n))
            kept[b, h] = torch.tensor(stay, dtype=torch.int32)
            rows = [[p[at[s][0], :, h, at[s][1]].clone() for s in stay] for p in pools]
            for i, s in enumerate(stay):
                for p, r in zip(pools, rows):
                    p[at[i][0], :, h, at[i][1]] = r[i]
            for s in range(n):
                weights[at[s][0], h, at[s][1]] = w[stay[s]] if s < keep else 0.0
    return pools, weights, torch.tensor([min(int(n), keep) for n in lens], dtype=torch.int32), kept
