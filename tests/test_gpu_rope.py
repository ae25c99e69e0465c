"""Rotary positions and the norm of query and key heads against their 64-bit
forms."""
import math

import pytest
import torch

import kv_ref
from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _rotation(a, rot, inter=False, magnitude=1.0):
    turns, _ = a.rope_turns(rot) if rot else (torch.empty(0, dtype=torch.int64), 1.0)
    return a.Rotation(turns.cuda(), inter, magnitude), kv_ref.turns_to_radians(turns.tolist())


def _check(x, y, pos, freq, inter, magnitude, what):
    want, size = kv_ref.rotate(x.double(), pos, freq, inter, magnitude)
    kv_ref.check_rows(y, want, size, kv_ref.ROTATION_ERROR, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot,inter", [
    (0, False), (2, False), (2, True), (16, False), (20, False), (36, True), (48, False), (62, False), (64, False),
    (64, True)])
def test_layouts_and_part_of_the_head(dtype, D, rot, inter):
    a = attn()
    q, k = _randn((37, 5, D), DTYPES[dtype], 1), _randn((37, 3, D), DTYPES[dtype], 2)
    pos = torch.randint(-5000, 200000, (37,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    r, freq = _rotation(a, rot, inter)
    yq, yk = a.attn_rope(q.cuda(), k.cuda(), pos.cuda(), r)
    check_status(a)
    for x, y in ((q, yq), (k, yk)):
        _check(x, y, pos[:, None], freq, inter, 1.0, f"{dtype} D{D} rot{rot}")
        # What does not turn passes through bit for bit.
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (100, False), (96, False)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 33, 1), (700, 7, 12), (9, 128, 1)])
def test_counts_of_tokens_and_heads(T, Hq, Hkv, rot, inter):
    a = attn()
    q, k = _randn((T, Hq, 128), torch.bfloat16, 4), _randn((T, Hkv, 128), torch.bfloat16, 5)
    pos = torch.arange(T, dtype=torch.int32) * 17
    r, freq = _rotation(a, rot, inter, magnitude=1.25)
    yq, yk = a.attn_rope(q.cuda(), k.cuda(), pos.cuda(), r)
    check_status(a)
    _check(q, yq, pos[:, None], freq, inter, 1.25, "q")
    _check(k, yk, pos[:, None], freq, inter, 1.25, "k")
    only, none = a.attn_rope(q.cuda(), None, pos.cuda(), r)
    assert none is None and torch.equal(only, yq)


def test_many_tokens_take_runs_of_heads():
    """Enough tokens that a warp takes several steps of heads, an odd number of them."""
    a = attn()
    q, k = _randn((9000, 23, 64), torch.float16, 6), _randn((9000, 5, 64), torch.float16, 7)
    pos = torch.arange(9000, dtype=torch.int32)
    r, freq = _rotation(a, 64)
    yq, yk = a.attn_rope(q.cuda(), k.cuda(), pos.cuda(), r)
    check_status(a)
    _check(q, yq, pos[:, None], freq, False, 1.0, "q")
    _check(k, yk, pos[:, None], freq, False, 1.0, "k")


@pytest.mark.parametrize("rot,inter", [(64, False), (128, True), (20, False)])
def test_dense_layout_and_positions_of_each_batch(rot, inter):
    a = attn()
    q, k = _randn((3, 4, 50, 128), torch.float32, 8), _randn((3, 2, 50, 128), torch.float32, 9)
    pos = torch.randint(0, 4000, (3, 50), generator=torch.Generator().manual_seed(10), dtype=torch.int32)
    r, freq = _rotation(a, rot, inter)
    yq, yk = a.attn_rope(q.cuda(), k.cuda(), pos.cuda(), r)
    check_status(a)
    _check(q, yq, pos[:, None], freq, inter, 1.0, "q")
    _check(k, yk, pos[:, None], freq, inter, 1.0, "k")


@pytest.mark.parametrize("rot", [128, 36])
def test_strided_slices_in_place_and_into_other_strides(rot):
    a = attn()
    T, Hq, Hkv, D = 65, 6, 2, 128
    qkv = _randn((T, Hq + 2 * Hkv, D), torch.bfloat16, 11)
    pos = torch.arange(T, dtype=torch.int32) + 77
    r, freq = _rotation(a, rot)
    dev = qkv.cuda()
    q, k = dev[:, :Hq], dev[:, Hq:Hq + Hkv]
    # Into head-major outputs.
    oq = torch.empty(Hq, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    yq, yk = a.attn_rope(q, k, pos.cuda(), r, out_q=oq)
    assert yq is oq
    _check(qkv[:, :Hq], yq, pos[:, None], freq, False, 1.0, "q")
    _check(qkv[:, Hq:Hq + Hkv], yk, pos[:, None], freq, False, 1.0, "k")
    # In place: the same bits, and v is left as it was.
    a.attn_rope(q, k, pos.cuda(), r, out_q=q, out_k=k)
    check_status(a)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])
    # One row for every token and head (strides of 0).
    one = _randn((1, 1, D), torch.bfloat16, 12)
    y, _ = a.attn_rope(one.cuda().expand(T, Hq, D), None, pos.cuda(), r)
    _check(one.expand(T, Hq, D), y, pos[:, None], freq, False, 1.0, "expanded")


def test_far_positions_keep_their_angle():
    """The angle is exact modulo a turn: at positions up to 2^31 - 1 and below zero the fp32
    bound of a small position holds."""
    a = attn()
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1048576, 999999999, -1, 0], dtype=torch.int32)
    q = _randn((6, 3, 128), torch.float32, 13)
    turns, _ = a.rope_turns(128)
    r = a.Rotation(turns.cuda())
    y, _ = a.attn_rope(q.cuda(), None, pos.cuda(), r)
    # Whole turns taken off in integers before the angle becomes a double.
    want, size = q.double().clone(), q.double().abs()
    for i, p in enumerate(pos.tolist()):
        angle = torch.tensor([((p * (int(t) % 2 ** 64)) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns],
                             dtype=torch.float64)
        u, v = q[i, :, :64].double(), q[i, :, 64:].double()
        want[i, :, :64], want[i, :, 64:] = u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()
        size[i, :, :64] = size[i, :, 64:] = u.abs() + v.abs()
    kv_ref.check_rows(y, want, size, kv_ref.ROTATION_ERROR, "far")


def test_gradient_is_the_rotation_back():
    """<g, rope(x + e d) - rope(x - e d)> / 2e against <rope at -t (g), d>."""
    a = attn()
    T, H, D = 21, 3, 64
    pos = (torch.arange(T, dtype=torch.int32) * 31).cuda()
    r, freq = _rotation(a, 48, True, 1.5)
    x, d, g = (_randn((T, H, D), torch.float32, s).cuda() for s in (14, 15, 16))
    gx, _ = a.attn_rope(g, None, -pos, r)
    want, size = kv_ref.rotate(g.double().cpu(), -pos.cpu()[:, None], freq, True, 1.5)
    kv_ref.check_rows(gx, want, size, kv_ref.ROTATION_ERROR, "gradient")
    up, _ = a.attn_rope(x + d, None, pos, r)
    dn, _ = a.attn_rope(x - d, None, pos, r)
    diff = (g.double() * (up.double() - dn.double())).sum() / 2
    # Each side of the difference is within ROTATION_ERROR of its rows, and the
    # inputs' sums are rounded once (2^-24).
    size = (g.abs() * (kv_ref.rotate((x.abs() + d.abs()).double().cpu(), pos.cpu()[:, None], freq, True, 1.5)[1]
                       ).cuda()).sum()
    assert abs(diff - (gx.double() * d.double()).sum()) <= 4 * (kv_ref.ROTATION_ERROR + 2.0 ** -24) * size


def test_infinities_stay_in_their_pair():
    a = attn()
    q = torch.ones(1, 1, 128, dtype=torch.bfloat16)
    q[..., 5] = math.inf
    q[..., 101] = math.nan
    q[..., 127] = -math.inf
    r, _ = _rotation(a, 64, False)
    y, _ = a.attn_rope(q.cuda(), None, torch.tensor([3], dtype=torch.int32).cuda(), r)
    y = y.cpu()[0, 0].float()
    odd = {5, 37, 101, 127}
    assert all(math.isfinite(y[i]) == (i not in odd) for i in range(128))
    assert y[127] == -math.inf and math.isnan(y[101])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 128, False), (128, 64, True), (64, 20, False),
                                         (128, 0, False)])
@pytest.mark.parametrize("weights", [True, False])
def test_norm_with_rotation(dtype, D, rot, inter, weights):
    a = attn()
    T, Hq, Hkv = 41, 6, 3
    qkv = _randn((T, Hq + Hkv, D), DTYPES[dtype], 17) * 3.0
    qw = kw = None
    if weights:
        qw, kw = (1.0 + 0.3 * _randn((D,), torch.float32, s) for s in (18, 19))
        qw, kw = qw.to(DTYPES[dtype]), kw.to(DTYPES[dtype])
    pos = torch.arange(T, dtype=torch.int32) * 5
    r, freq = _rotation(a, rot, inter)
    dev = qkv.cuda()
    yq, yk = a.attn_qk_norm_rope(dev[:, :Hq], dev[:, Hq:], qw.cuda() if weights else None,
                                 kw.cuda() if weights else None, pos.cuda(), r, eps=1e-5)
    check_status(a)
    for x, w, y in ((qkv[:, :Hq], qw, yq), (qkv[:, Hq:], kw, yk)):
        want, size = kv_ref.rotate(kv_ref.norm(x.double(), w, 1e-5), pos[:, None], freq, inter)
        kv_ref.check_rows(y, want, size, kv_ref.ROTATION_ERROR + kv_ref.norm_error(D), f"{dtype} D{D} rot{rot}")


def test_norm_of_zero_and_tiny_rows():
    a = attn()
    x = torch.zeros(3, 2, 64)
    x[1] = 1e-6
    x[2, 1] = 1e4
    r, freq = _rotation(a, 64)
    pos = torch.tensor([0, 9, 100], dtype=torch.int32)
    y, _ = a.attn_qk_norm_rope(x.cuda(), None, None, None, pos.cuda(), r, eps=1e-6)
    want, size = kv_ref.rotate(kv_ref.norm(x.double(), None, 1e-6), pos[:, None], freq)
    kv_ref.check_rows(y, want, size, kv_ref.ROTATION_ERROR + kv_ref.norm_error(64), "tiny rows")
    assert (y[0] == 0).all()


def test_no_tokens_launch_nothing():
    a = attn()
    r, _ = _rotation(a, 64)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = a.attn_rope(e, None, torch.empty(0, dtype=torch.int32, device="cuda"), r)
    assert y.shape == e.shape and a.last_launch_info()[2] == 0


def test_other_stream_and_graph():
    a = attn()
    r, freq = _rotation(a, 128)
    x, x2 = _randn((64, 8, 128), torch.bfloat16, 20), _randn((64, 8, 128), torch.bfloat16, 21)
    pos = torch.arange(64, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        xd = x.cuda()
        y, _ = a.attn_rope(xd, None, pos, r)
    side.synchronize()
    _check(x, y, pos.cpu()[:, None], freq, False, 1.0, "side stream")
    out = torch.empty_like(xd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.attn_rope(xd, None, pos, r, out_q=out)
    for src in (x2, x):
        xd.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        _check(src, out, pos.cpu()[:, None], freq, False, 1.0, "replay")


@pytest.mark.parametrize("inter", [False, True])
def test_the_angle_is_not_rounded_to_a_float(inter):
    """fp32 rows (1, 0) return cos and sin themselves.  sincospif is within 1 ulp, 2^-23 of a
    value, the turn by the rest of the phase rounds once more, and the phase's 32 bits leave
    2^-32 half turns: next to a half turn, where the sine is small, a phase rounded to a float
    is off by up to 2^-25 half turns, thirty times that."""
    a = attn()
    near_half = [2 ** 63 + s * ((64 + 128 * i) << 32) + (i << 20) for i in range(1, 1500, 47) for s in (-1, 1)]
    for seed in range(20):
        phases = near_half[:64] if seed == 0 else torch.randint(
            -2 ** 63, 2 ** 63 - 1, (64,), generator=torch.Generator().manual_seed(seed)).tolist()
        turns = torch.tensor([p - 2 ** 64 if p >= 2 ** 63 else p for p in phases], dtype=torch.int64)
        assert len(turns) == 64
        x = torch.zeros(1, 1, 128)
        first = slice(0, 128, 2) if inter else slice(0, 64)
        second = slice(1, 128, 2) if inter else slice(64, 128)
        x[..., first] = 1.0
        y, _ = a.attn_rope(x.cuda(), None, torch.ones(1, dtype=torch.int32, device="cuda"),
                           a.Rotation(turns.cuda(), inter))
        y = y.cpu().double()[0, 0]
        angle = torch.tensor([(p % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for p in phases], dtype=torch.float64)
        for got, want in ((y[first], angle.cos()), (y[second], angle.sin())):
            assert ((got - want).abs() <= 2.0 ** -22 * want.abs() + math.pi * 2.0 ** -32 + 2.0 ** -46).all()


def _bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot,inter", [(0, False), (2, True), (16, False), (20, False), (36, True), (48, False)])
def test_what_does_not_turn_keeps_its_bits(dtype, D, rot, inter):
    """Zeros of both signs, infinities and subnormals beyond rot_dim, compared as integers."""
    a = attn()
    x = _randn((33, 6, D), DTYPES[dtype], 22)
    x[::2, :, 1::3], x[1::2, :, 1::3], x[:, ::2, 2::5], x[..., -1] = -0.0, 0.0, -1e-7, -math.inf
    x[:, 3] = -0.0
    r, _ = _rotation(a, rot, inter, magnitude=1.25)
    y, _ = a.attn_rope(x.cuda(), None, torch.arange(33, dtype=torch.int32).cuda(), r)
    check_status(a)
    assert torch.equal(_bits(y.cpu())[..., rot:], _bits(x)[..., rot:])
