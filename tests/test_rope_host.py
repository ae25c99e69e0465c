"""The frequency tables, and what the rotary, append and 8-bit-cache calls
refuse before anything is launched (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import kv_ref


@pytest.fixture(scope="module")
def a():
    from transformer_attention_fwd_gb300 import build
    build.build()
    from transformer_attention_fwd_gb300 import attn
    return attn


def _radians(a, rot, **kw):
    turns, magnitude = a.rope_turns(rot, **kw)
    assert turns.shape == (rot // 2,) and turns.dtype == torch.int64
    return kv_ref.turns_to_radians(turns.tolist()), magnitude


def _close(got, want):
    # The table's resolution, 2^-64 turn, and the double's roundings of pow and division.  Weights
    # of a mean of f and f / factor carry up to 2^-51 absolute, times f, which is up to 16 (the
    # largest factor here) times the result: 2^-47 of it, and the other roundings under that again.
    assert ((got - want).abs() <= want.abs() * 2.0 ** -46 + 2 * math.pi * 2.0 ** -63).all()


@pytest.mark.parametrize("rot", [2, 4, 36, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_plain_and_linear_frequencies(a, rot, base):
    want = kv_ref.frequencies(rot, base)
    got, m = _radians(a, rot, base=base)
    _close(got, want)
    assert m == 1.0
    got, m = _radians(a, rot, base=base, scaling="linear", factor=4.0)
    _close(got, want / 4)
    assert m == 1.0


def test_enlarged_base(a):
    got, m = _radians(a, 64, scaling="base", factor=8.0)
    _close(got, kv_ref.frequencies(64, 10000.0 * 8.0 ** (64 / 62)))
    # The fastest pair keeps its frequency and the slowest is slowed by the factor.
    assert abs(float(got[0]) - 1) < 1e-12 and m == 1.0
    assert abs(float(kv_ref.frequencies(64)[-1] / got[-1]) - 8) < 1e-9


def test_scaling_by_wavelength(a):
    rot, factor, length = 128, 8.0, 8192.0
    f = kv_ref.frequencies(rot, 500000.0)
    got, m = _radians(a, rot, base=500000.0, scaling="wavelength", factor=factor, original_length=length)
    turns = length * f / (2 * math.pi)
    want = torch.where(turns >= 4, f, torch.where(turns <= 1, f / factor,
                                                  f * (turns - 1) / 3 + f / factor * (4 - turns) / 3))
    _close(got, want)
    assert m == 1.0 and (turns > 4).any() and (turns < 1).any() and ((turns > 1) & (turns < 4)).any()


def test_yarn(a):
    rot, factor, length = 128, 16.0, 4096.0
    f = kv_ref.frequencies(rot)
    got, m = _radians(a, rot, scaling="yarn", factor=factor, original_length=length)
    pair = [rot * math.log(length / (r * 2 * math.pi)) / (2 * math.log(10000.0)) for r in (32.0, 1.0)]
    lo, hi = math.floor(pair[0]), math.ceil(pair[1])
    slow = ((torch.arange(rot // 2).double() - lo) / (hi - lo)).clamp(0, 1)
    _close(got, f * (1 - slow) + f / factor * slow)
    assert abs(m - (0.1 * math.log(factor) + 1)) <= 2.0 ** -24 * 2
    assert a.rope_turns(rot, scaling="yarn", factor=1.0, original_length=length)[1] == 1.0


def test_frequencies_over_a_turn_wrap(a):
    """A factor below one speeds pairs up beyond a turn per position; whole turns drop out."""
    got, _ = _radians(a, 64, scaling="linear", factor=0.1)
    _close(got, torch.remainder(kv_ref.frequencies(64) * 10, 2 * math.pi))


@pytest.mark.parametrize("rot,kw,msg", [
    (0, {}, "rot_dim"), (7, {}, "rot_dim"), (-2, {}, "rot_dim"),
    (64, dict(base=1.0), "base"), (64, dict(base=math.nan), "base"),
    (64, dict(scaling="linear", factor=0.0), "factor"),
    (64, dict(scaling="linear", factor=math.inf), "factor"),
    (2, dict(scaling="base", factor=2.0), "rot_dim"),
    (64, dict(scaling="base", factor=1e-6), "must be > 1"),
    (64, dict(scaling="yarn", factor=2.0), "original_length"),
    (64, dict(scaling="wavelength", factor=2.0, original_length=100.0, low=4.0, high=4.0), "low"),
])
def test_bad_tables_are_refused(a, rot, kw, msg):
    with pytest.raises(a.AttnError, match=msg) as e:
        a.rope_turns(rot, **kw)
    assert e.value.status == a.ATTN_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="scaling"):
        a.rope_turns(64, scaling="other")


FAKE = 0x10000  # aligned, never read: validation fails first


def rows(a, x=FAKE, y=FAKE + (1 << 30), heads=4, xs=(0, 64, 256), ys=(0, 64, 256)):
    return a._Rows(x, y, heads, *xs, *ys)


def rotation(a, turns=FAKE, rot=64, inter=0, magnitude=1.0):
    return a._Rotation(turns, rot, inter, magnitude)


def _rope(a, q=None, k=None, positions=FAKE, B=1, T=3, D=64, rot=None, dtype=1, norm=None):
    q = rows(a) if q is None else q
    rot = rotation(a) if rot is None else rot
    if norm is None:
        return a.lib.attn_rope(q, k, positions, B, T, D, rot, dtype, None)
    return a.lib.attn_qk_norm_rope(q, k, norm[0], norm[1], norm[2], positions, B, T, D, rot, dtype, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=3), 1, "dtype"),
    (dict(D=96), 2, "D=96"),
    (dict(B=-1), 1, ">= 0"),
    (dict(B=1 << 16, T=1 << 15), 1, "31 bits"),
    (dict(positions=None), 1, "positions"),
    (dict(positions=FAKE + 2), 1, "positions"),
    (dict(rot=dict(rot=65)), 1, "rot_dim"),
    (dict(rot=dict(rot=66)), 1, "rot_dim"),
    (dict(rot=dict(turns=None)), 1, "turns"),
    (dict(rot=dict(turns=FAKE + 4)), 1, "turns"),
    (dict(rot=dict(magnitude=0.0)), 1, "magnitude"),
    (dict(rot=dict(magnitude=math.nan)), 1, "magnitude"),
    (dict(rot=dict(magnitude=65.0)), 1, "magnitude"),
    (dict(q=dict(heads=0)), 1, "q: heads"),
    (dict(k=dict(heads=0)), 1, "k: heads"),
    (dict(q=dict(x=None)), 1, "non-null"),
    (dict(q=dict(y=None)), 1, "non-null"),
    (dict(q=dict(x=FAKE + 8)), 1, "aligned"),
    (dict(q=dict(xs=(0, 65, 256))), 1, "multiples of 16"),
    (dict(q=dict(xs=(0, -64, 256))), 1, "strides"),
    (dict(q=dict(ys=(0, 64, 192))), 1, "overlap"),
    (dict(q=dict(ys=(0, 0, 256))), 1, "overlap"),
    (dict(q=dict(ys=(0, 64, 64))), 1, "overlap"),
    (dict(q=dict(xs=(0, 64, 1 << 62))), 1, "too large"),
    (dict(q=dict(y=FAKE, ys=(0, 64, 512))), 1, "share memory"),
    (dict(q=dict(y=FAKE + 128)), 1, "share memory"),
    (dict(norm=(FAKE + 2, None, 1e-6)), 1, "weight"),
    (dict(norm=(None, FAKE + 8, 1e-6)), 1, "weight"),
    (dict(norm=(None, None, -1.0)), 1, "eps"),
    (dict(norm=(None, None, math.nan)), 1, "eps"),
])
def test_rope_refuses(a, kw, code, msg):
    kw = dict(kw)
    for name, make in (("q", rows), ("k", rows), ("rot", rotation)):
        if name in kw:
            kw[name] = make(a, **kw[name])
    assert _rope(a, **kw) == code
    assert msg in a.last_error()


def test_rope_accepts_no_tokens(a):
    assert _rope(a, T=0, positions=None) == a.ATTN_OK
    assert _rope(a, B=0, positions=None) == a.ATTN_OK


def _append(a, e4m3, q=None, k="k", v="v", cu=FAKE, lens=FAKE, positions=None, table=FAKE, cache=FAKE, scales=FAKE,
            B=2, total=5, D=64, page=16, pages=4, blocks=8, rot=None, dtype=1):
    k = rows(a, y=None) if k == "k" else k
    v = rows(a, y=None) if v == "v" else v
    tail = (B, total, D, page, pages, blocks, rot, dtype, None)
    if e4m3:
        return a.lib.attn_append_paged_e4m3(q, k, v, cu, lens, positions, table, cache, scales, *tail)
    return a.lib.attn_append_paged(q, k, v, cu, lens, positions, table, cache, *tail)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=0), 2, "16-bit"),
    (dict(dtype=7), 1, "dtype"),
    (dict(B=0), 1, ">= 1"),
    (dict(total=-1), 1, ">= 0"),
    (dict(total=2 ** 31 - 1), 1, "total"),
    (dict(B=2 ** 31 - 1, pages=1), 1, "B and total"),
    (dict(k=dict(heads=2 ** 20 + 1, y=None), v=dict(heads=2 ** 20 + 1, y=None)), 1, "2^20"),
    (dict(page=0), 1, ">= 1"),
    (dict(blocks=0), 1, ">= 1"),
    (dict(D=80), 2, "D=80"),
    (dict(k=None), 1, "k and v"),
    (dict(v=None), 1, "k and v"),
    (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"),
    (dict(B=1 << 20, pages=1 << 12), 1, "31 bits"),
    (dict(rot=dict(rot=3)), 1, "rot_dim"),
    (dict(k=dict(heads=3, y=None)), 1, "same heads"),
    (dict(v=dict(heads=4)), 1, "v: y must be null"),
    (dict(q=dict(y=None)), 1, "q: x and y"),
    (dict(k=dict(y=None, x=FAKE + 2)), 1, "k: x and y must be 16-byte"),
    (dict(k=dict(ys=(0, 64, 0))), 1, "k: rows of y"),
    (dict(cu=None), 1, "non-null"), (dict(lens=None), 1, "non-null"), (dict(table=None), 1, "non-null"),
    (dict(cache=None), 1, "non-null"),
    (dict(cu=FAKE + 1), 1, "4-byte"), (dict(positions=FAKE + 2), 1, "4-byte"),
    (dict(cache=FAKE + 8), 1, "kv_cache"),
])
def test_append_refuses(a, e4m3, kw, code, msg):
    kw = dict(kw)
    for name, make in (("q", rows), ("k", rows), ("v", rows), ("rot", rotation)):
        if kw.get(name) is not None:
            kw[name] = make(a, **kw[name])
    assert _append(a, e4m3, **kw) == code
    assert msg in a.last_error()


def test_append_e4m3_needs_scales(a):
    assert _append(a, True, scales=None) == 1 and "scales" in a.last_error()
    assert _append(a, True, scales=FAKE + 2) == 1 and "4-byte" in a.last_error()
    assert _append(a, True, total=0, cu=None) == a.ATTN_OK


@pytest.mark.parametrize("kw,code,msg", [
    (dict(q=None), 1, "non-null"), (dict(scales=None), 1, "scales"), (dict(scales=FAKE + 1), 1, "scales"),
    (dict(kv=FAKE + 8), 1, "aligned"), (dict(dtype=0), 2, "16-bit"), (dict(dtype=9), 1, "dtype"),
    (dict(B=2 ** 31 - 1, Hq=1, Hkv=1, pages=1), 1, "B must be"),
    (dict(D=32), 2, "D=32"), (dict(Hq=5), 1, "multiple"), (dict(scale=0.0), 1, "scale"), (dict(B=0), 1, ">= 1"),
    (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"),
])
def test_decode_refuses(a, kw, code, msg):
    c = dict(q=FAKE, kv=FAKE, scales=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None, B=2, Hq=4, Hkv=2, D=64, page=16,
             pages=4, blocks=8, scale=0.1, dtype=1)
    c.update(kw)
    assert a.lib.attn_fwd_decode_paged_e4m3(
        c["q"], c["kv"], c["scales"], c["table"], c["lens"], c["o"], c["lse"], c["B"], c["Hq"], c["Hkv"], c["D"],
        c["page"], c["pages"], c["blocks"], c["scale"], c["dtype"], None) == code
    assert msg in a.last_error()


def test_binding_refuses_host_tensors(a):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        a.Rotation(torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError, match="int64"):
        a.Rotation(torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        a.attn_rope(x, None, torch.zeros(3, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="CUDA"):
        a.attn_append_paged(x, x, x, x, x, x)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        a.attn_append_paged_e4m3(x.float(), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        a.attn_fwd_decode_paged_e4m3(x[:, :, None], x, x, x, x)


def test_page_division_is_exact(a):
    """The kernels divide by the page size with one widening product: its arithmetic, here, over
    the divisors' and the numerators' borders."""
    for d in [1, 2, 3, 5, 7, 16, 24, 48, 255, 256, 257, 641, 4095, 65537, 2 ** 20 + 7, 2 ** 30 + 1, 2 ** 31 - 1025]:
        shift = 31 + (d - 1).bit_length()
        m = ((1 << shift) + d - 1) // d
        assert m < 2 ** 32
        ns = {0, 1, d - 1, d, d + 1, 2 ** 31 - 1, 2 ** 31 - 2}
        for q in (1, 2, 3, (2 ** 31 - 1) // d, (2 ** 31 - 1) // d - 1, (2 ** 31 - 1) // (2 * d)):
            ns |= {q * d - 1, q * d, q * d + 1}
        for n in ns:
            if 0 <= n < 2 ** 31:
                assert (n * m) >> shift == n // d, (n, d)
    assert ctypes.sizeof(a._Rows) == 72 and ctypes.sizeof(a._Rotation) == 24


def test_library_errors_come_as_the_bindings(a):
    """A status of the library, through the native calls, is the binding's exception."""
    with pytest.raises(a.AttnError) as e:
        a.rope_turns(7)
    assert e.value.status == a.ATTN_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="arguments"):
        a._native.rope(1)
    with pytest.raises(ValueError, match="q must be a tensor"):
        a.attn_rope([1.0], None, torch.zeros(1, dtype=torch.int32), None)


@pytest.mark.parametrize("rot", [2, 64, 128])
@pytest.mark.parametrize("base", [10000, 500000, 10 ** 15, 10 ** 19])
def test_tables_against_forty_digits(a, rot, base):
    """Within 2^-53 turns of base^(-2i/rot) / 2 pi: a double's pow (its exponent's rounding times
    ln base, at most 0.37 * 2^-53 of 1; an ulp, 2^-52), 2 pi and the division, 2^-52 * 1.93 / 2 pi;
    and where an entry is so small that this is less, within half a unit of 2^-64 of it."""
    import decimal
    with decimal.localcontext() as ctx:
        ctx.prec = 40
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510")
        for i, got in enumerate(a.rope_turns(rot, base=float(base))[0].tolist()):
            want = decimal.Decimal(base) ** (decimal.Decimal(-2 * i) / rot) / two_pi * 2 ** 64
            double = min(decimal.Decimal(2) ** 11, want * decimal.Decimal(2) ** -46)
            assert abs(got % 2 ** 64 - want) <= decimal.Decimal("0.5") + double, (i, got, want)
