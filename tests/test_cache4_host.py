"""What the calls of the 4-bit cache, of accumulated weights and of eviction refuse before
anything is launched (no GPU needed), and the plain forms their GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import kv4_ref

FAKE = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def a():
    from transformer_attention_fwd_gb300 import build
    build.build()
    from transformer_attention_fwd_gb300 import attn
    return attn


def rows(a, x=FAKE, y=None, heads=4, token=256, head=64):
    return ctypes.byref(a._Rows(x, y, heads, 0, head, token, 0, head, token))


def _append(a, **kw):
    c = dict(q=None, k=rows(a), v=rows(a), cu=FAKE, lens=FAKE, positions=None, table=FAKE, kv=FAKE, scales=FAKE,
             factors=None, B=2, total=5, D=64, page=16, pages=4, blocks=8, rot=None, dtype=1)
    c.update(kw)
    return a.lib.attn_append_paged_e2m1(c["q"], c["k"], c["v"], c["cu"], c["lens"], c["positions"], c["table"], c["kv"],
                                        c["scales"], c["factors"], c["B"], c["total"], c["D"], c["page"], c["pages"],
                                        c["blocks"], c["rot"], c["dtype"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=0), 2, "16-bit"), (dict(dtype=7), 1, "dtype"), (dict(B=0), 1, ">= 1"), (dict(total=-1), 1, ">= 0"),
    (dict(D=80), 2, "D=80"), (dict(k=None), 1, "k and v"), (dict(scales=None), 1, "scales"),
    (dict(scales=FAKE + 8), 1, "16-byte"), (dict(factors=FAKE + 2), 1, "factors"), (dict(kv=FAKE + 8), 1, "kv_cache"),
    (dict(cu=None), 1, "non-null"), (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"),
])
def test_append_refuses(a, kw, code, msg):
    assert _append(a, **kw) == code
    assert msg in a.last_error()


def test_append_accepts_no_tokens(a):
    assert _append(a, total=0, cu=None) == a.ATTN_OK


def _decode(a, **kw):
    c = dict(q=FAKE, kv=FAKE, scales=FAKE, factors=None, table=FAKE, lens=FAKE, o=FAKE, lse=None, weights=None, B=2,
             Hq=4, Hkv=2, D=64, page=16, pages=4, blocks=8, scale=0.1, dtype=1)
    c.update(kw)
    return a.lib.attn_fwd_decode_paged_e2m1(c["q"], c["kv"], c["scales"], c["factors"], c["table"], c["lens"], c["o"],
                                            c["lse"], c["weights"], c["B"], c["Hq"], c["Hkv"], c["D"], c["page"],
                                            c["pages"], c["blocks"], c["scale"], c["dtype"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(q=None), 1, "non-null"), (dict(scales=None), 1, "scales"), (dict(scales=FAKE + 4), 1, "scales"),
    (dict(factors=FAKE + 1), 1, "factors"), (dict(weights=FAKE + 2), 1, "weights"), (dict(kv=FAKE + 8), 1, "aligned"),
    (dict(dtype=0), 2, "16-bit"), (dict(dtype=9), 1, "dtype"), (dict(D=32), 2, "D=32"), (dict(Hq=5), 1, "multiple"),
    (dict(scale=0.0), 1, "scale"), (dict(scale=math.nan), 1, "scale"), (dict(B=0), 1, ">= 1"),
    (dict(B=2 ** 31 - 1, Hq=1, Hkv=1, pages=1), 1, "B must be"), (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"),
])
def test_decode_refuses(a, kw, code, msg):
    assert _decode(a, **kw) == code
    assert msg in a.last_error()


def test_decode_refuses_scores_beyond_any_memory(a):
    """Sizes whose product would pass 64 bits."""
    big = dict(B=1 << 12, Hq=1 << 18, Hkv=1 << 18, pages=1 << 17, page=(1 << 14) - 1)
    assert _decode(a, weights=FAKE, **big) == a.ATTN_ERR_NO_MEMORY and "2^44" in a.last_error()


def _weights(a, four, **kw):
    c = dict(q=rows(a), lse=FAKE, lse_head=5, lse_token=1, kv=FAKE, scales=FAKE, factors=None, table=FAKE, cu=FAKE,
             lens=FAKE, weights=FAKE, B=2, total=5, Hkv=2, D=64, page=16, pages=4, blocks=8, scale=0.1, dtype=1)
    c.update(kw)
    tail = (c["table"], c["cu"], c["lens"], c["weights"], c["B"], c["total"], c["Hkv"], c["D"], c["page"], c["pages"],
            c["blocks"], c["scale"], c["dtype"], None)
    if four:
        return a.lib.attn_weights_paged_e2m1(c["q"], c["lse"], c["lse_head"], c["lse_token"], c["kv"], c["scales"],
                                             c["factors"], *tail)
    return a.lib.attn_weights_paged(c["q"], c["lse"], c["lse_head"], c["lse_token"], c["kv"], *tail)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=0), 2, "16-bit"), (dict(dtype=7), 1, "dtype"), (dict(B=0), 1, ">= 1"), (dict(Hkv=0), 1, ">= 1"),
    (dict(total=-1), 1, "total"), (dict(D=96), 2, "D=96"), (dict(q=None), 1, "q must"), (dict(lse=None), 1, "lse"),
    (dict(lse=FAKE + 2), 1, "4-byte"), (dict(lse_head=-1), 1, "strides"), (dict(weights=None), 1, "non-null"),
    (dict(weights=FAKE + 1), 1, "4-byte"), (dict(kv=FAKE + 8), 1, "16-byte"), (dict(cu=None), 1, "cu_seqlens"),
    (dict(Hkv=3), 1, "multiple"), (dict(scale=-1.0), 1, "scale"), (dict(total=2 ** 29, Hkv=4), 1, "total*Hq"),
    (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"),
])
def test_weights_refuse(a, four, kw, code, msg):
    assert _weights(a, four, **kw) == code
    assert msg in a.last_error()


def test_weights_of_queries_with_outputs_are_refused(a):
    assert _weights(a, False, q=rows(a, y=FAKE)) == 1 and "y must be null" in a.last_error()
    assert _weights(a, False, q=rows(a, x=FAKE + 2)) == 1 and "16-byte" in a.last_error()
    assert _weights(a, True, scales=None) == 1 and "scales" in a.last_error()
    assert _weights(a, True, total=0, lse=None, cu=None) == a.ATTN_OK


def _evict(a, four, **kw):
    c = dict(kv=FAKE, scales=FAKE, weights=FAKE, table=FAKE, lens=FAKE, new=FAKE + 4096, kept=None, B=2, Hkv=2, D=64,
             page=16, pages=4, blocks=8, keep=5, recent=1, dtype=1)
    c.update(kw)
    tail = (c["weights"], c["table"], c["lens"], c["new"], c["kept"], c["B"], c["Hkv"], c["D"], c["page"], c["pages"],
            c["blocks"], c["keep"], c["recent"])
    if four:
        return a.lib.attn_evict_paged_e2m1(c["kv"], c["scales"], *tail, None)
    return a.lib.attn_evict_paged(c["kv"], *tail, c["dtype"], None)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(B=0), 1, ">= 1"), (dict(D=96), 2, "D=96"), (dict(keep=0), 1, "keep"), (dict(recent=6), 1, "recent"),
    (dict(recent=-1), 1, "recent"), (dict(keep=2 ** 31 - 1), 1, "keep"), (dict(new=None), 1, "new_lens"),
    (dict(pages=(2 ** 31 - 2048) // 16), 1, "max_pages_per_seq"),
    (dict(new=FAKE), 1, "seq_lens"), (dict(new=FAKE + 4), 1, "seq_lens"), (dict(kept=FAKE), 1, "share memory"),
    (dict(kept=FAKE + 4096 - 76), 1, "share memory"), (dict(table=FAKE + 4096, lens=FAKE + 8), 1, "share memory"), (dict(kept=FAKE + 2), 1, "4-byte"),
    (dict(weights=None), 1, "non-null"), (dict(kv=FAKE + 8), 1, "16-byte"), (dict(table=None), 1, "non-null"),
    (dict(pages=1 << 28), 1, "max_pages_per_seq*page_size"), (dict(B=1 << 20, Hkv=1 << 12), 1, "31 bits"),
])
def test_evict_refuses(a, four, kw, code, msg):
    assert _evict(a, four, **kw) == code
    assert msg in a.last_error()


def test_evict_refuses_lists_beyond_any_memory(a):
    assert _evict(a, False, B=1 << 12, Hkv=1 << 18, keep=1 << 30) == 1 and "2^42" in a.last_error()


def test_evict_refuses_types(a):
    assert _evict(a, False, dtype=0) == 2
    assert _evict(a, False, dtype=9) == 1
    assert _evict(a, True, scales=None) == 1 and "scales" in a.last_error()


def test_binding_refuses_host_tensors(a):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: a.attn_append_paged_e2m1(x, x, x, x, x, x, x),
                 lambda: a.attn_fwd_decode_paged_e2m1(x[:, :, None], x, x, x, x),
                 lambda: a.attn_weights_paged(x, x, x, x, x, x, x),
                 lambda: a.attn_weights_paged_e2m1(x, x, x, x, x, x, x, x),
                 lambda: a.attn_evict_paged(x, x, x, x, 5, 1),
                 lambda: a.attn_evict_paged_e2m1(x, x, x, x, x, 5, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: a.attn_append_paged_e2m1(x, x, x, None, x, x, x),
                 lambda: a.attn_weights_paged_e2m1(x, x, x, None, x, x, x, x),
                 lambda: a.attn_evict_paged_e2m1(x, None, x, x, x, 5, 1)):
        with pytest.raises(ValueError, match="scales"):
            call()


def test_plain_codes_round_to_nearest_even():
    y = torch.tensor([0.0, 0.25, 0.2501, 0.75, 0.7499, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 9.0, math.inf],
                     dtype=torch.float64)
    want = torch.tensor([0.0, 0.0, 0.5, 1.0, 0.5, 1.0, 1.5, 2.0, 2.0, 3.0, 4.0, 3.0, 4.0, 6.0, 6.0, 6.0],
                        dtype=torch.float64)
    assert torch.equal(kv4_ref.values(kv4_ref.e2m1(y)), want)
    assert torch.equal(kv4_ref.values(kv4_ref.e2m1(-y)), -want)
    codes = torch.arange(16)
    assert torch.equal(kv4_ref.e2m1(kv4_ref.values(codes)), codes)
    assert torch.equal(kv4_ref.unpack(kv4_ref.pack(codes)), codes)


def test_plain_quantisation_stays_within_its_steps():
    """No element is off by more than half the largest step (1 of 6) times the group's scale,
    and half an e4m3 step (2^-4) of the largest where the scale was rounded down."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 2, 3, 64, generator=g)
    f = 0.01 + torch.rand(2, 3, generator=g)
    codes, scale = kv4_ref.quantise(x, f[..., None])
    back = kv4_ref.values(codes) * (scale * f[..., None]).double().repeat_interleave(16, dim=-1)
    most = x.unflatten(-1, (-1, 16)).abs().amax(dim=-1).repeat_interleave(16, dim=-1).double()
    assert ((back - x).abs() <= most * (1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -20)).all()


def test_plain_eviction_by_hand():
    rows = torch.arange(10).reshape(1, 1, 1, 10, 1).expand(1, 2, 1, 10, 1).clone()
    w = torch.tensor([5.0, 1.0, 7.0, 7.0, math.nan, 0.0, 7.0, 2.0, 0.0, 0.0]).reshape(1, 1, 10)
    (pool,), weights, new, kept = kv4_ref.evict([rows], w, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([9]), 5, 2)
    assert kept.flatten().tolist() == [2, 3, 6, 7, 8] and new.tolist() == [5]
    assert pool[0, 0, 0, :, 0].tolist() == [2, 3, 6, 7, 8, 5, 6, 7, 8, 9]
    assert weights.flatten().tolist() == [7.0, 7.0, 7.0, 2.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]
