"""Calls on a stream that is not the current one: what they allocate must not be memory
that work queued on the current stream still uses."""
import pytest
import torch

from gpu_util import attn, check_status

pytestmark = pytest.mark.gpu


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).cuda()


def _append(a, e4m3):
    n, pages = 2048, 128
    k, v, q = _randn(n, 2, 128), _randn(n, 2, 128), _randn(n, 4, 128)
    table, cu, lens = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous(), _ints(0, n), _ints(n)
    rotation = a.Rotation.make(128)
    if e4m3:
        cache = torch.zeros(pages, 2, 2, 16, 128, device="cuda").to(torch.float8_e4m3fn)
        scales = torch.ones(pages, 2, 2, device="cuda")
        return lambda s: a.attn_append_paged_e4m3(k, v, cache, scales, table, cu, lens, rotation, q=q, stream=s)[:1]
    cache = torch.zeros(pages, 2, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    return lambda s: a.attn_append_paged(k, v, cache, table, cu, lens, rotation, q=q, stream=s)[:1]


def _paged(a, e4m3):
    B, pages = 64, 4
    q = _randn(B, 128, 1, 128)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    lens = torch.full((B,), 60, dtype=torch.int32, device="cuda")
    cache = _randn(B * pages, 2, 8, 16, 128)
    if e4m3:
        scales = torch.full((B * pages, 2, 8), 0.5, device="cuda")
        codes = cache.to(torch.float8_e4m3fn)
        return lambda s: a.attn_fwd_decode_paged_e4m3(q, codes, scales, table, lens, stream=s)
    return lambda s: a.attn_fwd_decode_paged(q, cache, table, lens, stream=s)


def _calls(a):
    x, y = _randn(2048, 4, 128), _randn(2048, 2, 128)
    pos, rotation = torch.arange(2048, dtype=torch.int32, device="cuda"), a.Rotation.make(128)
    q, kv, q1 = _randn(2, 8, 512, 128), _randn(2, 2, 512, 128), _randn(64, 32, 1, 128)
    kv1 = _randn(64, 8, 33, 128)
    cu = _ints(0, 700, 2048)
    return {
        "rope": lambda s: a.attn_rope(x, y, pos, rotation, stream=s),
        "norm": lambda s: a.attn_qk_norm_rope(x, y, None, None, pos, rotation, stream=s),
        "append": _append(a, False),
        "append e4m3": _append(a, True),
        "decode e4m3": _paged(a, True),
        "decode paged": _paged(a, False),
        "fwd": lambda s: a.attn_fwd(q, kv, kv, causal=True, stream=s),
        "prefill": lambda s: a.attn_fwd_prefill(q, kv, kv, stream=s),
        "window": lambda s: a.attn_fwd_window(q, kv, kv, 64, stream=s),
        "decode": lambda s: a.attn_fwd_decode(q1, kv1, kv1, stream=s),
        "varlen": lambda s: a.attn_fwd_varlen(x, y, y, cu, cu, True, stream=s),
    }


@pytest.mark.parametrize("name", ["rope", "norm", "append", "append e4m3", "decode e4m3", "decode paged", "fwd",
                                  "prefill", "window", "decode", "varlen"])
def test_outputs_on_a_given_stream_are_its_own(name):
    a = attn()
    call = _calls(a)[name]
    want = [t.clone() for t in call(None)]
    shapes = [(t.shape, t.dtype) for t in want]
    other = torch.cuda.Stream()
    call(other)  # whatever is set up once
    torch.cuda.synchronize()
    # Blocks of the outputs' sizes, freed while writes to them wait behind a delay of some 25 ms.
    blocks = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda._sleep(50_000_000)
    for b in blocks:
        b.fill_(7.0)
    at = {b.data_ptr() for b in blocks}
    del blocks, b
    got = call(other)
    assert not at & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    check_status(a)


def test_the_default_stream_by_its_handle():
    """A stream object whose handle is 0, and one known by its handle alone."""
    a = attn()
    x, pos, rotation = _randn(64, 4, 128), torch.arange(64, dtype=torch.int32, device="cuda"), a.Rotation.make(128)
    want, _ = a.attn_rope(x, None, pos, rotation)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (torch.cuda.default_stream(), torch.cuda.ExternalStream(side.cuda_stream)):
        got, _ = a.attn_rope(x, None, pos, rotation, stream=s)
        o, _ = a.attn_fwd(x[None], x[None], x[None], stream=s)
        s.synchronize()
        assert torch.equal(got, want) and torch.isfinite(o).all()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
