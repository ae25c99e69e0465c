"""What the weights of a paged cache refuse beyond test_cache4_host.py (no GPU needed)."""
import pytest

from test_cache4_host import _evict, _weights, a  # noqa: F401  (a fixture)


@pytest.mark.parametrize("four", [False, True])
def test_requests_whose_numbers_would_wrap_are_refused(a, four):  # noqa: F811
    """Blocks of a launch step over up to 65535 requests at a time."""
    for B in (2 ** 31 - 65536, 2 ** 31 - 1):
        assert _weights(a, four, B=B, Hkv=1, pages=1) == a.ATTN_ERR_INVALID_ARG
        assert "B must be" in a.last_error()
    assert _weights(a, four, B=2 ** 31 - 65537, Hkv=1, pages=1, total=0) == a.ATTN_OK


@pytest.mark.parametrize("four", [False, True])
def test_evictions_refuse_tensors_that_meet(a, four):  # noqa: F811
    """Each that is written with every other, at its first and its last byte."""
    G = 1 << 32
    place = dict(kept=1 * G, new=2 * G, weights=3 * G, kv=4 * G, scales=5 * G, lens=6 * G, table=7 * G)
    B, Hkv, D, page, pages, blocks, keep = 3, 2, 64, 16, 4, 8, 5
    size = dict(kept=4 * B * Hkv * keep, new=4 * B, weights=4 * blocks * Hkv * page, lens=4 * B, table=4 * B * pages,
                kv=2 * blocks * Hkv * page * (D // 2 if four else 2 * D), scales=2 * blocks * Hkv * page * D // 16)
    shape = dict(B=B, Hkv=Hkv, D=D, page=page, pages=pages, blocks=blocks, keep=keep)
    written = ["kept", "new", "weights", "kv"] + ["scales"] * four

    def refused(**kw):
        code = _evict(a, four, **{**shape, **place, **kw})
        return code == a.ATTN_ERR_INVALID_ARG and "share memory" in a.last_error()

    for x in written:
        for y in written + ["lens", "table"]:
            if x == y:
                continue
            step = 16 if {x, y} & {"kv", "scales"} else 4
            assert refused(**{x: place[y]}), (x, y)
            if x not in ("kv", "scales"):  # 16-byte aligned: up to the other's last bytes
                assert refused(**{x: place[y] + size[y] - 4}), (x, y)
            assert refused(**{x: place[y] - (size[x] - 4) // step * step}), (x, y)
    huge = dict(blocks=2 ** 31 - 1, page=2 ** 31 - 70000, pages=1)  # more than 64 bits of bytes
    assert _evict(a, four, **{**shape, **place, **huge}) == a.ATTN_ERR_INVALID_ARG
