"""What the weights of a paged cache refuse beyond test_cache4_host.py (no GPU needed)."""
import pytest

from test_cache4_host import _weights, a  # noqa: F401  (a fixture)


@pytest.mark.parametrize("four", [False, True])
def test_requests_whose_numbers_would_wrap_are_refused(a, four):  # noqa: F811
    """Blocks of a launch step over up to 65535 requests at a time."""
    for B in (2 ** 31 - 65536, 2 ** 31 - 1):
        assert _weights(a, four, B=B, Hkv=1, pages=1) == a.ATTN_ERR_INVALID_ARG
        assert "B must be" in a.last_error()
    assert _weights(a, four, B=2 ** 31 - 65537, Hkv=1, pages=1, total=0) == a.ATTN_OK
