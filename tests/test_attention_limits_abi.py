"""Limits of the attention entry points that keep every index of theirs in an int (CPU)."""
import pytest

from test_attention_abi import BAD, UNS, L, append, attend, desc, gather  # noqa: F401


@pytest.mark.parametrize("call", [append, attend, gather])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_longest_sequences(L, call, page):  # noqa: F811
    """The end of a sequence's last tile, 127 keys on, is an int too."""
    for tokens in (2 ** 31 - page, 2 ** 31 - 1024):
        assert call(L, desc(page=page, max_pages=tokens // page)) == UNS
    assert call(L, desc(page=page, max_pages=(2 ** 31 - 1024) // page - 1), ws=None) == BAD   # (of the shapes, nothing)
