"""Sizes of a paged cache's batch that the calls refuse, without a GPU."""
import pytest

from test_cache_cpu import _append, _fwd, lib  # noqa: F401


@pytest.mark.parametrize("B", [(1 << 29) + 1, (1 << 31) - 1])
def test_too_many_sequences(lib, B):  # noqa: F811
    """The kernels count sequences, and one more, in 32 bits."""
    assert _append(lib, B=B) == _fwd(lib, B=B) == lib.ATTN_ERR_TOO_LARGE
    assert lib.attn_cache_fwd_workspace_bytes(5, B, 4, 2, 64) == lib.ATTN_ERR_TOO_LARGE
