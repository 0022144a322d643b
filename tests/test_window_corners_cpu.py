"""Host-side corners of windowed attention and the paged cache (no GPU needed): calls
without query heads, limits that the header states, the workspace functions' checks."""
import pytest

from test_window_abi_cpu import _append, _bwd, _paged, deviceless, lib  # noqa: F401  (lib: the fixture)


@deviceless
def test_gradients_without_query_heads_are_written(lib):  # noqa: F811
    """H = 0 with K/V heads: dk and dv are sums over nothing, zeros that must be written, so
    the call needs them and does not end early; without K/V heads there is nothing."""
    assert _bwd(lib, H=0, Hkv=2, dk=None) == lib.DIT_ERR_INVALID_ARG
    assert _bwd(lib, H=0, Hkv=2, q=None, o=None, lse=None, do=None, dq=None, ws=None, wsb=0) == lib.DIT_ERR_CUDA   # (as far as the device)
    assert _bwd(lib, H=0, Hkv=2, Nq=-1) == lib.DIT_ERR_INVALID_ARG
    assert _bwd(lib, H=0, Hkv=0, dk=None, dv=None) == lib.DIT_OK
    assert _bwd(lib, H=0, Hkv=2, Nkv=0, kvl=0, dk=None, dv=None) == lib.DIT_OK
