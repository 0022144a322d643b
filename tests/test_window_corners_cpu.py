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


def test_workspace_functions_refuse_windows_that_the_calls_refuse(lib):  # noqa: F811
    """A negative bound is a ValueError there as in the calls, not a window without it."""
    asks = (lambda **w: lib.attn_fwd_window_workspace_bytes(1, 300, 4, 2, 64, 300, **w),
            lambda **w: lib.attn_bwd_window_workspace_bytes(1, 300, 300, 4, 2, 64, 300, **w),
            lambda **w: lib.attn_fwd_paged_workspace_bytes(1, 1, 4, 2, 64, 16, 400, **w))
    for ask in asks:
        for w in (dict(left=-1), dict(right=-1), dict(left=-2 ** 31), dict(sinks=-1), dict(frame=0), dict(left=2 ** 32), dict(sinks=2 ** 31)):
            with pytest.raises(ValueError):
                ask(**w)
        assert ask(left=None, right=None) >= 0 and ask(left=2 ** 31 - 1, right=2 ** 31 - 1, sinks=2 ** 31 - 1, frame=2 ** 30) >= 0
