"""Host-side corners of windowed attention and the paged cache (no GPU needed): calls
without query heads, limits that the header states, the workspace functions' checks."""
import pytest

from test_window_abi_cpu import _append, _bwd, _fwd, _paged, deviceless, lib  # noqa: F401  (lib: the fixture)


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


@deviceless
def test_limits_that_the_header_states(lib):  # noqa: F811
    """Just above each limit DIT_ERR_UNSUPPORTED, at it the call goes on (to the device)."""
    U = lib.DIT_ERR_UNSUPPORTED
    S = lib.Strides4
    # B * T * Hkv * D below 2^33
    wide = dict(sk=S(1 << 30, 4096, 128, 1), sv=S(1 << 30, 4096, 128, 1), Hkv=32, D=128)
    assert _append(lib, B=1, T=1 << 21, **wide) == U and _append(lib, B=1, T=(1 << 21) - 1, **wide) not in (U, lib.DIT_OK)
    assert _append(lib, B=65536) == U and _append(lib, B=65535) != U
    assert _append(lib, T=(1 << 29) + 1, B=1, Hkv=1, D=8) == U and _append(lib, T=1 << 29, B=1, Hkv=1, D=8) != U
    # page_size * table_width at most 2^31 - 256, pages below 2^31 - 1
    for call in (_append, _paged):
        assert call(lib, c=dict(page=8, width=(1 << 28) - 31)) == U and call(lib, c=dict(page=8, width=(1 << 28) - 32)) != U
        assert call(lib, c=dict(pages=(1 << 31) - 1)) == U and call(lib, c=dict(pages=(1 << 31) - 2)) != U
    # B * Hkv * ceil(T / n), n = 2 * floor(128 / (H / Hkv)), at most 2^31 - 16
    st = S(1 << 20, 1 << 10, 128, 1)

    def fwd(B, T, H, Hkv):
        return _fwd(lib, B=B, Nq=T, H=H, Hkv=Hkv, st=dict(q=st, o=st, k=st, v=st))

    def paged(B, T, H, Hkv):
        return _paged(lib, B=B, T=T, H=H, Hkv=Hkv, sq=st, so=st)
    for call in (fwd, paged):
        assert call(65535, 256, 32768, 32768) != U and call(65535, 257, 32768, 32768) == U      # 2^31 - 2^15, twice that
        assert call(65535, 2, 32768, 256) != U and call(65535, 2 * 128, 32768, 256) != U        # one token a tile: n = 2
        assert call(65535, 2 * 129, 32768, 256) == U                                            # 65,535 * 256 * 129
