"""Windowed attention and the paged cache at their corners on the GPU: no query heads,
many heads to a K/V head, queries before the first key, what nobody sees."""
import pytest
import torch

from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


def rand(shape, seed, s=1.0):
    return (torch.randn(shape, generator=wl.generator(DEV, seed), device=DEV) * s).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_without_query_heads_are_zeros(dl, dtype):
    B, N, Hkv, D = 2, 300, 3, 64
    q, kv = rand((B, N, 0, D), 1), rand((B, N, Hkv, D), 2)
    out, lse = dl.attn_fwd_window(q, kv, kv, left=5)
    assert out.shape == (B, N, 0, D) and lse.shape == (B, 0, N)
    dk, dv = (torch.full((B, N, Hkv, D), 9.0, dtype=dtype, device=DEV) for _ in range(2))
    for given in (dict(dk=dk, dv=dv), dict(grad_dtype=dtype)):
        grads = dl.attn_bwd_window(q, kv, kv, out, lse, q, left=5, sinks=2, **given)
        torch.cuda.synchronize()
        assert grads[0].shape == q.shape and all(g.dtype == dtype and (g == 0).all() for g in grads[1:])
