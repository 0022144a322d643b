"""GPU parity of dit_attn_bwd / dit_attn_bwd_masked with the 64-bit formulas,
element by element within the bounds train_ref derives from the kernel's
roundings, plus differences of the forward pass, determinism, strided views,
captured replays and refusals."""
import math

import pytest
import torch

import train_ref as ref
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


def _inputs(B, Nq, Nkv, H, D, seed, scale_q=1.5):
    g = wl.generator(DEV, seed)

    def t(n, s=1.0):
        return (torch.randn((B, n, H, D), generator=g, device=DEV) * s).to(torch.bfloat16)
    return t(Nq, scale_q), t(Nkv), t(Nkv), t(Nq, 0.25), g


def _allow(B, Nq, Nkv, kvl, mask=None):
    a = torch.zeros((B, 1, Nq, Nkv), dtype=torch.bool, device=DEV)
    a[..., :kvl] = True
    if mask is not None:
        R = mask.shape[1]
        a[:, 0, :R, :kvl] &= mask[..., :kvl].to(DEV)
    return a


def _forward(q, k, v, scale, allow, out_dtype):
    o, lse = ref.attn_forward(q, k, v, scale, allow)
    return o.to(out_dtype).contiguous(), lse.float().contiguous()


def _check(grads, q, k, v, out, lse, dout, scale, allow, dlse=None):
    want = ref.attn_bwd(q, k, v, out, lse, dout, scale, allow, dlse, grads[0].dtype == torch.bfloat16)
    for name, g, (r, b) in zip(("dq", "dk", "dv"), grads, want):
        ref.check(g, r, b, name)


CASES = [(1, 1, 1, 1, 64), (1, 1, 257, 2, 128), (2, 130, 3, 1, 64), (1, 128, 128, 2, 128), (1, 129, 255, 3, 64),
         (2, 300, 511, 2, 128), (1, 1024, 1024, 2, 64), (1, 17, 2500, 1, 128), (3, 2111, 40, 1, 64), (1, 700, 1900, 5, 128)]


@pytest.mark.parametrize("B,Nq,Nkv,H,D", CASES)
@pytest.mark.parametrize("out_dtype,grad_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_matches_the_formulas(dl, B, Nq, Nkv, H, D, out_dtype, grad_dtype):
    q, k, v, dout, _ = _inputs(B, Nq, Nkv, H, D, 100 + Nq + Nkv)
    scale = D ** -0.5
    for kvl in sorted({Nkv, max(1, Nkv - 1), (Nkv + 1) // 2}):
        allow = _allow(B, Nq, Nkv, kvl)
        out, lse = _forward(q, k, v, scale, allow, out_dtype)
        kk, vv = k.clone(), v.clone()
        kk[:, kvl:] = float("nan")       # pad keys are never read
        vv[:, kvl:] = float("inf")
        grads = dl.attn_bwd(q, kk, vv, out, lse, dout, key_valid_len=kvl, grad_dtype=grad_dtype)
        torch.cuda.synchronize()
        _check(grads, q, k, v, out, lse, dout, scale, allow)
        assert (grads[1][:, kvl:] == 0).all() and (grads[2][:, kvl:] == 0).all()


def _mask(kind, B, R, Nk, g):
    i, j = torch.arange(R)[:, None], torch.arange(Nk)[None, :]
    if kind == "frames":
        m = (i // 100) == (j // 100)
    elif kind == "causal":
        m = j <= i
    elif kind == "random":
        m = torch.rand((R, Nk), generator=torch.Generator().manual_seed(R + Nk)) < 0.1
    else:   # "holes": rows with nothing, whole tiles of rows with nothing, one key only
        m = torch.rand((R, Nk), generator=torch.Generator().manual_seed(R)) < 0.5
        m[::7] = False
        m[128:min(R, 300)] = False
        m[-1] = False
        m[-1, Nk // 2] = True
    m = m[None].repeat(B, 1, 1).contiguous()
    if B > 1:
        m[1] = m[1].roll(3, 1)
    return m


@pytest.mark.parametrize("kind", ["frames", "causal", "random", "holes"])
@pytest.mark.parametrize("B,Nq,Nkv,H,D,rows,kvl", [(2, 300, 300, 2, 64, 300, 300), (1, 640, 640, 2, 128, 600, 600),
                                                   (1, 513, 1000, 1, 128, 513, 999), (2, 200, 77, 3, 64, 150, 70)])
def test_masked_matches_the_formulas(dl, kind, B, Nq, Nkv, H, D, rows, kvl):
    q, k, v, dout, g = _inputs(B, Nq, Nkv, H, D, 7 + Nq)
    m = _mask(kind, B, rows, kvl, g)
    allow = _allow(B, Nq, Nkv, kvl, m)
    scale = 0.11
    out, lse = _forward(q, k, v, scale, allow, torch.bfloat16)
    bits = wl.pack_mask_bits(m).to(DEV)
    grads = dl.attn_bwd_masked(q, k, v, out, lse, dout, bits, key_valid_len=kvl, scale=scale)
    torch.cuda.synchronize()
    _check(grads, q, k, v, out, lse, dout, scale, allow)
    empty = ~allow[:, 0].any(-1)
    assert (grads[0][empty] == 0).all()


def test_shared_mask_and_no_mask_rows(dl):
    B, N, H, D = 2, 260, 2, 64
    q, k, v, dout, g = _inputs(B, N, N, H, D, 9)
    m = _mask("causal", 1, N, N, g)
    allow = _allow(B, N, N, N, m.repeat(B, 1, 1))
    out, lse = _forward(q, k, v, D ** -0.5, allow, torch.bfloat16)
    bits = wl.pack_mask_bits(m).to(DEV)
    _check(dl.attn_bwd_masked(q, k, v, out, lse, dout, bits), q, k, v, out, lse, dout, D ** -0.5, allow)
    full = _allow(B, N, N, N)
    out, lse = _forward(q, k, v, D ** -0.5, full, torch.bfloat16)
    a = dl.attn_bwd_masked(q, k, v, out, lse, dout, bits, mask_rows=0)
    b = dl.attn_bwd(q, k, v, out, lse, dout)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_after_the_forward_call_and_against_differences(dl):
    """Gradients of sum(O dO) + sum(LSE dLSE) behind the library's own forward
    call, along random directions, against differences of the fp64 loss.  The
    bound: the elementwise bounds times |direction|, and the difference's own
    error (central, step 1e-4: third derivatives enter at 1e-8 of the loss'
    scale, rounding at 2^-53 / 1e-4)."""
    B, Nq, Nkv, H, D, kvl = 1, 140, 200, 2, 64, 190
    q, k, v, dout, g = _inputs(B, Nq, Nkv, H, D, 31)
    dlse = torch.randn((B, H, Nq), generator=g, device=DEV)
    out, lse = dl.attn_fwd(q, k, v, key_valid_len=kvl)
    grads = dl.attn_bwd(q, k, v, out, lse, dout, dlse=dlse, key_valid_len=kvl, grad_dtype=torch.float32)
    scale, allow = D ** -0.5, _allow(B, Nq, Nkv, kvl)
    _check(grads, q, k, v, out, lse, dout, scale, allow, dlse)
    # the forward call's own O and LSE instead of exact ones: what they change in the formulas
    exact_out, exact_lse = ref.attn_forward(q, k, v, scale, allow)
    near = ref.attn_bwd(q, k, v, out, lse, dout, scale, allow, dlse, False)
    true = ref.attn_bwd(q, k, v, exact_out, exact_lse, dout, scale, allow, dlse, False)

    def loss(a, b, c):
        o, l = ref.attn_forward(a, b, c, scale, allow)
        return float((o * dout.double()).sum() + (l * dlse.double()).sum())
    size = float((exact_out * dout.double()).abs().sum() + (exact_lse * dlse.double()).abs().sum())
    for i in range(3):
        d = torch.randn([q, k, v][i].shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-4
        args = [t.double() for t in (q, k, v)]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = float((grads[i].double() * d).sum())
        room = float(((near[i][1] + (near[i][0] - true[i][0]).abs()) * d.abs()).sum()) + 1e-6 * size
        assert abs(got - diff) <= room, (i, got, diff, room)
        assert abs(float((true[i][0] * d).sum()) - diff) <= 1e-6 * size      # the formulas themselves


def test_key_chunks_add_up(dl):
    """Ring-style training: the merged (O, LSE) with each key chunk's call gives
    that chunk's dK, dV and a share of dQ; the shares add to the whole."""
    B, N, H, D = 1, 500, 2, 128
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 41)
    allow = _allow(B, N, N, N)
    out, lse = _forward(q, k, v, D ** -0.5, allow, torch.float32)
    cuts = [0, 190, 300, 500]
    dq = torch.zeros((B, N, H, D), device=DEV)
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        x, y, z = dl.attn_bwd(q, k[:, a:b], v[:, a:b], out, lse, dout, grad_dtype=torch.float32)
        dq += x
        parts.append((y, z))
    dk, dv = (torch.cat([p[i] for p in parts], 1) for i in range(2))
    _check((dq, dk, dv), q, k, v, out, lse, dout, D ** -0.5, allow)


@pytest.mark.parametrize("D", [64, 128])
def test_fused_views_in_and_out_leave_the_rest_alone(dl, D):
    B, N, H, kvl = 2, 333, 3, 300
    qkv = wl.randn_bf16((B, N, 3, H, D), 51, DEV)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    dout = wl.randn_bf16((B, N, 2, H, D), 52, DEV)[:, :, 1]
    allow = _allow(B, N, N, kvl)
    out, lse = _forward(q, k, v, D ** -0.5, allow, torch.bfloat16)
    wide = torch.full((B, N + 5, 4, H, D), -7.0, dtype=torch.bfloat16, device=DEV)
    g = wide[:, :N, :3]
    grads = dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=kvl, dq=g[:, :, 0], dk=g[:, :, 1], dv=g[:, :, 2])
    torch.cuda.synchronize()
    _check(grads, q, k, v, out, lse, dout, D ** -0.5, allow)
    assert (wide[:, N:] == -7.0).all() and (wide[:, :, 3] == -7.0).all()


def test_no_keys_no_queries(dl):
    B, H, D = 2, 2, 64
    q, k, v, dout, _ = _inputs(B, 50, 30, H, D, 61)
    out = torch.zeros((B, 50, H, D), device=DEV)
    lse = torch.full((B, H, 50), -math.inf, device=DEV)
    for g in dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=0):
        assert (g == 0).all()
    dq, dk, dv = dl.attn_bwd(q[:, :0], k, v, out[:, :0], lse[..., :0].contiguous(), dout[:, :0])
    assert dq.numel() == 0 and (dk == 0).all() and (dv == 0).all()


def test_repeats_bit_for_bit_alone_and_captured(dl):
    B, N, H, D = 1, 900, 3, 128          # few items: cut into pieces and summed
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 71)
    out, lse = _forward(q, k, v, D ** -0.5, _allow(B, N, N, N), torch.bfloat16)
    first = dl.attn_bwd(q, k, v, out, lse, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = dl.attn_bwd(q, k, v, out, lse, dout, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    grads = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(dl.attn_bwd_workspace_bytes(B, N, N, H, D, N), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        dl.attn_bwd(q, k, v, out, lse, dout, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
    for _ in range(3):
        for t in grads:
            t.fill_(float("nan"))
        ws.fill_(0xFF)                    # nothing kept from one call for the next
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, grads))


def test_scores_far_from_zero(dl):
    """LSE of several thousands: P comes from differences of large numbers."""
    B, N, H, D = 1, 200, 1, 64
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 81, scale_q=60.0)
    allow = _allow(B, N, N, N)
    out, lse = _forward(q, k, v, 2.0, allow, torch.float32)
    assert float(lse.abs().max()) > 2000
    _check(dl.attn_bwd(q, k, v, out, lse, dout, scale=2.0), q, k, v, out, lse, dout, 2.0, allow)


def test_longer_than_the_ring(dl):
    """Every barrier goes round many times; sampled heads against the formulas."""
    B, N, H, D = 1, 4200, 8, 128
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 91)
    allow = _allow(B, N, N, 4133)
    out, lse = _forward(q, k, v, D ** -0.5, allow, torch.bfloat16)
    grads = dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=4133)
    for h in (0, 5):
        s = slice(h, h + 1)
        _check([g[:, :, s] for g in grads], q[:, :, s], k[:, :, s], v[:, :, s], out[:, :, s], lse[:, s], dout[:, :, s],
               D ** -0.5, allow)


@pytest.mark.parametrize("D,grad_dtype", [(64, torch.bfloat16), (128, torch.float32), (128, torch.bfloat16)])
def test_last_query_items_cut(dl, D, grad_dtype):
    """256 key and 256 query items on 152 SMs: the last query items run in pieces
    (the workspace then holds more than the statistics and the counter)."""
    B, N, H, kvl = 1, 4070, 8, 4001
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 93)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert dl.attn_bwd_workspace_bytes(B, N, N, H, D, kvl) > H * 2 * 32 * 128 * 4 + 512
    scale, allow = D ** -0.5, _allow(B, N, N, kvl)
    out, lse = _forward(q, k, v, scale, allow, torch.bfloat16)
    grads = dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=kvl, grad_dtype=grad_dtype)
    for h in (0, 4, 5, 6, 7):
        s = slice(h, h + 1)
        _check([g[:, :, s] for g in grads], q[:, :, s], k[:, :, s], v[:, :, s], out[:, :, s], lse[:, s], dout[:, :, s], scale, allow)
    again = dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=kvl, grad_dtype=grad_dtype)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    # a mask over the same rows: none of them is cut
    m = torch.ones((1, N, kvl), dtype=torch.bool)
    bits = wl.pack_mask_bits(m).to(DEV)
    masked = dl.attn_bwd_masked(q, k, v, out, lse, dout, bits, key_valid_len=kvl, grad_dtype=grad_dtype)
    assert torch.equal(masked[1], grads[1]) and torch.equal(masked[2], grads[2])
    _check([g[:, :, 7:] for g in masked], q[:, :, 7:], k[:, :, 7:], v[:, :, 7:], out[:, :, 7:], lse[:, 7:], dout[:, :, 7:], scale, allow)


def test_refusals(dl):
    from dit_long_sequence_gb300 import binding as E
    B, N, H, D = 1, 64, 2, 64
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 95)
    out, lse = dl.attn_fwd(q, k, v)

    def status(fn):
        with pytest.raises(dl.DitError) as e:
            fn()
        torch.cuda.synchronize()
        return e.value.status
    assert status(lambda: dl.attn_bwd(q, k, v, out, lse, dout[:, :1].expand(B, N, H, D))) == E.DIT_ERR_INVALID_ARG
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    assert status(lambda: dl.attn_bwd(q, k, v, out, lse, dout, workspace=small)) == E.DIT_ERR_INVALID_ARG
    host = torch.zeros((B, N, H, D), dtype=torch.bfloat16, pin_memory=True)
    dq = torch.empty_like(q)
    assert status(lambda: dl.attn_bwd(q, k, v, out, lse, dout, dq=dq, dk=host, dv=torch.empty_like(q))) == E.DIT_ERR_INVALID_ARG
    assert (host == 0).all()
    assert status(lambda: dl.attn_bwd(q, k, v, out, lse, dout, scale=-1.0)) == E.DIT_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        dl.attn_bwd(q, k, v, out, lse, dout.float())
    with pytest.raises(ValueError):
        dl.attn_bwd(q, k, v, out, lse[:, :, :-1], dout)
    with pytest.raises(ValueError):
        dl.attn_bwd_masked(q, k, v, out, lse, dout, torch.zeros((3, N, 4), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        dl.attn_bwd_masked(q, k, v, out, lse, dout, torch.zeros((1, N, 3), dtype=torch.int32, device=DEV))
