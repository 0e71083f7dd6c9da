"""Per-head norm with rotation on the GPU against 64 bits.

Tolerance: the float32 chain (sum of squares, rsqrt, three products, one sum) is
below 2^-20 of |n_a| + |n_b| for the pair; the store rounds by at most 2^-8 (bf16)."""
import pytest
import torch

from hybrid_testutil import rope_reference

pytestmark = pytest.mark.gpu


def _tables(P, rot):
    f = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _inputs(T, Hq, Hkv, d, rot, dtype, packed, P=5000, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    x = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(dtype)
    q, k = x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, P, (T,), generator=g).to(torch.int32)
    return x, q, k, 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g), pos, *_tables(P, rot)


def _ok(got, ref, size, dtype):
    bound = 2.0 ** -20 * size + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 2.0 ** -24 * ref.abs()) + 1e-30
    assert ((got.double().cpu() - ref).abs() <= bound).all(), ((got.double().cpu() - ref).abs() / bound).max()


@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [
    (1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (7, 4, 2, 128, 32), (33, 3, 3, 80, 48), (2, 2, 1, 256, 256),
    (5, 6, 2, 16, 16), (9, 7, 1, 200, 64), (700, 16, 4, 128, 128), (9000, 24, 8, 128, 64),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved,packed,weights", [(False, True, True), (True, False, True), (False, False, False)])
def test_norm_rope(kda_lib, cuda_dev, T, Hq, Hkv, d, rot, dtype, interleaved, packed, weights):
    import serving_kda_chunked_gated_gb300.kda as kda
    x, q, k, qw, kw, pos, cos, sin = _inputs(T, Hq, Hkv, d, rot, dtype, packed)
    if not weights:
        qw = kw = None
    n = min(T, 1200)                          # a long batch is checked at its first and last tokens
    at = torch.cat([torch.arange(n // 2), torch.arange(T - (n - n // 2), T)])
    xd = x.to(cuda_dev)
    dq = xd[:, :Hq * d].unflatten(1, (Hq, d))
    dk = xd[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    if not packed:
        dq, dk = dq.contiguous(), dk.contiguous()
    to = lambda t: None if t is None else t.to(cuda_dev)                     # noqa: E731
    yq, yk = kda.qk_norm_rope(dq, dk, to(cos), to(sin), to(pos), q_weight=to(qw), k_weight=to(kw), interleaved=interleaved)
    for got, src, w in ((yq, q, qw), (yk, k, kw)):
        ref, size = rope_reference(src[at], w, cos, sin, pos[at], interleaved)
        _ok(got[at.to(cuda_dev)], ref, size, dtype)


def test_in_place_and_one_weight(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    _, q, k, qw, _, pos, cos, sin = _inputs(37, 6, 2, 128, 64, torch.bfloat16, False)
    a, b = q.to(cuda_dev), k.to(cuda_dev)
    qo, ko = kda.qk_norm_rope(a, b, cos.to(cuda_dev), sin.to(cuda_dev), pos.to(cuda_dev), q_weight=qw.to(cuda_dev), out=(a, b))
    assert qo is a and ko is b
    for got, src, w in ((a, q, qw), (b, k, None)):
        ref, size = rope_reference(src, w, cos, sin, pos, False)
        _ok(got, ref, size, torch.bfloat16)


def test_far_positions_and_skipped_ones(kda_lib, cuda_dev):
    """Positions of the table's end are exact (the angles come from the table); positions outside leave their rows."""
    import serving_kda_chunked_gated_gb300.kda as kda
    P = 300000
    _, q, k, qw, kw, pos, cos, sin = _inputs(6, 2, 1, 64, 64, torch.float32, False, P=P)
    pos = torch.tensor([P - 1, P, -1, 0, 2 ** 31 - 1, P - 2], dtype=torch.int32)
    qo, ko = torch.full_like(q, 5.0).to(cuda_dev), torch.full_like(k, 5.0).to(cuda_dev)
    kda.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), cos.to(cuda_dev), sin.to(cuda_dev), pos.to(cuda_dev),
                     q_weight=qw.to(cuda_dev), k_weight=kw.to(cuda_dev), out=(qo, ko))
    on = torch.tensor([0, 3, 5])
    for got, src, w in ((qo, q, qw), (ko, k, kw)):
        ref, size = rope_reference(src[on], w, cos, sin, pos[on], False)
        _ok(got.cpu()[on], ref, size, torch.float32)
        assert (got.cpu()[[1, 2, 4]] == 5.0).all()


def test_zero_row_and_empty(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    cos, sin = (x.to(cuda_dev) for x in _tables(10, 32))
    z = torch.zeros(2, 3, 64, device=cuda_dev)
    qo, ko = kda.qk_norm_rope(z, z[:, :1].contiguous(), cos, sin, torch.zeros(2, dtype=torch.int32, device=cuda_dev))
    assert (qo == 0).all() and (ko == 0).all()
    e = torch.zeros(0, 3, 64, device=cuda_dev)
    qo, ko = kda.qk_norm_rope(e, e, cos, sin, torch.zeros(0, dtype=torch.int32, device=cuda_dev))
    assert qo.shape == (0, 3, 64)


@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [
    (6000, 5, 1, 64, 64), (5000, 7, 5, 64, 32), (4000, 8, 2, 48, 16), (3000, 5, 1, 128, 128), (3000, 7, 5, 128, 64),
    (2500, 6, 2, 128, 128), (2500, 13, 3, 96, 32), (3000, 16, 8, 128, 128), (1500, 5, 1, 256, 256), (1500, 7, 5, 256, 64),
    (1200, 14, 6, 200, 48), (2000, 0, 9, 128, 128), (2000, 9, 0, 64, 64),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_long_batches_with_partial_head_groups(kda_lib, cuda_dev, T, Hq, Hkv, d, rot, dtype, interleaved):
    """Batches long enough that a lane group takes four or eight heads (all widths), head counts that
    leave the last group of q or k partly empty: every row, and nothing behind the outputs."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator(device=cuda_dev).manual_seed(T + d)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_dev)                         # noqa: E731
    x = r(T, (Hq + Hkv) * d).to(dtype)
    heads = lambda y, H: y.unflatten(1, (H, d)) if H else y.new_empty(T, 0, d)           # noqa: E731
    q, k = heads(x[:, :Hq * d], Hq), heads(x[:, Hq * d:], Hkv)
    pos = torch.randint(0, 900, (T,), generator=g, device=cuda_dev).to(torch.int32)
    cos, sin = (t.to(cuda_dev) for t in _tables(900, rot))
    qw, kw = 1 + 0.2 * r(d), 1 + 0.2 * r(d)
    room = [torch.full(((T * H + 16) * d,), 7.0, dtype=dtype, device=cuda_dev) for H in (Hq, Hkv)]
    out = tuple(b[:T * H * d].view(T, H, d) for b, H in zip(room, (Hq, Hkv)))
    kda.qk_norm_rope(q, k, cos, sin, pos, q_weight=qw, k_weight=kw, interleaved=interleaved, out=out)
    assert all((b[T * H * d:] == 7.0).all() for b, H in zip(room, (Hq, Hkv)))
    for got, src, w in ((out[0], q, qw), (out[1], k, kw)):
        if src.shape[1]:
            ref, size = rope_reference(src.cpu(), w.cpu(), cos.cpu(), sin.cpu(), pos.cpu(), interleaved)
            _ok(got, ref, size, dtype)
