"""The one-token step where no unit (a sequence with some of its key heads) is cut: batches of many short sequences under narrow page
tables, units spread over the workers by where they start in the list, one launch and no join.  Against the plain 64-bit form, with empty
and skipped sequences among the others, units in plenty and in want of workers, one worker to a CTA and eight."""
import pytest
import torch

import paged_testutil
from paged_testutil import E4M3, Cache, attention, check_lse, check_out, rand_rows

BF = torch.bfloat16
STEP = {"bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}      # rounding of the step's weights


def _lens(n, most, holes):
    """n lengths of 1 .. most in a scattered order; holes: every 7th sequence is empty, every 11th skipped (None)."""
    lens = [1 + (i * 7919) % most for i in range(n)]
    if holes:
        lens = [None if i % 11 == 3 else 0 if i % 7 == 2 else x for i, x in enumerate(lens)]
    return lens


def _quantise(x):
    """``paged_testutil.quantise`` with the exponent from the largest magnitude's own: hundreds of small sequences are made here."""
    x = x.double()
    fine = torch.isfinite(x).all(-1)
    y = torch.where(fine[..., None], x, torch.zeros_like(x))
    a = y.abs().amax(-1)
    m, ex = torch.frexp(a)
    e = torch.where(a > 0, ex - 9 + (m > 0.875).to(ex.dtype), torch.full_like(ex, -100)).clamp(-100, 119)
    z = torch.ldexp(y.abs(), -e[..., None])
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    up, down = torch.searchsorted(mid, z, right=True), torch.searchsorted(mid, z)
    i = torch.where(up % 2 == 0, up, down)
    codes = (i + 128 * torch.signbit(y)).to(torch.uint8)
    return codes, torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def test_the_quick_form_of_the_8_bit_rows():
    g = torch.Generator().manual_seed(40)
    x = torch.randn(400, 2, 64, generator=g) * 2.0 ** torch.randint(-110, 120, (400, 2, 1), generator=g)
    x[0, 0], x[1, 1], x[2, 0, 3] = 0, 448.0, float("inf")
    for a, b in zip(_quantise(x.to(BF)), paged_testutil.quantise(x.to(BF))):
        assert torch.equal(a, b)


# sequences, longest, query and key heads, d, page, tables' width in pages
BATCHES = [
    (400, 48, 8, 8, 128, 16, 4),        # a worker of 8 warps to a CTA: 152 of them, several units each
    (450, 48, 9, 3, 64, 16, 4),         # a warp to a worker, three groups of heads: more units than workers
    (256, 64, 32, 8, 128, 64, 2),       # 8 tiles a sequence at most
    (100, 250, 32, 16, 64, 32, 8),      # 16 tiles, two groups of eight heads
    (200, 150, 40, 2, 128, 16, 10),     # groups of 20 query heads: three tiles of them
    (37, 16, 6, 6, 128, 16, 1),         # fewer units than workers
    (3, 40, 4, 2, 64, 16, 3),
    (1, 64, 16, 1, 128, 16, 4),
    (2000, 20, 2, 1, 64, 32, 1),        # units of one tile by the thousand
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("holes", [False, True])
@pytest.mark.parametrize("n,most,hq,hkv,d,page,wide", BATCHES)
def test_whole_units(kda_lib, cuda_dev, monkeypatch, kind, fresh, holes, n, most, hq, hkv, d, page, wide):
    import serving_kda_chunked_gated_gb300.kda as kda
    monkeypatch.setattr(paged_testutil, "quantise", _quantise)
    g = torch.Generator().manual_seed(41)
    lens = _lens(n, most, holes)
    total = [most if x is None else x for x in lens]
    K, V = ([x.to(BF).float() for x in rand_rows(g, total, hkv, d, 0.4)] for _ in "kv")
    q = torch.randn(n, hq, d, generator=g).to(BF)
    need = max(-(-t // page) for t in total)
    room = dict(total=total, extra=wide - need)
    full = Cache(K, V, page, kind, cuda_dev, **room)
    assert full.tables.shape[1] == wide
    # a skipped sequence's length lies before or behind what its table holds
    ll = torch.tensor([(-1 if i % 2 else wide * page + 1) if x is None else x for i, x in enumerate(lens)], dtype=torch.int32, device=cuda_dev)
    more, c = {}, full
    qd = q.to(cuda_dev)
    if fresh:
        short = [x if m is None else x[:max(0, m - 1)] for x, m in zip(K, lens)]
        shortv = [x if m is None else x[:max(0, m - 1)] for x, m in zip(V, lens)]
        c = Cache(short, shortv, page, kind, cuda_dev, **room)
        last = lambda y: torch.stack([x[-1] if len(x) else torch.full((hkv, d), 5.0) for x in y]).to(BF).to(cuda_dev)       # noqa: E731
        more = dict(k=last(K), v=last(V))
    out = torch.full((n, hq, d), 7.0, dtype=BF, device=cuda_dev)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=cuda_dev)
    before = kda.launch_count()
    o, lse = kda.paged_decode(qd, c.k, c.v, c.tables, ll, out=out, want_lse=True, workspace=ws, **more, **c.scales)
    assert kda.launch_count() == before + 1                   # nothing cut, nothing joined
    live = torch.tensor([x is not None for x in lens])
    HK, HV = ([x[:0] if m is None else x for x, m in zip(y, lens)] for y in (full.host["k"], full.host["v"]))
    ro, rl, size = attention(q, [1] * n, HK, HV)
    assert (o[~live.to(cuda_dev)] == 7).all()
    check_out(o.cpu()[live], ro[live], size[live], STEP[kind])
    check_lse(lse.cpu()[live], rl[live])
    for name in "kv":                                         # the new rows where they belong, the others as they were
        a, b = c.flat(name), full.flat(name)
        for x, y in ((a, b),) if kind == "bf16" else zip(a, b):
            x, y = (t.view(torch.int16) if t.dtype == BF else t for t in (x, y))
            assert torch.equal(x, y)
    if not fresh:
        again = kda.paged_decode(qd, c.k, c.v, c.tables, ll, out=out.clone().fill_(7.0), workspace="cache", **c.scales)
        assert torch.equal(o, again)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,hkv", [(1, 1), (500, 8), (300, 3)])
def test_nothing_but_empty_or_skipped_sequences(kda_lib, cuda_dev, monkeypatch, kind, n, hkv):
    import serving_kda_chunked_gated_gb300.kda as kda
    monkeypatch.setattr(paged_testutil, "quantise", _quantise)
    g = torch.Generator().manual_seed(42)
    x = rand_rows(g, [16] * n, hkv, 64)
    c = Cache(x, x, 16, kind, cuda_dev)
    before = c.flat("k")
    new = torch.ones(n, hkv, 64, dtype=BF, device=cuda_dev)
    q = torch.randn(n, 2 * hkv, 64, generator=g).to(BF).to(cuda_dev)
    for length in (-1, 0, c.tables.shape[1] * 16 + 1):
        ll = torch.full((n,), length, dtype=torch.int32, device=cuda_dev)
        out = torch.full((n, 2 * hkv, 64), 7.0, dtype=BF, device=cuda_dev)
        o, lse = kda.paged_decode(q, c.k, c.v, c.tables, ll, k=new, v=new, out=out, want_lse=True, **c.scales)
        assert (o == (7 if length else 0)).all()
        assert length or (lse == -torch.inf).all()
        for a, b in ((before, c.flat("k")),) if kind == "bf16" else zip(before, c.flat("k")):
            a, b = (t.view(torch.int16) if t.dtype == BF else t for t in (a, b))
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_captured_batch_follows_its_lengths(kda_lib, cuda_dev):
    """Whole units, replayed with other lengths: the spread over the workers goes by the lengths on the device."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(43)
    n, page = 300, 16
    K, V = (rand_rows(g, [48] * n, 4, 128, 0.4) for _ in "kv")
    c = Cache(K, V, page, "bf16", cuda_dev)
    q = torch.randn(n, 8, 128, generator=g).to(BF)
    qd, ll = q.to(cuda_dev), torch.ones(n, dtype=torch.int32, device=cuda_dev)
    out = torch.empty(n, 8, 128, dtype=BF, device=cuda_dev)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kda.paged_decode(qd, c.k, c.v, c.tables, ll, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.paged_decode(qd, c.k, c.v, c.tables, ll, out=out, workspace="cache")
    for lens in ([48] * n, _lens(n, 48, True), [0] * (n - 1) + [48], [1] * n):
        ll.copy_(torch.tensor([-5 if x is None else x for x in lens], dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        live = torch.tensor([x is not None for x in lens])
        HK, HV = ([x[:m or 0] for x, m in zip(y, lens)] for y in (c.host["k"], c.host["v"]))
        ro, _, size = attention(q, [1] * n, HK, HV)
        check_out(out.cpu()[live], ro[live], size[live], STEP["bf16"])
        assert (out.cpu()[~live] == 7).all()
