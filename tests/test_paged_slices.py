"""Tables, lengths and bounds as a scheduler slices them out of larger arrays: they start at any int32, the entry points
want 16 bytes' alignment.  The binding hands over aligned copies, and only of those that need it."""
import ctypes

import pytest
import torch

from paged_testutil import Cache, attention, check_out, rand_rows

BF = torch.bfloat16
CHUNK, STEP = 2.0 ** -8, {"bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}      # rounding of the softmax weights


def _words(address, n):
    return list((ctypes.c_int32 * n).from_address(address))


def test_addresses():
    import serving_kda_chunked_gated_gb300.kda as kda
    pages = torch.zeros(4, 16, 2, 64, dtype=BF)
    tables, lens = torch.arange(15, dtype=torch.int32).view(3, 5), torch.arange(1, 5, dtype=torch.int32)
    dev = torch.device("cpu")
    c = kda._paged_cache(pages, pages, None, None, tables[1:], lens[1:3], dev)
    assert c.tables % 16 == 0 and c.lens % 16 == 0
    assert _words(c.tables, 10) == list(range(5, 15)) and _words(c.lens, 2) == [2, 3]
    c = kda._paged_cache(pages, pages, None, None, tables, lens[:3], dev)
    assert (c.tables, c.lens) == (tables.data_ptr(), lens.data_ptr())             # aligned ones as they are
    for bad in (tables[:, 1:], tables[1:].long(), tables[1]):                     # a copy makes none of these right
        with pytest.raises(kda.KDAError):
            kda._paged_cache(pages, pages, None, None, bad, lens[1:], dev)


def _off(x, by=1):
    """``x`` in memory that starts ``by`` words behind an aligned address."""
    flat = torch.full((x.numel() + by,), -7, dtype=torch.int32, device=x.device)
    flat[by:] = x.flatten()
    y = flat[by:].view(x.shape)
    assert y.data_ptr() % 16 == 4 * by
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_calls(kda_lib, cuda_dev, kind):
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(61)
    lens, hist = [5, 130, 1], [40, 0, 300]
    total = [a + b for a, b in zip(lens, hist)]
    K, V = ([x.to(BF).float() for x in rand_rows(g, total, 2, 64, 0.4)] for _ in "kv")
    full = Cache(K, V, 16, kind, cuda_dev)
    c = Cache([x[:h] for x, h in zip(K, hist)], [x[:h] for x, h in zip(V, hist)], 16, kind, cuda_dev, total=total)
    q = torch.randn(sum(lens), 4, 64, generator=g).to(BF)
    cu = torch.tensor([0, 5, 135, 136], dtype=torch.int32)
    k, v = (torch.cat([x[h:] for x, h in zip(y, hist)]).to(BF).to(cuda_dev) for y in (K, V))
    for by in (1, 2, 3):
        tables, ll, cud = _off(full.tables, by), _off(full.lens, by), _off(cu.to(cuda_dev), by)
        kda.paged_write(k, v, c.k, c.v, tables, ll, cu_seqlens=cud, **c.scales)
        rk, rv = kda.paged_read(c.k, c.v, tables, ll, 136, cu_seqlens=cud, dtype=torch.float32, **c.scales)
        for got, host in ((rk, full.host["k"]), (rv, full.host["v"])):
            assert torch.equal(got.cpu().double(), torch.cat([x[h:] for x, h in zip(host, hist)]))
        for ws in (None, "cache"):
            o = kda.paged_prefill(q.to(cuda_dev), c.k, c.v, tables, ll, cu_seqlens=cud, cu_seqlens_host=cu, workspace=ws, **c.scales)
            ro, _, size = attention(q, lens, full.host["k"], full.host["v"])
            check_out(o, ro, size, CHUNK)
            o = kda.paged_decode(q[:3].to(cuda_dev), c.k, c.v, tables, ll, workspace=ws, **c.scales)
            ro, _, size = attention(q[:3], [1] * 3, full.host["k"], full.host["v"])
            check_out(o, ro, size, STEP[kind])
    # one sequence out of the batch: a row of an odd-width table, one length
    wide = torch.nn.functional.pad(full.tables, (0, 4 - full.tables.shape[1] % 4 + 1), value=-1)
    assert wide.shape[1] % 4 == 1
    o = kda.paged_decode(q[:1].to(cuda_dev), c.k, c.v, wide[1:2], full.lens[1:2], **c.scales)
    ro, _, size = attention(q[:1], [1], full.host["k"][1:2], full.host["v"][1:2])
    check_out(o, ro, size, STEP[kind])


@pytest.mark.gpu
def test_a_captured_call_follows_the_slices(kda_lib, cuda_dev):
    """The copies are part of a captured call: a replay reads the slices as they are then."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(62)
    K, V = (rand_rows(g, [200, 90, 33], 2, 64, 0.4) for _ in "kv")
    a, b = (Cache(K, V, 16, "bf16", cuda_dev, seed=s) for s in (1, 2))
    q = torch.randn(3, 4, 64, generator=g).to(BF)
    qd, tables, ll = q.to(cuda_dev), _off(a.tables), _off(a.lens)
    k, v = a.k.clone(), a.v.clone()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    cud = _off(cu.to(cuda_dev))
    s = torch.cuda.Stream()
    calls = lambda: (kda.paged_decode(qd, k, v, tables, ll, workspace="cache"),                           # noqa: E731
                     kda.paged_prefill(qd, k, v, tables, ll, cu_seqlens=cud, cu_seqlens_host=cu, workspace="cache"))
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step, pre = calls()
    for src, lens in ((a, [200, 90, 33]), (b, [77, 1, 20])):
        for x, y in ((k, src.k), (v, src.v), (tables, src.tables)):
            x.copy_(y)
        ll.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        HK, HV = ([x[:m] for x, m in zip(y, lens)] for y in (src.host["k"], src.host["v"]))
        ro, _, size = attention(q, [1] * 3, HK, HV)
        check_out(step, ro, size, STEP["bf16"])
        check_out(pre, ro, size, CHUNK)
