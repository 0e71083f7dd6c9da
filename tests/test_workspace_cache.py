"""workspace="cache": which calls share a buffer (no GPU: torch's stream queries are replaced), and
what the calls compute on the GPU when streams, threads and captured graphs use it side by side."""
import threading
import types

import pytest
import torch

from hybrid_testutil import gdn_inputs


@pytest.fixture
def fake(monkeypatch):
    """The current stream and whether it is being captured, as the test sets them."""
    import serving_kda_chunked_gated_gb300.kda as kda
    now = types.SimpleNamespace(kda=kda, stream=0, capturing=False, dev=torch.device("cpu"))
    monkeypatch.setattr(kda, "_WS_CACHE", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=now.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now.capturing)

    class given:                                           # torch.cuda.stream(s): s is current within
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.was, now.stream = now.stream, now.stream if self.s is None else self.s.cuda_stream

        def __exit__(self, *a):
            now.stream = self.was

    monkeypatch.setattr(torch.cuda, "stream", given)
    return now


def test_one_buffer_for_each_stream(fake):
    get = lambda n: fake.kda._cached_workspace(fake.dev, n)                  # noqa: E731
    a = get(100)
    assert get(50) is a and get(100) is a
    fake.stream = 7
    b = get(100)
    assert b is not a and b.data_ptr() != a.data_ptr()
    assert get(200) is not b and get(10).numel() == 200
    fake.stream = 0
    assert get(100) is a                         # untouched by the other stream's growth


def test_one_buffer_for_each_thread(fake):
    """Two threads may interleave their kernels on one stream."""
    mine, other = fake.kda._cached_workspace(fake.dev, 100), []
    t = threading.Thread(target=lambda: other.append(fake.kda._cached_workspace(fake.dev, 100)))
    t.start()
    t.join()
    assert other[0].data_ptr() != mine.data_ptr()


def test_captured_calls_keep_away_from_the_cache(fake):
    a = fake.kda._cached_workspace(fake.dev, 100)
    fake.capturing = True
    b, c = (fake.kda._cached_workspace(fake.dev, 100) for _ in range(2))
    assert len({x.data_ptr() for x in (a, b, c)}) == 3
    big = fake.kda._cached_workspace(fake.dev, 1000)
    fake.capturing = False
    assert fake.kda._cached_workspace(fake.dev, 100) is a and big.numel() == 1000


def test_host_prefill_staging_follows_the_same_rule(fake, monkeypatch):
    """``prefill_from_host``: calls on two streams, and a stream given in the call, have staging buffers of their own."""
    kda, used = fake.kda, []
    monkeypatch.setattr(kda, "_STAGING", {})
    lib = types.SimpleNamespace(kda_prefill_from_host_staging_size=lambda a, slab: 64,
                                kda_prefill_from_host=lambda a, slab, at, n, s: used.append(at) or 0)
    monkeypatch.setattr(kda, "load_library", lambda: lib)
    monkeypatch.setattr(torch, "device", lambda *a: fake.dev)

    x = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    f = torch.zeros(4, 1, 128)
    call = lambda **kw: kda.prefill_from_host(x, x, x, f, f, f, out=(x, None, f), slab=64, **kw)     # noqa: E731
    call()
    fake.stream = 7
    call()
    call(stream=types.SimpleNamespace(cuda_stream=9))
    fake.stream = 0
    call()
    call(stream=types.SimpleNamespace(cuda_stream=9))
    assert used[0] == used[3] and used[2] == used[4] and len(set(used)) == 3


@pytest.mark.parametrize("workspace", [None, "cache"])
def test_temporaries_belong_to_the_stream_that_uses_them(fake, monkeypatch, workspace):
    """What a call with stream= allocates and drops again (bounds, workspace): on another stream's pool
    the next call could have it while this one still runs."""
    kda, made = fake.kda, []
    empty, to, tensor = torch.empty, torch.Tensor.to, torch.tensor

    def note(kind, x):
        made.append((kind, x.dtype, fake.stream))
        return x

    monkeypatch.setattr(torch, "empty", lambda *a, **k: note("empty", empty(*a, **k)))
    monkeypatch.setattr(torch, "tensor", lambda *a, **k: note("device" if "device" in k else "host", tensor(*a, **k)))
    monkeypatch.setattr(torch.Tensor, "to", lambda x, *a, **k: note("host" if a == ("cpu",) else "device", to(x, *a, **k)))
    monkeypatch.setattr(kda, "load_library", lambda: types.SimpleNamespace(
        kda_prefill_records=lambda *a: 0, kda_short_conv=lambda *a: 0, kda_prefill=lambda *a: 0,
        kda_prefill_workspace_size=lambda a: 64))
    x, f = torch.zeros(4, 1, 128, dtype=torch.bfloat16), torch.zeros(4, 1, 128)
    s = types.SimpleNamespace(cuda_stream=9)
    kda.prefill(x, x, x, f, f, f, workspace=workspace, stream=s)
    kda.prefill_records(x, x, x, f, f, f, stream=s)
    kda.short_conv(f[:, 0], f[:, 0], stream=s)
    temporary = [m for m in made if m[1] == torch.uint8 or (m[0] == "device" and m[1] == torch.int32)]
    assert len(temporary) == 5 and all(m[2] == 9 for m in temporary), made


def _call(kda, g, cu, cu_host, **kw):
    return kda.gdn_prefill(**g, cu_seqlens=cu, cu_seqlens_host=cu_host, workspace="cache", **kw)


def _gdn(lens, seed, dev):
    d, cu = gdn_inputs(lens, 4, 8, seed=seed)
    return {k: x.to(dev) for k, x in d.items()}, cu.to(dev), cu


@pytest.mark.gpu
def test_two_streams_and_a_thread(kda_lib, cuda_dev):
    """Calls on two streams, and of two threads on one stream, at the same time: the bits of calls alone."""
    import serving_kda_chunked_gated_gb300.kda as kda
    sets = [_gdn(lens, seed, cuda_dev) for seed, lens in enumerate(([900, 30, 129], [64, 1100]))]
    alone = [_call(kda, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(_call(kda, *sets[i], stream=s))
    torch.cuda.synchronize()

    def work(i):
        for _ in range(20):
            got[i].append(_call(kda, *sets[i], stream=streams[0]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 25
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, alone[i]))
    kda.release_workspace_cache()


@pytest.mark.gpu
def test_graph_then_a_larger_call_then_replay(kda_lib, cuda_dev):
    """A captured call, a larger eager one, other tensors over whatever memory that gave back, a replay."""
    import serving_kda_chunked_gated_gb300.kda as kda
    kda.release_workspace_cache()
    small, large = _gdn([400], 5, cuda_dev), _gdn([3000, 700], 6, cuda_dev)
    want, want_l = _call(kda, *small), _call(kda, *large)
    kda.release_workspace_cache()
    _call(kda, *small)                                     # the cache holds a buffer that the graph could have taken
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = _call(kda, *small)
        o2, S2 = _call(kda, *small)                        # two calls of one capture
    got = _call(kda, *large)
    filler = [torch.full((1 << 20,), float("nan"), device=cuda_dev) for _ in range(64)]
    for _ in range(2):
        for x in (o, S, o2, S2):
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((o, S, o2, S2), want + want))
    assert all(torch.equal(a, b) for a, b in zip(got, want_l))
    assert all(torch.isnan(x).all() for x in filler)
    kda.release_workspace_cache()


@pytest.mark.gpu
def test_prefill_of_the_channel_gated_rule(kda_lib, cuda_dev):
    """``prefill`` takes its cached buffer the same way."""
    import serving_kda_chunked_gated_gb300.kda as kda
    kda.release_workspace_cache()
    g = torch.Generator().manual_seed(2)

    def inputs(T):
        r = lambda *s: torch.randn(*s, generator=g)        # noqa: E731
        q, k, v = (r(T, 4, 128).to(torch.bfloat16) for _ in range(3))
        cu = torch.tensor([0, T], dtype=torch.int32)
        return [x.to(cuda_dev) for x in (q, k, v, r(T, 4, 128), torch.sigmoid(r(T, 4)), torch.zeros(4), cu)]

    sets = [inputs(500), inputs(1300)]
    alone = [kda.prefill(*x) for x in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[kda.prefill(*x, workspace="cache", stream=s) for x, s in zip(sets, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for r in got:
        for have, want in zip(r, alone):
            assert torch.equal(have[0], want[0]) and torch.equal(have[1], want[1])
    assert kda.cached_workspace(cuda_dev) is None          # nothing ran on this stream
    with torch.cuda.stream(streams[1]):
        assert kda.device_error(kda.cached_workspace(cuda_dev)) == kda.KDA_OK
    kda.release_workspace_cache()


@pytest.mark.gpu
def test_streams_given_with_no_bounds_and_no_workspace(kda_lib, cuda_dev):
    """Calls on two streams in turn, each with its own length: bounds and workspaces that the call makes itself."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(3)
    sets = []
    for T in (300, 1700, 64):
        r = lambda *s: torch.randn(*s, generator=g)        # noqa: E731
        q, k, v = (r(T, 4, 128).to(torch.bfloat16) for _ in range(3))
        sets.append([x.to(cuda_dev) for x in (q, k, v, r(T, 4, 128), torch.sigmoid(r(T, 4)), torch.zeros(4), r(512, 4))])
    conv = lambda x, **kw: kda.short_conv(x[0].flatten(1), x[6], **kw)       # noqa: E731
    alone = [[*kda.prefill(*x[:6])[:2], *conv(x)] for x in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[[*kda.prefill(*x[:6], stream=s)[:2], *conv(x, stream=s)] for x, s in zip(sets, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for have, want in zip(r, alone) for a, b in zip(have, want))
