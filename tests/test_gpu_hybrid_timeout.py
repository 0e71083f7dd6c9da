"""A bounded wait that gives up inside the delta rule's or the window's prefill is reported,
the kernels end, and the next call is right again."""
import pytest
import torch

from hybrid_testutil import check_window, gdn_inputs, gdn_reference, rel, window_reference

pytestmark = pytest.mark.gpu


@pytest.fixture
def wait_limit_zero(kda_lib):
    import serving_kda_chunked_gated_gb300.kda as kda
    kda.set_wait_limit(0)
    yield
    kda.set_wait_limit(kda.WAIT_LIMIT_DEFAULT)
    torch.cuda.synchronize()
    kda.device_error(None)


# (no sequence longer than 24 tokens: the recurrence, which waits for nothing)
@pytest.mark.parametrize("lens", [[1, 25], [200], [128, 0, 700]])
def test_gdn_prefill(kda_lib, cuda_dev, wait_limit_zero, lens):
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs(lens, 1, 2, seed=31)
    g = {k: x.to(cuda_dev) for k, x in d.items()}
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device=cuda_dev)
    kda.gdn_prefill(**g, cu_seqlens=cu.to(cuda_dev), workspace=ws)
    assert kda.device_error(ws) == kda.KDA_ERR_TIMEOUT
    kda.set_wait_limit(kda.WAIT_LIMIT_DEFAULT)
    o, S = kda.gdn_prefill(**g, cu_seqlens=cu.to(cuda_dev), workspace=ws)
    assert kda.device_error(ws) == kda.KDA_OK
    ro, rS = gdn_reference(**d, cu=cu)
    assert rel(S, rS) < 1e-5 and rel(o, ro) < 4.5e-3


@pytest.mark.parametrize("T,window,sinks", [(1, 1, 0), (300, 100, 4), (900, 500, 0)])
def test_window_prefill(kda_lib, cuda_dev, wait_limit_zero, T, window, sinks):
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(T, h, 128, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    call = lambda: kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), window, sinks)     # noqa: E731
    assert kda.device_error(None) == kda.KDA_OK
    call()
    assert kda.device_error(None) == kda.KDA_ERR_TIMEOUT
    kda.set_wait_limit(kda.WAIT_LIMIT_DEFAULT)
    o = call()
    assert kda.device_error(None) == kda.KDA_OK
    cu = torch.tensor([0, T])
    ro, _, size = window_reference(q, k, v, cu, cu, window, sinks)
    check_window(o, ro, size)


def _window_call(dev, T=300):
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(T, h, 128, generator=g).to(torch.bfloat16).to(dev) for h in (4, 2, 2))
    return lambda **kw: kda.window_prefill(q, k, v, 100, 4, **kw)


def test_window_words_keep_callers_apart(kda_lib, cuda_dev, wait_limit_zero):
    """Two streams with a word each: the one whose wait gave up learns of it, whoever reads before it."""
    import serving_kda_chunked_gated_gb300.kda as kda
    call = _window_call(cuda_dev)
    words = [torch.zeros(1, dtype=torch.int32, device=cuda_dev) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    kda.device_error(None)
    torch.cuda.synchronize()
    call(error=words[1], stream=streams[1])
    kda.set_wait_limit(kda.WAIT_LIMIT_DEFAULT)
    call(error=words[0], stream=streams[0])
    torch.cuda.synchronize()
    assert kda.device_error(None) == kda.KDA_OK
    assert kda.device_error(words[0], streams[0]) == kda.KDA_OK
    assert kda.device_error(words[1], streams[1]) == kda.KDA_ERR_TIMEOUT
    assert kda.device_error(words[1], streams[1]) == kda.KDA_OK


def test_window_reports_are_not_lost_to_a_reader_beside_them(kda_lib, cuda_dev, wait_limit_zero):
    """One thread reads the shared word all the time; every call that gives up shows in one of its
    answers.  (Copied and then cleared, a report that came up between the two left no trace.)"""
    import threading
    import time
    import serving_kda_chunked_gated_gb300.kda as kda
    call, seen, stop = _window_call(cuda_dev, 1), [0], threading.Event()
    kda.device_error(None)
    side = torch.cuda.Stream()

    def read():
        while not stop.is_set():
            seen[0] += kda.device_error(None, side) == kda.KDA_ERR_TIMEOUT

    reader = threading.Thread(target=read)
    reader.start()
    lost = 0
    try:
        for _ in range(300):
            before = seen[0]
            call()
            torch.cuda.current_stream().synchronize()
            end = time.monotonic() + 1.0
            while seen[0] == before and time.monotonic() < end:
                time.sleep(0)
            lost += seen[0] == before
            if lost:
                break
    finally:
        stop.set()
        reader.join()
    assert lost == 0
