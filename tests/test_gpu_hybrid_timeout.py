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
