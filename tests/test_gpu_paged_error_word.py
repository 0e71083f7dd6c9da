"""A word of the caller's that keeps the reports of all chunk calls it is given to: one read behind a stack of layers tells
whether a wait gave up in any of them, whatever workspaces they had."""
import ctypes

import numpy as np
import pytest
import torch

from paged_testutil import Cache, attention, check_out, rand_rows
from test_paged_abi import ALIGN, FAKE, _prefill


def test_refusals(kda_lib):
    cu = np.array([0, 1, 4, 5], dtype=np.int32)
    a = _prefill(cu, error=FAKE + 4)
    assert kda_lib.kda_paged_prefill(ctypes.byref(a), None) == ALIGN
    assert kda_lib.kda_paged_prefill_workspace_size(ctypes.byref(a)) == 0
    cu = np.array([0, 0, 0, 0], dtype=np.int32)
    assert kda_lib.kda_paged_prefill(ctypes.byref(_prefill(cu, error=None)), None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("workspace", ["given", "cache", None])
def test_layers(kda_lib, cuda_dev, kind, workspace):
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(71)
    K, V = (rand_rows(g, [400, 70], 2, 64, 0.3) for _ in "kv")
    c = Cache(K, V, 32, kind, cuda_dev)
    q = torch.randn(90, 4, 64, generator=g).to(torch.bfloat16)
    cu = torch.tensor([0, 60, 90], dtype=torch.int32)
    word, other = (torch.zeros(1, dtype=torch.int32, device=cuda_dev) for _ in "ab")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev) if workspace == "given" else workspace
    call = lambda error: kda.paged_prefill(q.to(cuda_dev), *c.args, cu_seqlens=cu.to(cuda_dev), cu_seqlens_host=cu, workspace=ws,  # noqa: E731
                                           error=error, **c.scales)
    call(word)
    assert kda.device_error(word) == kda.KDA_OK
    kda.set_wait_limit(0)
    try:
        call(word)                                        # this layer gives up
    finally:
        kda.set_wait_limit(kda.WAIT_LIMIT_DEFAULT)
    o = call(word)                                        # the next ones do not
    call(other)
    call(None)
    if workspace == "given":
        assert kda.device_error(ws) == kda.KDA_OK         # the workspace's word is the last call's
    assert kda.device_error(other) == kda.KDA_OK
    assert kda.device_error(word) == kda.KDA_ERR_TIMEOUT
    assert kda.device_error(word) == kda.KDA_OK
    ro, _, size = attention(q, [60, 30], c.host["k"], c.host["v"])
    check_out(o, ro, size, 2.0 ** -8)


@pytest.mark.gpu
def test_a_word_that_the_kernel_cannot_take(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=cuda_dev)
    pages = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device=cuda_dev)
    one = torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev)
    for bad in (torch.zeros(1, dtype=torch.int64, device=cuda_dev), torch.zeros(2, dtype=torch.int32, device=cuda_dev),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(kda.KDAError):
            kda.paged_prefill(x, pages, pages, one, one[0] + 1, error=bad)
