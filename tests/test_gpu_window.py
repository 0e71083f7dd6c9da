"""Windowed attention with sinks on the GPU (prefill, cache fill, decode) against 64 bits.
Tolerances: hybrid_testutil.check_window; lse: float32 scores of d exact products, 2^-20
relative to their size plus the logarithm's rounding."""
import pytest
import torch

from hybrid_testutil import check_window, visible, window_reference

pytestmark = pytest.mark.gpu


def _cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)


def _inputs(lens, hist, Hq, Hkv, d, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    klens = [a + b for a, b in zip(lens, hist)]
    r = lambda n, h: (size * torch.randn(n, h, d, generator=g)).to(torch.bfloat16)      # noqa: E731
    return r(sum(lens), Hq), r(sum(klens), Hkv), r(sum(klens), Hkv), _cu(lens), _cu(klens)


def _lse_ok(lse, ref, q, k, scale):
    size = q.float().norm(dim=-1).max().item() * k.float().norm(dim=-1).max().item() * abs(scale)
    assert (lse.double().cpu() - ref).abs().max().item() <= 2.0 ** -20 * (size + 1) + 2.0 ** -22 * ref.abs().max().item()


@pytest.mark.parametrize("lens,hist,Hq,Hkv,d,window,sinks", [
    ([1], [0], 1, 1, 128, 1, 0), ([5], [0], 2, 1, 64, 3, 1), ([130], [0], 2, 2, 128, 1, 4),
    ([127, 128, 129], [0, 0, 0], 2, 1, 128, 128, 0), ([300], [0], 3, 1, 64, 100, 5), ([300], [0], 2, 1, 128, 129, 130),
    ([257], [0], 4, 4, 64, 1000, 4), ([0, 40, 0, 200], [3, 500, 0, 1], 2, 1, 128, 150, 7),
    ([600], [0], 5, 1, 128, 256, 0), ([1, 1, 1], [700, 0, 128], 8, 2, 64, 300, 64), ([900], [100], 2, 1, 128, 640, 200),
])
def test_prefill(kda_lib, cuda_dev, lens, hist, Hq, Hkv, d, window, sinks):
    import serving_kda_chunked_gated_gb300.kda as kda
    q, k, v, cu, cuk = _inputs(lens, hist, Hq, Hkv, d, seed=window)
    ro, rl, size = window_reference(q, k, v, cu, cuk, window, sinks)
    o, lse = kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), window, sinks, cu.to(cuda_dev), cu,
                                cuk.to(cuda_dev), cuk, want_lse=True)
    check_window(o, ro, size)
    _lse_ok(lse, rl, q, k, d ** -0.5)


@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 1.0), (1.0, 4.0), (1e-3, 0.5)])
def test_prefill_scales(kda_lib, cuda_dev, scale, size):
    """No scale, a negative one, scores in the hundreds (one key takes all), almost equal weights."""
    import serving_kda_chunked_gated_gb300.kda as kda
    q, k, v, cu, cuk = _inputs([333], [0], 2, 1, 128, seed=4, size=size)
    ro, rl, sz = window_reference(q, k, v, cu, cuk, 200, 3, scale)
    o, lse = kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), 200, 3, scale=scale, want_lse=True)
    if size < 2:
        check_window(o, ro, sz)
    else:
        # scores near 400: each float32 score is off by up to 2^-24 of the sum of its products' sizes (a few
        # thousand), and a weight by that factor's exponential, about 2^-11; under a bf16 half step
        check_window(o, ro, sz + 2.0 ** -11 * sz)
    _lse_ok(lse, rl, q, k, scale)


def test_prefill_packed_projection_and_stream(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    T, Hq, Hkv, d = 211, 6, 2, 64
    x = torch.randn(T, (Hq + 2 * Hkv) * d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    cut = lambda y: (y[:, :Hq * d].unflatten(1, (Hq, d)), y[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)),   # noqa: E731
                     y[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)))
    q, k, v = cut(x)
    cu = _cu([T])
    ro, _, size = window_reference(q, k, v, cu, cu, 50, 2)
    st = torch.cuda.Stream()
    xd = x.to(cuda_dev)
    st.wait_stream(torch.cuda.current_stream())
    o = kda.window_prefill(*cut(xd), 50, 2, stream=st)
    st.synchronize()
    check_window(o, ro, size)


def test_prefill_unseen_rows_may_hold_anything(kda_lib, cuda_dev):
    """NaN and infinity in keys and values that no query of a sequence sees (behind the
    window, in other sequences) change nothing, bit for bit."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens, hist, W, sinks = [70, 100, 30], [0, 400, 0], 60, 4
    q, k, v, cu, cuk = _inputs(lens, hist, 2, 1, 128, seed=8)
    call = lambda k, v: kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), W, sinks, cu.to(cuda_dev), cu,   # noqa: E731
                                           cuk.to(cuda_dev), cuk, want_lse=True)
    o, lse = call(k, v)
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        hidden = slice(70 + sinks, 70 + 400 - W + 1)        # positions that the first query has left behind
        k2[hidden], v2[hidden] = bad, bad
        o2, lse2 = call(k2, v2)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        k2, v2 = k.clone(), v.clone()
        k2[70:570], v2[70:570] = bad, bad                   # the whole middle sequence
        o2, lse2 = call(k2, v2)
        for s in (slice(0, 70), slice(170, 200)):
            assert torch.equal(o2[s], o[s]) and torch.equal(lse2[s], lse[s])


@pytest.mark.parametrize("d,Hq,Hkv,window,sinks,extra", [
    (64, 2, 1, 5, 0, 0), (128, 4, 2, 40, 3, 0), (64, 17, 1, 129, 16, 9), (128, 40, 2, 300, 1, 1), (64, 3, 3, 1, 2, 0),
])
def test_prefill_fill_then_decode(kda_lib, cuda_dev, d, Hq, Hkv, window, sinks, extra):
    """Prompts fill the ring caches, then tokens are decoded until every ring has wrapped;
    each step against the whole history in 64 bits.  Slots that nobody uses keep their rows."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens = [1, window + sinks + 7, max(1, sinks - 1), 2 * window + 3]
    N, steps = len(lens), min(window + 3, 24)
    full = [n + steps for n in lens]
    q, k, v, cu, _ = _inputs(full, [0] * N, Hq, Hkv, d, seed=window + sinks)
    rows = sinks + window + extra
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32)
    kc = torch.full((6, rows, Hkv, d), 9.0, dtype=torch.bfloat16, device=cuda_dev)
    vc = kc.clone()
    at = torch.cat([torch.arange(int(cu[n]), int(cu[n]) + lens[n]) for n in range(N)])
    cul = _cu(lens)
    o = kda.window_prefill(q[at].to(cuda_dev), k[at].to(cuda_dev), v[at].to(cuda_dev), window, sinks, cul.to(cuda_dev), cul,
                           k_cache=kc, v_cache=vc, slots=slots.to(cuda_dev))
    ro, _, size = window_reference(q, k, v, cu, cu, window, sinks)
    check_window(o, ro[at], size[at], "prefill")
    R = rows - sinks
    for n in range(N):                                       # the cache rows hold exactly what they should
        expect = torch.full((rows, Hkv, d), 9.0, dtype=torch.bfloat16)
        for p in visible(lens[n] - 1, window, sinks):
            expect[p if p < sinks else sinks + (p - sinks) % R] = k[int(cu[n]) + p]
        held = kc[int(slots[n])].cpu()
        written = (held != 9.0).any(-1).any(-1)
        assert torch.equal(held[written], expect[written]) and torch.equal(held, expect)
    for s in range(steps):
        i = torch.tensor([int(cu[n]) + lens[n] + s for n in range(N)])
        pos = torch.tensor([lens[n] + s for n in range(N)], dtype=torch.int32)
        o = kda.window_decode(q[i].to(cuda_dev), k[i].to(cuda_dev), v[i].to(cuda_dev), kc, vc, pos.to(cuda_dev), window,
                              sinks, slots=slots.to(cuda_dev))
        check_window(o, ro[i], size[i], f"step {s}")
    assert (kc[[1, 3]] == 9.0).all() and (vc[[1, 3]] == 9.0).all()


def test_decode_first_token_skips_and_graph(kda_lib, cuda_dev):
    """Position 0 (only itself visible) with a cache full of NaN; bad slots and positions
    leave everything; a captured step replays on new inputs."""
    import serving_kda_chunked_gated_gb300.kda as kda
    N, Hq, Hkv, d, W, sinks = 5, 4, 2, 128, 20, 2
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(N, h, d, generator=g).to(torch.bfloat16).to(cuda_dev) for h in (Hq, Hkv, Hkv))
    kc = torch.full((4, W + sinks, Hkv, d), float("nan"), dtype=torch.bfloat16, device=cuda_dev)
    vc = kc.clone()
    slots = torch.tensor([1, 4, -1, 0, 2], dtype=torch.int32, device=cuda_dev)
    pos = torch.tensor([0, 0, 0, 0, -1], dtype=torch.int32, device=cuda_dev)
    out = torch.full((N, Hq, d), 3.0, dtype=torch.bfloat16, device=cuda_dev)
    kda.window_decode(q, k, v, kc, vc, pos, W, sinks, slots=slots, out=out)
    want = v.repeat_interleave(Hq // Hkv, 1)
    for n in (0, 3):
        assert torch.equal(out[n], want[n])                  # one key: weight 1
    for n in (1, 2, 4):
        assert (out[n] == 3.0).all()
    assert torch.equal(kc[1, 0], k[0]) and torch.equal(vc[0, 0], v[3])
    assert torch.isnan(kc[2:]).all() and torch.isnan(kc[:2, 1:]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = kda.window_decode(q, k, v, kc, vc, pos, W, sinks, slots=slots)
    q.mul_(2), v.mul_(-1), slots.copy_(torch.tensor([0, 1, 2, 3, 9], dtype=torch.int32))
    graph.replay()
    assert torch.equal(o[:4], v.repeat_interleave(Hq // Hkv, 1)[:4])


def test_decode_long_window_split_over_ctas(kda_lib, cuda_dev):
    """One sequence over a long cache: every CTA of the cluster has a part, few of them the last tile."""
    import serving_kda_chunked_gated_gb300.kda as kda
    W, sinks, Hq, Hkv, d = 5000, 3, 6, 1, 128
    g = torch.Generator().manual_seed(2)
    kc, vc = (torch.randn(1, W + sinks, Hkv, d, generator=g).to(torch.bfloat16) for _ in "kv")
    q, k, v = (torch.randn(1, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    for pos in (0, 2, 3, 17, 4999, 5003, 123456, 2 ** 31 - 2):
        kd, vd = kc.to(cuda_dev), vc.to(cuda_dev)
        o = kda.window_decode(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), kd, vd,
                              torch.tensor([pos], dtype=torch.int32, device=cuda_dev), W, sinks)
        row = lambda p: p if p < sinks else sinks + (p - sinks) % W                          # noqa: E731
        K, V = kc[0].clone(), vc[0].clone()
        K[row(pos)], V[row(pos)] = k[0], v[0]
        assert torch.equal(kd[0].cpu(), K) and torch.equal(vd[0].cpu(), V)
        rows = torch.tensor([row(p) for p in visible(pos, W, sinks)])
        s = torch.einsum("hd,kd->hk", q[0].double(), K[rows, 0].double()) * d ** -0.5
        w = torch.softmax(s, -1)
        check_window(o, (w @ V[rows, 0].double())[None], (w @ V[rows, 0].double().abs())[None], f"position {pos}")


@pytest.mark.parametrize("N,W", [(11, 1100), (15, 1100), (20, 1100), (24, 1100), (33, 1100), (40, 1100), (60, 1100),
                                 (77, 1100), (160, 300), (5, 40), (310, 30), (310, 500), (310, 600)])
def test_decode_any_cluster_size(kda_lib, cuda_dev, N, W):
    """Batch sizes that give each sequence from eight CTAs down to one and from eight warps to two, at
    positions up to the last int32."""
    import serving_kda_chunked_gated_gb300.kda as kda
    sinks, Hq, Hkv, d = 2, 3, 1, 64
    g = torch.Generator().manual_seed(N)
    kc, vc = (torch.randn(N, W + sinks, Hkv, d, generator=g).to(torch.bfloat16) for _ in "kv")
    q, k, v = (torch.randn(N, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pos = torch.randint(0, 4000, (N,), generator=g, dtype=torch.int32)
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, 0, 1
    kd, vd = kc.to(cuda_dev), vc.to(cuda_dev)
    o = kda.window_decode(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), kd, vd, pos.to(cuda_dev), W, sinks)
    ro, size = torch.empty(N, Hq, d, dtype=torch.float64), torch.empty(N, Hq, d, dtype=torch.float64)
    for n in range(N):
        row = lambda p: p if p < sinks else sinks + (p - sinks) % W                          # noqa: E731
        p = int(pos[n])
        kc[n, row(p)], vc[n, row(p)] = k[n], v[n]
        rows = torch.tensor([row(j) for j in visible(p, W, sinks)])
        w = torch.softmax(torch.einsum("hd,kd->hk", q[n].double(), kc[n, rows, 0].double()) * d ** -0.5, -1)
        ro[n], size[n] = w @ vc[n, rows, 0].double(), w @ vc[n, rows, 0].double().abs()
    check_window(o, ro, size, f"{N} sequences")
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


@pytest.mark.parametrize("N", [33, 64, 700])
def test_prefill_many_sequences(kda_lib, cuda_dev, N):
    """Packed batches of more than one group of 32 sequences, empty ones among them, some resumed."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens, hist = [(11 * i) % 23 for i in range(N)], [(5 * i) % 7 for i in range(N)]
    lens[N // 2], lens[3], hist[-1] = 200, 0, 150
    q, k, v, cu, cuk = _inputs(lens, hist, 2, 1, 64, seed=N)
    ro, rl, size = window_reference(q, k, v, cu, cuk, 20, 2)
    o, lse = kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), 20, 2, cu.to(cuda_dev), cu, cuk.to(cuda_dev),
                                cuk, want_lse=True)
    check_window(o, ro, size)
    _lse_ok(lse, rl, q, k, 64 ** -0.5)


FIRST_CALL = """
import torch, serving_kda_chunked_gated_gb300.kda as kda
x = lambda *s, d=torch.bfloat16: torch.randn(*s, device="cuda").to(d)
f = torch.float32
q, k, v, kc, vc = x(3, 4, 128), x(3, 2, 128), x(3, 2, 128), x(3, 300, 2, 128), x(3, 300, 2, 128)
pos = torch.tensor([1, 299, 1000], dtype=torch.int32, device="cuda")
cos, sin, w, st, z, be = x(1001, 64, d=f), x(1001, 64, d=f), x(128, d=f), x(3, 2, 128, 128, d=f), x(3, 2, d=f), x(3, 2, d=f)
cu = torch.tensor([0, 1, 3], dtype=torch.int32)
cud, A = cu.cuda(), torch.zeros(2, device="cuda")
lq, lk, lv, lz, lb = x(60, 2, 128), x(60, 2, 128), x(60, 2, 128), x(60, 2, d=f), x(60, 2, d=f)
cl = torch.tensor([0, 20, 60], dtype=torch.int32)
cld = cl.cuda()
def step():
    S = st.clone()
    return [kda.window_decode(q, k, v, kc, vc, pos, 296, 4), *kda.qk_norm_rope(q, k, cos, sin, pos, w, w),
            kda.gdn_decode_step(k, k, v, z, be, A, S), S, kda.window_prefill(q, k, v, 2, 1, cud, cu),
            *kda.gdn_prefill(lq, lk, lv, lz, lb, A, cld, cl)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    held = step()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in held]
g.replay()
eager = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, held, eager))
print("captured")
"""


def test_first_calls_captured(kda_lib, cuda_dev):
    """A fresh process whose first call of every operator is a captured one: replays equal eager calls."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("N,Hq,Hkv,d,W", [(3, 4, 2, 128, 400), (40, 24, 4, 64, 900), (200, 8, 8, 128, 300), (400, 16, 1, 64, 200)])
def test_decode_rounds_once(kda_lib, cuda_dev, N, Hq, Hkv, d, W):
    """The weights keep 16 bits: what is left against 64 bits is the output's own rounding (2^-8 of it at
    most), 2^-17 of every weight in two bf16 parts, and 2^-17 of it from its score (below 8 in size, at most
    eight float32 steps of 2^-23 each)."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator(device=cuda_dev).manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_dev).to(torch.bfloat16)      # noqa: E731
    q, k, v, kc, vc = r(N, Hq, d), r(N, Hkv, d), r(N, Hkv, d), r(N, W, Hkv, d), r(N, W, Hkv, d)
    pos = torch.full((N,), 5 * W + 3, dtype=torch.int32, device=cuda_dev)
    o = kda.window_decode(q, k, v, kc, vc, pos, W)
    K, V = (x.double().transpose(1, 2) for x in (kc, vc))                                # rows in any order: all are seen
    w = torch.softmax(q.double().unflatten(1, (Hkv, Hq // Hkv)) @ K.transpose(-1, -2) * d ** -0.5, -1)
    want, size = (w @ V).flatten(1, 2), (w @ V.abs()).flatten(1, 2)
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -16 * size + 1e-30
    assert ((o.double() - want).abs() <= bound).all(), ((o.double() - want).abs() / bound).max()


def _reference_on(dev, q, k, v, cu_q, cu_k, window, sinks):
    """window_reference on the GPU, head by head: (o, lse, size) in 64 bits."""
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    o, size = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    for n in range(len(cu_q) - 1):
        a, b, ka, kb = int(cu_q[n]), int(cu_q[n + 1]), int(cu_k[n]), int(cu_k[n + 1])
        p = torch.arange(kb - ka - (b - a), kb - ka, device=dev)[:, None]
        j = torch.arange(kb - ka, device=dev)
        see = (j <= p) & ((j > p - window) | (j < sinks))
        for h in range(Hq):
            K, V = (x[ka:kb, h // (Hq // Hkv)].to(dev).double() for x in (k, v))
            s = (q[a:b, h].to(dev).double() @ K.T * d ** -0.5).masked_fill(~see, float("-inf"))
            r = torch.logsumexp(s, -1, keepdim=True)
            w = (s - r).exp()
            o[a:b, h], size[a:b, h], lse[a:b, h] = (w @ V).cpu(), (w @ V.abs()).cpu(), r[:, 0].cpu()
    return o, lse, size


@pytest.mark.parametrize("lens,hist,Hq,Hkv,d,window,sinks", [
    # tiles of 8 and 16 heads, the cap at 16 (32 and 48 query heads to a key head)
    ([300, 1, 70], [0, 90, 33], 8, 1, 128, 100, 5), ([300, 1, 70], [0, 90, 33], 16, 1, 128, 100, 5),
    ([200, 37], [0, 300], 32, 1, 64, 150, 0), ([200, 37], [0, 300], 64, 2, 128, 129, 130), ([77], [10], 48, 1, 64, 40, 3),
    ([513], [0], 16, 2, 64, 300, 1), ([130], [700], 24, 3, 128, 500, 20),
    # six units and more for each CTA, of two tiles to ten, with heads of 128 and of 64
    ([1500, 333, 40], [0, 700, 0], 128, 8, 128, 300, 20), ([5000], [0], 64, 8, 128, 1000, 0),
    ([3000, 1100], [0, 129], 64, 8, 64, 700, 64),
])
def test_prefill_wide_groups_and_many_units(kda_lib, cuda_dev, lens, hist, Hq, Hkv, d, window, sinks):
    import serving_kda_chunked_gated_gb300.kda as kda
    q, k, v, cu, cuk = _inputs(lens, hist, Hq, Hkv, d, seed=Hq + d)
    ro, rl, size = _reference_on(cuda_dev, q, k, v, cu, cuk, window, sinks)
    o, lse = kda.window_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), window, sinks, cu.to(cuda_dev), cu,
                                cuk.to(cuda_dev), cuk, want_lse=True)
    check_window(o, ro, size)
    _lse_ok(lse, rl, q, k, d ** -0.5)
