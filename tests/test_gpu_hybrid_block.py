"""The hybrid stack's mixers as a model runs them: a linear-attention layer (ShortConv +
Swish, gated delta rule, output gate) and a local softmax layer (per-head norm with
rotation, windowed attention), on packed prompts, then token by token from the states and
caches that the prompts left.  The decoded outputs are those of the same layers over the
whole sequences in 64 bits.

Tolerance: the prompts and the tokens go through the layers in bf16 at the same places
(convolution, attention and gate outputs), each a rounding of at most 2^-8, on top of the
layers' own: 1e-2 relative to a head's outputs, six such roundings in quadrature."""
import pytest
import torch

from hybrid_testutil import gdn_reference, rel, rope_reference, visible

pytestmark = pytest.mark.gpu

HK, HV, HQ, HKV, D, W, SINKS, CONV = 2, 4, 4, 2, 128, 50, 3, 4
TOL = 1e-2


def _bf(g, *s, scale=1.0):
    return (scale * torch.randn(*s, generator=g)).to(torch.bfloat16)


def _weights(g):
    C = (2 * HK + HV) * D
    return dict(conv=torch.randn(C, CONV, generator=g) / CONV, A=torch.log(1 + 7 * torch.rand(HV, generator=g)),
                qw=1 + 0.1 * torch.randn(D, generator=g), kw=1 + 0.1 * torch.randn(D, generator=g))


def _tables(P=4096):
    f = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _linear_reference(x, z, beta, g_in, w):
    """One sequence: convolution and Swish (rounded to bf16 as the kernel stores them), the rule, the gate."""
    T = x.shape[0]
    pad = torch.cat([torch.zeros(CONV - 1, x.shape[1]), x.float()])
    pre = sum(w["conv"].double()[:, i] * pad[i:i + T].double() for i in range(CONV))
    y = (pre * torch.sigmoid(pre)).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, D)) for t in y.split([HK * D, HK * D, HV * D], 1))
    o, S = gdn_reference(q, k, v, z, beta, w["A"], [0, T])
    return o, S, torch.sigmoid(g_in.double()) * o / (o.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()


def _window_reference(x, w, cos, sin):
    T = x.shape[0]
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([HQ * D, HKV * D, HKV * D], 1))
    pos = torch.arange(T)
    q = rope_reference(q, w["qw"], cos, sin, pos, False)[0].to(torch.bfloat16).double()
    k = rope_reference(k, w["kw"], cos, sin, pos, False)[0].to(torch.bfloat16).double()
    o = torch.zeros(T, HQ, D, dtype=torch.float64)
    for t in range(T):
        j = torch.tensor(visible(t, W, SINKS))
        for h in range(HQ):
            s = k[j, h // (HQ // HKV)] @ q[t, h] * D ** -0.5
            o[t, h] = torch.softmax(s, 0) @ v[j, h // (HQ // HKV)].double()
    return o


def test_prompts_then_tokens(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator().manual_seed(17)
    w = _weights(g)
    lens, steps = [140, 1, 67], 5
    full = [n + steps for n in lens]
    C = (2 * HK + HV) * D
    xl = [_bf(g, n, C) for n in full]
    xw = [_bf(g, n, (HQ + 2 * HKV) * D) for n in full]
    z = [1.5 * torch.randn(n, HV, generator=g) - 3 for n in full]
    beta = [torch.sigmoid(torch.randn(n, HV, generator=g)) for n in full]
    gin = [_bf(g, n, HV, D) for n in full]
    cos, sin = _tables()
    dev = lambda t: t.to(cuda_dev)                                                   # noqa: E731
    cat = lambda ts: dev(torch.cat([t[:n] for t, n in zip(ts, lens)]))               # noqa: E731
    at = lambda ts, s: dev(torch.stack([t[n + s] for t, n in zip(ts, lens)]))        # noqa: E731
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    cud, wd = dev(cu), {k: dev(t) for k, t in w.items()}
    slots = torch.tensor([2, 0, 3], dtype=torch.int32)
    sd, cosd, sind = dev(slots), dev(cos), dev(sin)
    N, pool = len(lens), 5
    conv_pool = torch.zeros(pool, CONV - 1, C, device=cuda_dev)
    state_pool = torch.zeros(pool, HV, D, D, device=cuda_dev)
    kc, vc = (torch.zeros(pool, SINKS + W, HKV, D, dtype=torch.bfloat16, device=cuda_dev) for _ in "kv")

    # the prompts
    y, conv = kda.short_conv(cat(xl), wd["conv"], cu_seqlens=cud)
    q, k, v = (t.unflatten(1, (-1, D)).contiguous() for t in y.split([HK * D, HK * D, HV * D], 1))
    o, S = kda.gdn_prefill(q, k, v, cat(z), cat(beta), wd["A"], cu_seqlens=cud, cu_seqlens_host=cu)
    yl = kda.gate_norm(o, cat(gin))
    conv_pool[sd.long()], state_pool[sd.long()] = conv, S
    pos = dev(torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]))
    split = lambda x: [t.unflatten(1, (-1, D)) for t in x.split([HQ * D, HKV * D, HKV * D], 1)]       # noqa: E731
    qw, kw, vw = split(cat(xw))
    qr, kr = kda.qk_norm_rope(qw, kw, cosd, sind, pos, q_weight=wd["qw"], k_weight=wd["kw"])
    ow = kda.window_prefill(qr, kr, vw, W, SINKS, cu_seqlens=cud, cu_seqlens_host=cu, k_cache=kc, v_cache=vc, slots=sd)
    got_l, got_w = [yl[cu[n]:cu[n + 1]] for n in range(N)], [ow[cu[n]:cu[n + 1]] for n in range(N)]

    # the tokens
    for s in range(steps):
        y = kda.short_conv_step(at(xl, s), wd["conv"], conv_pool, slots=sd)
        q, k, v = (t.unflatten(1, (-1, D)).contiguous() for t in y.split([HK * D, HK * D, HV * D], 1))
        o = kda.gdn_decode_step(q, k, v, at(z, s), at(beta, s), wd["A"], state_pool, slots=sd)
        yl = kda.gate_norm(o, at(gin, s))
        pos = dev(torch.tensor([n + s for n in lens], dtype=torch.int32))
        qw, kw, vw = split(at(xw, s))
        qr, kr = kda.qk_norm_rope(qw, kw, cosd, sind, pos, q_weight=wd["qw"], k_weight=wd["kw"])
        ow = kda.window_decode(qr, kr, vw, kc, vc, pos, W, SINKS, slots=sd)
        for n in range(N):
            got_l[n] = torch.cat([got_l[n], yl[n:n + 1]])
            got_w[n] = torch.cat([got_w[n], ow[n:n + 1]])

    for n in range(N):
        _, S, yl = _linear_reference(xl[n], z[n], beta[n], gin[n], w)
        rw = _window_reference(xw[n], w, cos, sin)
        for h in range(HV):
            assert rel(got_l[n][:, h], yl[:, h]) < TOL, (n, h, rel(got_l[n][:, h], yl[:, h]))
            assert rel(got_l[n][lens[n]:, h], yl[lens[n]:, h]) < TOL
            # the convolution's bf16 outputs may differ by a step where its float32 sum and the 64-bit
            # one fall on two sides of a rounding boundary: 2^-8 of single values
            assert rel(state_pool[slots[n], h], S[0, h]) < 1e-3
        for h in range(HQ):
            assert rel(got_w[n][:, h], rw[:, h]) < TOL and rel(got_w[n][lens[n]:, h], rw[lens[n]:, h]) < TOL
    assert (state_pool[[1, 4]] == 0).all() and (kc[[1, 4]] == 0).all()


def test_two_streams_at_once(kda_lib, cuda_dev):
    """Every mixer on two streams at the same time, workspaces apart: the bits of one call after another."""
    import serving_kda_chunked_gated_gb300.kda as kda
    bf = torch.bfloat16

    def inputs(seed, lens):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)                                          # noqa: E731
        T = sum(lens)
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
        d = dict(q=r(T, 8, 128).to(bf), k=r(T, 4, 128).to(bf), v=r(T, 8, 128).to(bf), z=r(T, 8) - 3, beta=torch.sigmoid(r(T, 8)),
                 A=torch.zeros(8), cos=r(T, 64), sin=r(T, 64), pos=torch.arange(T, dtype=torch.int32), cu=cu,
                 kc=torch.zeros(len(lens), 210, 4, 128).to(bf), vc=torch.zeros(len(lens), 210, 4, 128).to(bf),
                 last=torch.tensor(lens, dtype=torch.int32), ws=torch.zeros(1 << 25, dtype=torch.uint8))
        return {n: x.to(cuda_dev) for n, x in d.items()}, cu

    def run(d, cu, stream):
        n = len(cu) - 1
        o, S = kda.gdn_prefill(d["k"], d["k"], d["v"], d["z"], d["beta"], d["A"], d["cu"], cu, workspace=d["ws"], stream=stream)
        q, k = kda.qk_norm_rope(d["q"], d["k"], d["cos"], d["sin"], d["pos"], stream=stream)
        w = kda.window_prefill(q, k, k, 200, 10, d["cu"], cu, k_cache=d["kc"], v_cache=d["vc"], stream=stream)
        kda.gdn_decode_step(k[:n], k[:n], d["v"][:n], d["z"][:n], d["beta"][:n], d["A"], S, stream=stream)
        x = kda.window_decode(q[:n], k[:n], k[:n], d["kc"], d["vc"], d["last"], 200, 10, stream=stream)
        return [o, S, q, k, w, x, d["kc"], d["vc"]]

    sets = [([700, 30, 129], 1), ([64, 900], 2)]
    alone = []
    for lens, seed in sets:
        alone.append([t.clone() for t in run(*inputs(seed, lens), torch.cuda.current_stream())])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        data = [inputs(seed, lens) for lens, seed in sets]
        torch.cuda.synchronize()
        both = [run(*d, s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(kda.device_error(d["ws"]) == kda.KDA_OK for d, _ in data) and kda.device_error(None) == kda.KDA_OK


def test_offsets_past_32_bits(kda_lib, cuda_dev):
    """State pools, ring caches and packed projections whose last elements lie behind 2^32 bytes (and
    2^31 elements): the same bits as from small ones."""
    import serving_kda_chunked_gated_gb300.kda as kda
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(cuda_dev)                                 # noqa: E731
    # delta rule: the last slot of a pool of 2^17 + 1 states of 64 KiB (8.6 GB)
    slots = 2 ** 17 + 1
    q, k, v, z, beta, A = r(1, 1, 128).to(bf), r(1, 1, 128).to(bf), r(1, 1, 128).to(bf), r(1, 1), torch.sigmoid(r(1, 1)), r(1)
    small = r(1, 1, 128, 128)
    pool = torch.empty(slots, 1, 128, 128, device=cuda_dev)
    pool[-1] = small[0]
    at = torch.tensor([slots - 1], dtype=torch.int32, device=cuda_dev)
    assert torch.equal(kda.gdn_decode_step(q, k, v, z, beta, A, pool, slots=at), kda.gdn_decode_step(q, k, v, z, beta, A, small))
    assert torch.equal(pool[-1], small[0])
    del pool
    # window: positions near the end of rings of 2^21 + 300 rows of 8 heads of 128 (4.3 GB each)
    W, rows = 250, 2 ** 21 + 300
    q, k, v, hist = r(1, 16, 128).to(bf), r(1, 8, 128).to(bf), r(1, 8, 128).to(bf), r(W - 1, 8, 128).to(bf)
    want = None
    for n, pos in ((W, W - 1), (rows, rows - 1)):
        kc, vc = (torch.empty(1, n, 8, 128, dtype=bf, device=cuda_dev) for _ in "kv")
        kc[0, pos - W + 1:pos], vc[0, pos - W + 1:pos] = hist, -hist
        o = kda.window_decode(q, k, v, kc, vc, torch.tensor([pos], dtype=torch.int32, device=cuda_dev), W)
        assert torch.equal(kc[0, pos], k[0]) and torch.equal(vc[0, pos], v[0])
        want = o if want is None else want
        assert torch.equal(o, want)
        del kc, vc
    # norm and rotation, window prefill: tokens 2^31 + 64 elements apart
    far = torch.empty(2 ** 31 + 4096, dtype=bf, device=cuda_dev)
    step = 2 ** 31 + 64
    tok = r(2, 16 + 2 + 2, 128).to(bf)
    heads = lambda a, n: torch.as_strided(far, (2, n, 128), (step, 128, 1), a * 128)         # noqa: E731
    heads(0, 20).copy_(tok)
    cos, sin, pos = r(4, 64), r(4, 64), torch.tensor([1, 3], dtype=torch.int32, device=cuda_dev)
    got = kda.qk_norm_rope(heads(0, 16), heads(16, 2), cos, sin, pos)
    ref = kda.qk_norm_rope(tok[:, :16].contiguous(), tok[:, 16:18].contiguous(), cos, sin, pos)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = kda.window_prefill(heads(0, 16), heads(16, 2), heads(18, 2), 5)
    assert torch.equal(got, kda.window_prefill(*(x.contiguous() for x in (tok[:, :16], tok[:, 16:18], tok[:, 18:])), 5))


def test_prompts_captured(kda_lib, cuda_dev):
    """The prompts' calls in a graph: bounds left out (one sequence) and given, the ring caches filled beside the
    prefill.  Each replay on new inputs leaves the bits of the same calls outside a graph."""
    import serving_kda_chunked_gated_gb300.kda as kda
    g = torch.Generator(device=cuda_dev).manual_seed(53)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_dev)                              # noqa: E731
    bf, T = torch.bfloat16, 700
    x = dict(q=r(T, 4, 128).to(bf), k=r(T, 2, 128).to(bf), v=r(T, 2, 128).to(bf), z=r(T, 2) - 3, beta=torch.sigmoid(r(T, 2)))
    A, kc, vc = torch.zeros(2, device=cuda_dev), *(torch.zeros(3, 110, 2, 128, dtype=bf, device=cuda_dev) for _ in "kv")
    cu = torch.tensor([0, 300, 300, T], dtype=torch.int32)
    cud, slots = cu.to(cuda_dev), torch.tensor([2, 1, 0], dtype=torch.int32, device=cuda_dev)

    def run():
        a = kda.gdn_prefill(x["k"], x["k"], x["v"], x["z"], x["beta"], A)
        w = kda.window_prefill(x["q"], x["k"], x["v"], 100, 10)
        k0, v0 = kc[:1], vc[:1]
        u = kda.window_prefill(x["q"], x["k"], x["v"], 60, 3, k_cache=k0, v_cache=v0)
        t = kda.window_prefill(x["q"], x["k"], x["v"], 100, 10, cud, cu, k_cache=kc, v_cache=vc, slots=slots)
        return [*a, w, u, t]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(2):
        for n, t in x.items():
            t.copy_(torch.sigmoid(r(*t.shape)) if n == "beta" else r(*t.shape) - (3 if n == "z" else 0))
        for c in (kc, vc):
            c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held + [kc, vc]]
        for c in (kc, vc):
            c.zero_()
        want = run() + [kc, vc]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kda.device_error(None) == kda.KDA_OK
