"""Scalar-gated delta rule on the GPU (prefill and decode) against its recurrence in 64 bits.

Tolerances.  States: float32 throughout; each product that reaches them keeps 16
bits or more of its float32 operand (two bf16 parts, 2^-17), a few such roundings
for each 128-token chunk, so 1e-5 relative to the state's norm per head.  Outputs:
the chunked form rounds the state, the masked products and the update to bf16 once
each for its output alone, and the output itself: four roundings of at most 2^-8,
2^-8 / sqrt(3) in root mean square, which add up in quadrature to
2 * 2^-8 / sqrt(3) = 4.5e-3."""
import pytest
import torch

from hybrid_testutil import gdn_inputs, gdn_reference, rel

pytestmark = pytest.mark.gpu

TOL_S, TOL_O = 1e-5, 4.5e-3


def _dev(d, dev):
    return {k: x.to(dev) for k, x in d.items()}


def _check(o, S, ro, rS, lens, tol_o=TOL_O):
    # a state or output below float32's smallest normal number, 2^-126, has no float32 value to
    # be compared with (the library flushes denormals): it counts as zero on both sides
    small = 2.0 ** -126
    rS, ro = rS.masked_fill(rS.abs() < small, 0.0), ro.masked_fill(ro.abs() < small, 0.0)
    assert torch.isfinite(o.float()).all() and torch.isfinite(S).all()
    for n in range(rS.shape[0]):
        for h in range(rS.shape[1]):
            assert rel(S[n, h], rS[n, h]) < TOL_S, (n, h, lens[n], rel(S[n, h], rS[n, h]))
    if o.numel():
        for h in range(o.shape[1]):
            assert rel(o[:, h], ro[:, h]) < tol_o, (h, rel(o[:, h], ro[:, h]))


@pytest.mark.parametrize("lens,Hk,Hv,gate,s0", [
    ([1], 1, 1, "softplus", True), ([2], 2, 2, "bounded", False), ([16, 17], 1, 3, "softplus", True),
    ([127], 2, 2, "softplus", False), ([128], 1, 2, "bounded", True), ([129], 2, 4, "softplus", True),
    ([0, 5, 0, 130, 1, 256, 0], 2, 4, "softplus", True), ([700], 1, 2, "softplus", False), ([385], 4, 4, "bounded", True),
])
@pytest.mark.parametrize("recurrent", [False, True])
def test_prefill(kda_lib, cuda_dev, lens, Hk, Hv, gate, s0, recurrent):
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs(lens, Hk, Hv, seed=len(lens) + lens[0])
    S0 = d.pop("S0") if s0 else (d.pop("S0"), None)[1]
    ro, rS = gdn_reference(**d, cu=cu, S0=S0, gate=gate)
    g = _dev(d, cuda_dev)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=cuda_dev).fill_(255)      # whatever it held
    o, S = kda.gdn_prefill(**g, cu_seqlens=cu.to(cuda_dev), cu_seqlens_host=cu, gate=gate, recurrent=recurrent,
                           S0=None if S0 is None else S0.to(cuda_dev), workspace=ws)
    assert recurrent or kda.device_error(ws) == kda.KDA_OK
    _check(o, S, ro, rS, lens)


def test_prefill_float32(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([70, 3], 2, 4, dtype=torch.float32)
    ro, rS = gdn_reference(**d, cu=cu)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev))
    assert o.dtype == torch.float32
    _check(o, S, ro, rS, [70, 3], tol_o=TOL_S)


@pytest.mark.parametrize("z_mean,beta", [(9.0, None), (-30.0, None), (-3.0, 0.0), (-3.0, 1.0), (-30.0, 1.0)])
def test_prefill_extreme_gates(kda_lib, cuda_dev, z_mean, beta):
    """Decays of almost nothing in one token, no decay at all, writes of strength 0 and 1
    with strongly correlated keys (the triangular inverse at its worst)."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([300], 1, 2, z_mean=z_mean, seed=7)
    base = torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(1))
    d["k"] = (base + 0.5 * torch.randn(300, 1, 128, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    if beta is not None:
        d["beta"].fill_(beta)
    ro, rS = gdn_reference(**d, cu=cu)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev))
    _check(o, S, ro, rS, [300])


def test_prefill_no_l2norm_scale_g_min(kda_lib, cuda_dev):
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([200], 1, 2, seed=3)
    d["k"] = (d["k"].float() * 0.15).to(torch.bfloat16)
    ro, rS = gdn_reference(**d, cu=cu, l2=False, scale=0.25, gate="bounded", g_min=-1.5)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), qk_l2norm=False, scale=0.25, gate="bounded",
                           g_min=-1.5)
    _check(o, S, ro, rS, [200])


def test_prefill_split_resume_matches_whole(kda_lib, cuda_dev):
    """The state carried between two calls, in place (S_T = S0)."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([500], 2, 4, seed=5)
    S = d["S0"].to(cuda_dev)
    ro, rS = gdn_reference(**d, cu=cu)
    g = _dev(d, cuda_dev)
    g.pop("S0")
    parts = []
    for a, b in ((0, 177), (177, 500)):
        x = {k: (t[a:b].contiguous() if k != "A" else t) for k, t in g.items()}
        out = dict(o=torch.empty_like(x["v"]), S_T=S)
        parts.append(kda.gdn_prefill(**x, S0=S, out=out)[0])
    _check(torch.cat(parts), S, ro, rS, [500])


def test_prefill_neighbours_do_not_leak(kda_lib, cuda_dev):
    """NaN and infinity in one packed sequence leave the others bit for bit as they were."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens = [100, 60, 200]
    d, cu = gdn_inputs(lens, 1, 2, seed=9)
    g = _dev(d, cuda_dev)
    o, S = kda.gdn_prefill(**g, cu_seqlens=cu.to(cuda_dev))
    for bad in (float("nan"), float("inf")):
        h = {k: x.clone() for k, x in g.items()}
        for name in ("q", "k", "v", "z", "beta"):
            h[name][100:160] = bad
        h["S0"][1] = bad
        o2, S2 = kda.gdn_prefill(**h, cu_seqlens=cu.to(cuda_dev))
        for n, (a, b) in ((0, (0, 100)), (2, (160, 360))):
            assert torch.equal(o2[a:b], o[a:b]) and torch.equal(S2[n], S[n])


def test_prefill_graph_stream_and_state_only(kda_lib, cuda_dev):
    """Captured and replayed on new inputs, on a stream of its own; want_o=False gives the same states."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens = [130, 1, 40]
    d1, cu = gdn_inputs(lens, 2, 4, seed=11)
    d2, _ = gdn_inputs(lens, 2, 4, seed=12)
    g, cud = _dev(d1, cuda_dev), cu.to(cuda_dev)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=cuda_dev)
    call = lambda **kw: kda.gdn_prefill(**g, cu_seqlens=cud, cu_seqlens_host=cu, workspace=ws, **kw)     # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o_s, S_s = call(stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = call()
    for d in (d2, d1):
        for n, x in d.items():
            g[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        ro, rS = gdn_reference(**d, cu=cu)
        _check(o, S, ro, rS, lens)
    assert torch.equal(o, o_s) and torch.equal(S, S_s)
    none, S3 = call(want_o=False)
    assert none is None and torch.equal(S3, S)
    o4, none = call(want_state=False)
    assert none is None and torch.equal(o4, o)


@pytest.mark.parametrize("N,Hk,Hv,gate", [(1, 1, 1, "softplus"), (5, 2, 6, "bounded"), (40, 4, 8, "softplus")])
def test_decode(kda_lib, cuda_dev, N, Hk, Hv, gate):
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([1] * N, Hk, Hv, seed=N)
    S0 = d.pop("S0")
    ro, rS = gdn_reference(**d, cu=cu, S0=S0, gate=gate)
    g = _dev(d, cuda_dev)
    slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32)
    state = torch.full((N + 3, Hv, 128, 128), 7.0)
    state[slots.long()] = S0
    state = state.to(cuda_dev)
    o = kda.gdn_decode_step(**g, state=state, slots=slots.to(cuda_dev), gate=gate)
    got = state.cpu()
    _check(o, got[slots.long()], ro, rS, [1] * N)
    rest = sorted(set(range(N + 3)) - set(slots.tolist()))
    assert (got[rest] == 7.0).all()


def test_decode_skips_slots_out_of_range_and_follows_prefill(kda_lib, cuda_dev):
    """A prefill's states go on token by token; a bad slot leaves its row and all states alone."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens = [150, 20]
    d, cu = gdn_inputs(lens, 1, 2, seed=21)
    ro, rS = gdn_reference(**d, cu=cu)
    g = _dev(d, cuda_dev)
    at = torch.tensor([[149, 169]])
    head = torch.cat([torch.arange(149), torch.arange(150, 169)])
    part = {k: (x[head].contiguous() if k not in ("A", "S0") else x) for k, x in g.items()}
    _, S = kda.gdn_prefill(**part, cu_seqlens=torch.tensor([0, 149, 168], dtype=torch.int32, device=cuda_dev))
    x = {k: t[at[0]].contiguous() for k, t in g.items() if k not in ("A", "S0")}
    before = S.clone()
    out = torch.full((2, 2, 128), 3.0, dtype=torch.bfloat16, device=cuda_dev)
    kda.gdn_decode_step(**x, A=g["A"], state=S, slots=torch.tensor([-1, 2], dtype=torch.int32, device=cuda_dev), out=out)
    assert torch.equal(S, before) and (out == 3.0).all()
    o = kda.gdn_decode_step(**x, A=g["A"], state=S)
    _check(o, S, ro[at[0]], rS, lens)


def test_prefill_many_sequences(kda_lib, cuda_dev):
    """More sequences than the host lists for the kernels, empty ones and one of two chunks among them."""
    import serving_kda_chunked_gated_gb300.kda as kda
    for n in (1024, 1025):
        lens = [(7 * i) % 13 for i in range(n)]
        lens[n // 2], lens[-1], lens[0] = 131, 0, 30
        d, cu = gdn_inputs(lens, 1, 1, seed=n)
        d.pop("S0")
        ro, rS = gdn_reference(**d, cu=cu)
        o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), cu_seqlens_host=cu)
        _check(o, S, ro, rS, lens)


def test_prefill_no_tokens(kda_lib, cuda_dev):
    """Only empty sequences: the states pass through, or nothing is asked for."""
    import serving_kda_chunked_gated_gb300.kda as kda
    bf, e = torch.bfloat16, lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=cuda_dev)     # noqa: E731
    cu = torch.zeros(4, dtype=torch.int32)
    q, k, v = e(0, 2, 128, dt=bf), e(0, 2, 128, dt=bf), e(0, 4, 128, dt=bf)
    S0 = torch.randn(3, 4, 128, 128, device=cuda_dev)
    for rec in (False, True):
        args = (q, k, v, e(0, 4), e(0, 4), torch.zeros(4, device=cuda_dev), cu.to(cuda_dev), cu)
        assert torch.equal(kda.gdn_prefill(*args, S0=S0, recurrent=rec)[1], S0)
        assert (kda.gdn_prefill(*args, recurrent=rec)[1] == 0).all()
        assert kda.gdn_prefill(*args, want_state=False, recurrent=rec)[0].numel() == 0


@pytest.mark.parametrize("gate", ["softplus", "bounded"])
def test_prefill_short_sequences_beside_long_ones(kda_lib, cuda_dev, gate):
    """One-token sequences packed with prompts (the former by the recurrence, beside the latter's scan):
    states in place, and what a captured call leaves on its second replay."""
    import serving_kda_chunked_gated_gb300.kda as kda
    lens = [1] * 20 + [200, 0, 24, 25] + [1] * 20 + [129, 3]
    d, cu = gdn_inputs(lens, 2, 4, seed=5)
    S0 = d.pop("S0")
    ro, rS = gdn_reference(**d, cu=cu, S0=S0, gate=gate)
    g, cud, S = _dev(d, cuda_dev), cu.to(cuda_dev), S0.to(cuda_dev)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=cuda_dev).fill_(255)
    out = {"o": torch.empty_like(g["v"]), "S_T": S}
    call = lambda: kda.gdn_prefill(**g, cu_seqlens=cud, cu_seqlens_host=cu, gate=gate, S0=S, out=out, workspace=ws)     # noqa: E731
    call()
    assert kda.device_error(ws) == kda.KDA_OK
    _check(out["o"], S, ro, rS, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        S.copy_(S0)
        graph.replay()
        _check(out["o"], S, ro, rS, lens)
    assert kda.device_error(ws) == kda.KDA_OK


@pytest.mark.parametrize("near_whole", [False, True])
def test_prefill_slow_decay_over_half_a_million_tokens(kda_lib, cuda_dev, near_whole):
    """Without writes (beta 0) the state is S0 times the product of all decays, and a bias of any step shows:
    steps of some 1e-6, 4096 chunks.  near_whole: steps just below a multiple of 2^-32 (base 2).

    Tolerance: a chunk's factor is rounded by 2^-25 and the state's update by 2^-24 at most, uniformly
    distributed and independent over 4096 chunks: 64 sqrt(1 / 3) (2^-24 + 2^-25) = 3.3e-6; the gate's
    float32 log-decay is within 2^-19 (its exponential's 2 + |1.2 z| units in the last place), of a total
    of 0.6: 1.2e-6.  Together below TOL_S."""
    import serving_kda_chunked_gated_gb300.kda as kda
    T = 1 << 19
    g = torch.Generator().manual_seed(23)
    z = -18 + 6 * torch.rand(2 * T if not near_whole else 12 * T, generator=g)
    if near_whole:
        step = torch.log1p(z.double().exp()) / torch.log(torch.tensor(2.0, dtype=torch.float64)) * 2.0 ** 32
        z = z[step - step.floor() > 0.8]
    z = z[:T]
    assert len(z) == T
    S0 = torch.randn(1, 1, 128, 128, generator=g)
    x = torch.randn(T, 1, 128, generator=g).to(torch.bfloat16).to(cuda_dev)
    zero = torch.zeros(T, 1, device=cuda_dev)
    _, S = kda.gdn_prefill(x, x, x, z[:, None].to(cuda_dev), zero, torch.zeros(1, device=cuda_dev), S0=S0.to(cuda_dev))
    want = S0.double() * torch.exp(-torch.log1p(z.double().exp()).sum())
    assert rel(S, want) < TOL_S, rel(S, want)


@pytest.mark.parametrize("T,Hk,Hv,gate,z_mean", [(20000, 1, 2, "softplus", -3.0), (20000, 1, 2, "bounded", -1.5),
                                                 (9001, 1, 1, "softplus", -9.0)])
def test_prefill_hundreds_of_chunks(kda_lib, cuda_dev, T, Hk, Hv, gate, z_mean):
    """The error does not grow with the chunks: long prompts, ordinary and slow decay, against 64 bits."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([T], Hk, Hv, seed=T, z_mean=z_mean)
    ro, rS = gdn_reference(**d, cu=cu, gate=gate)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), gate=gate)
    _check(o, S, ro, rS, [T])


@pytest.mark.parametrize("lens,Hk,Hv,gate", [([3000], 1, 2, "softplus"), ([1, 700, 0, 129, 24], 2, 6, "bounded")])
def test_prefill_float32_long_and_packed(kda_lib, cuda_dev, lens, Hk, Hv, gate):
    """Tolerance as for the states: float32 throughout, an output rounds to 2^-24."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs(lens, Hk, Hv, seed=lens[0], dtype=torch.float32)
    ro, rS = gdn_reference(**d, cu=cu, gate=gate)
    for recurrent in (False, True):
        o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), cu_seqlens_host=cu, gate=gate,
                               recurrent=recurrent)
        _check(o, S, ro, rS, lens, tol_o=TOL_S)


@pytest.mark.parametrize("keys,beta", [("same", None), ("same", 1.0), ("near", 1.0), ("turned", None)])
def test_prefill_keys_alike(kda_lib, cuda_dev, keys, beta):
    """A token repeated, or keys that differ by a few percent, and no decay: what the updates write then cancels
    from token to token, and an output formed from rounded updates would be off by many of its own roundings.

    Tolerance of the outputs as above.  States: V'' = T R cancels the same way, and each of a chunk's 128 updates
    is off by 2^-17 of R, uniformly distributed: sqrt(128 / 3) 2^-17 sqrt(2) = 7e-5 at most."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([700], 1, 2, z_mean=-30.0, seed=41)
    g = torch.Generator().manual_seed(41)
    k = torch.randn(1, 1, 128, generator=g)
    d["k"] = (k + (0.05 if keys == "near" else 0.0) * torch.randn(700, 1, 128, generator=g)).to(torch.bfloat16)
    if keys == "turned":
        d["k"][1::2] *= -1
    if beta is not None:
        d["beta"].fill_(beta)
    ro, rS = gdn_reference(**d, cu=cu)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev))
    for h in range(2):
        assert rel(o[:, h], ro[:, h]) < TOL_O, rel(o[:, h], ro[:, h])
        assert rel(S[0, h], rS[0, h]) < 7e-5, rel(S[0, h], rS[0, h])


ONCE = 2.4e-3    # bf16's own rounding, 2^-8 / sqrt(3) = 2.26e-3 at most in root mean square, and two operands of 11 bits


@pytest.mark.parametrize("lens,Hk,Hv,gate", [([700], 1, 2, "softplus"), ([300, 129, 64], 2, 2, "bounded")])
def test_prefill_outputs_round_once(kda_lib, cuda_dev, lens, Hk, Hv, gate):
    """Each of the masked product's operands is rounded to 11 bits (2^-11 / sqrt(3) = 2.8e-4), o to 8."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs(lens, Hk, Hv, seed=43)
    ro, rS = gdn_reference(**d, cu=cu, gate=gate)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), gate=gate)
    _check(o, S, ro, rS, lens, tol_o=ONCE)


@pytest.mark.parametrize("what", ["v tiny", "v huge", "v of all sizes", "zero v", "q, k of all sizes", "k huge", "scale tiny"])
def test_prefill_sizes_beyond_fp16(kda_lib, cuda_dev, what):
    """Values, queries and keys (not normalised) far outside fp16's range: nothing of the masked product may be
    lost.  Sizes change by powers of two up to 2^12 from token to token, where they do."""
    import serving_kda_chunked_gated_gb300.kda as kda
    d, cu = gdn_inputs([500], 1, 2, seed=47)
    g = torch.Generator().manual_seed(47)
    sizes = torch.exp2(torch.randint(-6, 7, (500, 1, 1), generator=g).float())
    kw, times = {}, lambda n, x: d.__setitem__(n, (d[n].float() * x).to(torch.bfloat16))          # noqa: E731
    if what == "v tiny":
        times("v", 1e-20)
        d["S0"].mul_(1e-20)
    elif what == "v huge":
        times("v", 1e20)
        d["S0"].mul_(1e20)
    elif what == "v of all sizes":
        times("v", sizes)
    elif what == "zero v":
        d["v"].zero_()
        d["S0"].zero_()
    elif what == "scale tiny":
        kw["scale"] = 1e-9
    else:
        kw["l2"] = False
        times("k", 0.15)                                     # norms near 1
        times("q", 1e4 * sizes if what[0] == "q" else 1e-9)
        if what[0] == "q":
            # a key's size with a write strength that keeps its update stable
            s = torch.exp2(torch.randint(-6, 1, (500, 1), generator=g).float())
            times("k", s[..., None])
        else:
            times("k", 2.0 ** 20)
            d["beta"].mul_(2.0 ** -40)
    ro, rS = gdn_reference(**d, cu=cu, **kw)
    o, S = kda.gdn_prefill(**_dev(d, cuda_dev), cu_seqlens=cu.to(cuda_dev), scale=kw.get("scale", 1.0),
                           qk_l2norm=kw.get("l2", True))
    if what == "zero v":
        assert (o == 0).all() and (S == 0).all()
        return
    _check(o, S, ro, rS, [500], tol_o=ONCE)
    # and token by token: no row is off by more than the largest of its chunk's and its own roundings
    for h in range(2):
        row = ro[:, h].norm(dim=-1)
        off = (o[:, h].double().cpu() - ro[:, h]).norm(dim=-1)
        assert (off <= 2.0 ** -8 * row + 2.0 ** -9 * torch.stack([row[c // 128 * 128:c + 1].max() for c in range(500)])).all()
