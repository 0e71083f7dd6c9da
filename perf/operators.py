"""Cases of the hybrid token mixers: the scalar-gated delta rule (prefill and decode), the per-head
norm with rotation of queries and keys, and sliding-window attention with sinks (prefill and decode).

``listed()`` names the measured cases, ``draw()`` gives more of the same ranges, ``run()`` is one pass
through an operator: in its plain form (elementary torch operations in 32 bits), or, with ``own``
set, through the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

D = 128     # key and value width of the delta rule's heads


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one long document resumed from a prefix state: the sequential chunk pass decides
        dict(name="gdn_prefill_128k", op="gdn_prefill", lens="131072", hk=16, hv=32, gate="softplus", s0=True),
        # the ordinary prompt, as many key heads as value heads, the bounded gate
        dict(name="gdn_prefill_8k", op="gdn_prefill", lens="8192", hk=32, hv=32, gate="bounded", s0=False),
        # a packed batch of prompts with one-token and odd lengths
        dict(name="gdn_prefill_ragged", op="gdn_prefill", lens="1,17,64,129,1000,4097,2500,0,333", hk=4, hv=16,
             gate="softplus", s0=True),
        # a full serving batch, states through a slot table
        dict(name="gdn_decode_256", op="gdn_decode", n=256, hk=16, hv=32, gate="softplus"),
        # one sequence: latency
        dict(name="gdn_decode_1", op="gdn_decode", n=1, hk=4, hv=8, gate="softplus"),
        # the queries and keys of a long prompt, read out of the packed projection
        dict(name="rope_32k", op="rope", t=32768, hq=32, hkv=8, d=128, rot=128, style="half", dtype="bf16"),
        # a decode batch in float32, half of each head rotated, neighbouring pairs
        dict(name="rope_f32_257", op="rope", t=257, hq=16, hkv=2, d=64, rot=32, style="pairs", dtype="f32"),
        # a long document through a short window
        dict(name="window_prefill_128k", op="window_prefill", lens="131072", hist="0", hq=32, hkv=8, d=128, window=512,
             sinks=4, cache=False),
        # the ordinary prompt through a long window
        dict(name="window_prefill_8k", op="window_prefill", lens="8192", hist="0", hq=32, hkv=8, d=128, window=4096,
             sinks=4, cache=False),
        # packed prompts of odd lengths, one resumed after earlier tokens, that also fill the ring caches
        dict(name="window_prefill_ragged", op="window_prefill", lens="1,333,64,1023,2049,130", hist="0,0,700,0,1,129",
             hq=24, hkv=4, d=64, window=1000, sinks=16, cache=True),
        # a full serving batch over long windows
        dict(name="window_decode_256", op="window_decode", n=256, hq=32, hkv=8, d=128, window=4096, sinks=4),
        # three sequences, short window: latency
        dict(name="window_decode_3", op="window_decode", n=3, hq=24, hkv=4, d=64, window=127, sinks=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdn_prefill", "gdn_prefill", "gdn_decode", "rope", "window_prefill", "window_prefill",
                     "window_decode"])
    if op == "gdn_prefill":
        hk = rng.choice([1, 2, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 3, 4])
        n = rng.choice([1, 1, 2, 5, 8])
        lens = [_log_int(rng, 1, 16384 // n) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), hk=hk, hv=min(hv, 32) if hk < 16 else rng.choice([16, 32]),
                    gate=rng.choice(["softplus", "bounded"]), s0=rng.random() < 0.5)
    if op == "gdn_decode":
        hk = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, n=_log_int(rng, 1, 256), hk=hk, hv=hk * rng.choice([1, 2]),
                    gate=rng.choice(["softplus", "bounded"]))
    if op == "rope":
        d = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, t=_log_int(rng, 1, 20000), hq=hkv * rng.choice([1, 2, 3, 4]), hkv=hkv, d=d,
                    rot=d // rng.choice([1, 2, 4]), style=rng.choice(["half", "pairs"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4])
    d, sinks = rng.choice([64, 128]), rng.choice([0, 1, 4, 64])
    if op == "window_prefill":
        n = rng.choice([1, 1, 2, 4, 6])
        lens = [_log_int(rng, 1, 12000 // n) for _ in range(n)]
        hist = [0 if rng.random() < 0.7 else _log_int(rng, 1, 3000) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), hist=",".join(map(str, hist)), hq=hq, hkv=hkv, d=d,
                    window=_log_int(rng, 1, 3500), sinks=sinks, cache=rng.random() < 0.3)
    return dict(op=op, n=_log_int(rng, 1, 200), hq=hq, hkv=hkv, d=d, window=_log_int(rng, 1, 4000), sinks=sinks)


def _ints(text):
    return [int(x) for x in str(text).split(",")]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _window_plan(lens, hist, window):
    """Blocks of at most B queries that lie in one sequence, for the plain form."""
    B = 256 if window <= 1024 else 512
    cu_q, cu_k = _cu(lens), _cu([a + b if a else 0 for a, b in zip(lens, hist)])
    rows = []
    for n, (ln, h) in enumerate(zip(lens, hist)):
        for a in range(0, ln, B):
            rows.append((cu_q[n] + a, min(B, ln - a), h + a, cu_k[n]))
    return B, torch.tensor(rows, dtype=torch.int64).reshape(-1, 4)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)           # noqa: E731
    bf = lambda x: x.to(torch.bfloat16)                                # noqa: E731
    st = dict(case=case)
    if op in ("gdn_prefill", "gdn_decode"):
        hk, hv = case["hk"], case["hv"]
        lens = _ints(case["lens"]) if op == "gdn_prefill" else None
        T = sum(lens) if lens is not None else case["n"]
        # q, k, v come out of ShortConv + Swish
        act = lambda x: bf(x * torch.sigmoid(x))                       # noqa: E731
        st["q"], st["k"], st["v"] = act(rn(T, hk, D)), act(rn(T, hk, D)), act(rn(T, hv, D))
        # decay logits with the bias in them: retention between about 0.2 and 1 for each token and head
        st["z"] = rn(T, hv) * 1.5 - 3.0
        st["beta"] = torch.sigmoid(rn(T, hv))
        st["A"] = torch.log(1 + 7 * torch.rand(hv, generator=g, device=dev))
        if op == "gdn_prefill":
            cu = _cu(lens)
            st["cu_host"] = torch.tensor(cu, dtype=torch.int32)
            st["cu"] = st["cu_host"].to(dev)
            st["S0"] = 0.1 * rn(len(lens), hv, D, D) if case["s0"] else None
            C = 64
            nc = max(1, max(-(-n // C) for n in lens))
            at = torch.full((len(lens), nc * C), -1, dtype=torch.int64)
            for n, ln in enumerate(lens):
                at[n, :ln] = torch.arange(cu[n], cu[n + 1])
            st["at"], st["chunk"] = at.to(dev), C
        else:
            slots = case["n"] + case["n"] // 4 + 1
            st["state"] = 0.3 * rn(slots, hv, D, D)
            st["slots"] = torch.randperm(slots, generator=g, device=dev)[:case["n"]].to(torch.int32)
        return st
    if op == "rope":
        T, hq, hkv, d, rot = (case[x] for x in ("t", "hq", "hkv", "d", "rot"))
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        qkv = rn(T, (hq + 2 * hkv) * d).to(dt)                          # one packed projection
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["qw"], st["kw"] = 1 + 0.1 * rn(d), 1 + 0.1 * rn(d)
        P = 65536                                                       # positions of the served context
        freq = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device=dev) * 2 / rot)
        ang = torch.arange(P, dtype=torch.float64, device=dev)[:, None] * freq
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = ((torch.arange(T, device=dev) + torch.randint(0, 1000, (1,), generator=g, device=dev)) % P
                     if T > 1024 else torch.randint(0, P, (T,), generator=g, device=dev)).to(torch.int32)
        return st
    hq, hkv, d, W, sinks = (case[x] for x in ("hq", "hkv", "d", "window", "sinks"))
    if op == "window_prefill":
        lens, hist = _ints(case["lens"]), _ints(case["hist"])
        klens = [a + b if a else 0 for a, b in zip(lens, hist)]
        st["q"], st["k"], st["v"] = bf(rn(sum(lens), hq, d)), bf(rn(sum(klens), hkv, d)), bf(rn(sum(klens), hkv, d))
        st["cu_host"], st["cuk_host"] = (torch.tensor(_cu(x), dtype=torch.int32) for x in (lens, klens))
        st["cu"], st["cuk"] = st["cu_host"].to(dev), st["cuk_host"].to(dev)
        st["block"], plan = _window_plan(lens, hist, W)
        st["plan"] = plan.to(dev)
        if case["cache"]:
            slots = len(lens) + 2
            st["kc"], st["vc"] = (torch.zeros(slots, sinks + W, hkv, d, dtype=torch.bfloat16, device=dev) for _ in "kv")
            st["slots"] = torch.randperm(slots, generator=g, device=dev)[:len(lens)].to(torch.int32)
            # rows of the packed keys that the caches hold afterwards, and where
            src, seq, row = [], [], []
            cuk = _cu(klens)
            for n, ln in enumerate(klens):
                for p in sorted(set(range(min(sinks, ln))) | set(range(max(sinks, ln - W), ln))):
                    src.append(cuk[n] + p)
                    seq.append(n)
                    row.append(p if p < sinks else sinks + (p - sinks) % W)
            st["fill"] = tuple(torch.tensor(x, dtype=torch.int64, device=dev) for x in (src, seq, row))
        return st
    n = case["n"]
    slots = n + n // 8 + 1
    st["q"], st["k"], st["v"] = bf(rn(n, hq, d)), bf(rn(n, hkv, d)), bf(rn(n, hkv, d))
    st["kc"], st["vc"] = (torch.randn(slots, sinks + W, hkv, d, generator=g, device=dev, dtype=torch.bfloat16) for _ in "kv")
    # most sequences are far past the window; a few have just begun
    pos = torch.randint(0, 8 * (W + sinks), (n,), generator=g, device=dev) + (W + sinks)
    early = torch.rand(n, generator=g, device=dev) < 0.1
    st["pos"] = torch.where(early, torch.randint(0, W + sinks, (n,), generator=g, device=dev), pos).to(torch.int32)
    st["slots"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return dict(gdn_prefill=_gdn_prefill, gdn_decode=_gdn_decode, rope=_rope, window_prefill=_window_prefill,
                window_decode=_window_decode)[state["case"]["op"]](state)


def _run_own(s):
    import serving_kda_chunked_gated_gb300.kda as kda
    c = s["case"]
    op = c["op"]
    if op == "gdn_prefill":
        o, S_T = kda.gdn_prefill(s["q"], s["k"], s["v"], s["z"], s["beta"], s["A"], cu_seqlens=s["cu"],
                                 cu_seqlens_host=s["cu_host"], S0=s["S0"], gate=c["gate"], workspace="cache")
        return {"o": o, "S": S_T}
    if op == "gdn_decode":
        o = kda.gdn_decode_step(s["q"], s["k"], s["v"], s["z"], s["beta"], s["A"], s["state"], slots=s["slots"],
                                gate=c["gate"])
        return {"o": o, "state": s["state"]}
    if op == "rope":
        q, k = kda.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["pos"], q_weight=s["qw"], k_weight=s["kw"],
                                interleaved=c["style"] == "pairs")
        return {"q": q, "k": k}
    if op == "window_prefill":
        more = dict(k_cache=s["kc"], v_cache=s["vc"], slots=s["slots"]) if c["cache"] else {}
        o, lse = kda.window_prefill(s["q"], s["k"], s["v"], window=c["window"], sinks=c["sinks"], cu_seqlens=s["cu"],
                                    cu_seqlens_host=s["cu_host"], cu_seqlens_k=s["cuk"],
                                    cu_seqlens_k_host=s["cuk_host"], want_lse=True, **more)
        return {"o": o, "lse": lse, **({"kc": s["kc"], "vc": s["vc"]} if c["cache"] else {})}
    o = kda.window_decode(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], window=c["window"], sinks=c["sinks"],
                          slots=s["slots"])
    return {"o": o, "kc": s["kc"], "vc": s["vc"]}


def _log_decay(z, A, gate):
    """The log of the retention, in 64 bits: its sums over a chunk are what the exponents are made of."""
    z, e = z.double(), torch.exp(A.double())
    if gate == "bounded":
        return -5.0 / (1 + torch.exp(-e * z))
    return -e * (torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs())))


def _l2(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower A [..., n, n], n a power of two: inverted diagonal blocks of
    doubling size, [[X, 0], [B, Y]]^-1 = [[X^-1, 0], [-Y^-1 B X^-1, Y^-1]]."""
    n = A.shape[-1]
    X = torch.eye(n, device=A.device, dtype=A.dtype).expand(A.shape).contiguous()
    b = 1
    while b < n:    # log2 n steps, each over all blocks at once
        i = torch.arange(0, n, 2 * b, device=A.device)[:, None] + torch.arange(b, device=A.device)
        hi, lo = i[:, :, None], i[:, None, :]
        top = X[..., hi, lo]
        bot = X[..., hi + b, lo + b]
        X[..., hi + b, lo] = -(bot @ A[..., hi + b, lo] @ top)
        b *= 2
    return X


def _gdn_prefill(s):
    c, at, C = s["case"], s["at"], s["chunk"]
    N, L = at.shape
    hk, hv = c["hk"], c["hv"]
    nc, live = L // C, (at >= 0)
    take = at.clamp(min=0)

    def chunks(x):          # [T, h, ...] -> [N, nc, h, C, ...], zeros behind a sequence's end
        y = x[take] * live.view(N, L, *([1] * (x.dim() - 1)))
        return y.unflatten(1, (nc, C)).transpose(2, 3)

    rep = hv // hk
    q = chunks(_l2(s["q"].float())).repeat_interleave(rep, dim=2)
    k = chunks(_l2(s["k"].float())).repeat_interleave(rep, dim=2)
    v, beta = chunks(s["v"].float()), chunks(s["beta"])
    gc = chunks(_log_decay(s["z"], s["A"], c["gate"])).cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    rel = torch.exp((gc[..., :, None] - gc[..., None, :]).masked_fill(~low, -1e30)).float()
    A = (beta[..., None] * (k @ k.transpose(-1, -2)) * rel).tril(-1)
    X = _unit_lower_inverse(A)
    e = torch.exp(gc).float()[..., None]
    U = X @ (beta[..., None] * v)
    Wm = X @ (beta[..., None] * e * k)
    P = (q @ k.transpose(-1, -2)) * rel
    qe = q * e
    kend = (k * torch.exp(gc[..., -1:] - gc).float()[..., None]).transpose(-1, -2)
    last = e[..., -1:, :]
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(N, hv, D, D, device=q.device)
    out = torch.empty_like(v)
    for i in range(nc):     # the recurrence itself: each chunk starts from the state the one before it left
        w = U[:, i] - Wm[:, i] @ S
        out[:, i] = qe[:, i] @ S + P[:, i] @ w
        S = S * last[:, i] + kend[:, i] @ w
    out = out.transpose(2, 3).flatten(1, 2)
    o = torch.empty_like(s["v"])
    o[at[live]] = out[live].to(torch.bfloat16)
    return {"o": o, "S": S}


def _gdn_decode(s):
    c = s["case"]
    rep = c["hv"] // c["hk"]
    q = _l2(s["q"].float()).repeat_interleave(rep, dim=1)
    k = _l2(s["k"].float()).repeat_interleave(rep, dim=1)
    v, at = s["v"].float(), s["slots"].long()
    a = torch.exp(_log_decay(s["z"], s["A"], c["gate"])).float()
    S = s["state"][at] * a[..., None, None]
    u = s["beta"][..., None] * (v - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"][at] = S
    return {"o": (q[..., None] * S).sum(-2).to(torch.bfloat16), "state": s["state"]}


def _turn(x, w, cos, sin, style, eps=1e-6):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w
    rot = 2 * cos.shape[-1]
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if style == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, s = cos[:, None], sin[:, None]
    p, r = a * c - b * s, b * c + a * s
    z = torch.cat([p, r], -1) if style == "half" else torch.stack([p, r], -1).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _rope(s):
    at = s["pos"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    return {"q": _turn(s["q"], s["qw"], cos, sin, s["case"]["style"]),
            "k": _turn(s["k"], s["kw"], cos, sin, s["case"]["style"])}


def _window_prefill(s):
    c, B, plan = s["case"], s["block"], s["plan"]
    W, sinks, hq, hkv, d = c["window"], c["sinks"], c["hq"], c["hkv"], c["d"]
    dev = s["q"].device
    q0, nq, p0, k0 = (x[:, None] for x in plan.unbind(1))
    i = torch.arange(B, device=dev)
    qi = (q0 + i).clamp(max=s["q"].shape[0] - 1)
    pq = p0 + i                                                      # positions of the queries
    pk = p0 - (W - 1) + torch.arange(B + W - 1, device=dev)          # positions of the block's keys
    ps = torch.arange(sinks, device=dev).expand(plan.shape[0], sinks)
    key = torch.cat([pk, ps], 1)
    kk, pp = key[:, None, :], pq[:, :, None]
    see = (kk >= 0) & (kk <= pp)
    n = pk.shape[1]
    see[:, :, :n] &= kk[:, :, :n] > pp - W
    see[:, :, n:] &= kk[:, :, n:] <= pp - W                          # the sinks that the window has left behind
    ki = (k0 + key.clamp(min=0)).clamp(max=s["k"].shape[0] - 1)
    g = hq // hkv
    q = s["q"].float()[qi].unflatten(2, (hkv, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)      # [nb, hkv, g B, d]
    k, v = (s[x].float()[ki].transpose(1, 2) for x in "kv")                                # [nb, hkv, L, d]
    x = ((q @ k.transpose(-1, -2)) * d ** -0.5).unflatten(2, (g, B))
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = torch.exp(x.sub_(m))
    l = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (g, B)) / l
    lse = (m + torch.log(l)).squeeze(-1)
    live = (i < nq)
    at = (q0 + i)[live]
    out = torch.empty_like(s["q"])
    out[at] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].to(torch.bfloat16)
    ls = torch.empty(s["q"].shape[0], hq, device=dev)
    ls[at] = lse.permute(0, 3, 1, 2).flatten(2, 3)[live]
    if not c["cache"]:
        return {"o": out, "lse": ls}
    src, seq, row = s["fill"]
    s["kc"][s["slots"].long()[seq], row] = s["k"][src]
    s["vc"][s["slots"].long()[seq], row] = s["v"][src]
    return {"o": out, "lse": ls, "kc": s["kc"], "vc": s["vc"]}


def _window_decode(s):
    c = s["case"]
    W, sinks, hq, hkv, d = c["window"], c["sinks"], c["hq"], c["hkv"], c["d"]
    pos, at = s["pos"].long(), s["slots"].long()
    row = torch.where(pos < sinks, pos, sinks + (pos - sinks) % W)
    s["kc"][at, row] = s["k"]
    s["vc"][at, row] = s["v"]
    r = torch.arange(W, device=pos.device)
    held = pos[:, None] - (pos[:, None] - sinks - r) % W             # the position that each ring row holds
    see = torch.cat([torch.arange(sinks, device=pos.device) <= pos[:, None], (held >= sinks) & (held > pos[:, None] - W)], 1)
    k, v = (s[x][at].float().transpose(1, 2) for x in ("kc", "vc"))
    q = s["q"].float().unflatten(1, (hkv, hq // hkv))
    x = ((q @ k.transpose(-1, -2)) * d ** -0.5).masked_fill(~see[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x @ v) / x.sum(-1, keepdim=True)
    return {"o": o.flatten(1, 2).to(torch.bfloat16), "kc": s["kc"], "vc": s["vc"]}


# ---------------------------------------------------------------------------
# what one pass has to read, write and compute
# ---------------------------------------------------------------------------

def _pairs(lens, hist, W, sinks):
    """Query-key pairs that the window and the sinks leave visible."""
    total = 0
    for ln, h in zip(lens, hist):
        for a, b in ((h, h + ln),):
            # position p sees min(p + 1, W) keys of the window and min(sinks, max(0, p - W + 1)) before it
            m = min(max(W, a), b)
            total += (m * (m + 1) - a * (a + 1)) // 2 + (b - m) * W
            if sinks:
                lo, hi = max(a, W - 1), max(b, W - 1)
                top = min(max(W - 1 + sinks, lo), hi)
                f = lambda p: (p - W + 1) * (p - W + 2) // 2        # noqa: E731
                total += (f(top - 1) - f(lo - 1) if top > lo else 0) + (hi - top) * sinks
    return total


def work(case):
    op = case["op"]
    if op in ("gdn_prefill", "gdn_decode"):
        lens = _ints(case["lens"]) if op == "gdn_prefill" else [1] * case["n"]
        T, hk, hv = sum(lens), case["hk"], case["hv"]
        states = (len(lens) * (1 + bool(case["s0"]))) if op == "gdn_prefill" else 2 * case["n"]
        return {"bytes": T * (2 * hk * D * 2 + 2 * hv * D * 2 + hv * 8) + hv * 4 + states * hv * D * D * 4,
                "flops": T * hv * 7 * D * D}
    if op == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        x = case["t"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 2 * x * e + case["t"] * (4 * case["rot"] + 4), "flops": 7 * x}
    hq, hkv, d, W, sinks = (case[x] for x in ("hq", "hkv", "d", "window", "sinks"))
    if op == "window_prefill":
        lens, hist = _ints(case["lens"]), _ints(case["hist"])
        klens = [a + b if a else 0 for a, b in zip(lens, hist)]
        seen = [min(k, min(sinks, k) + n + W - 1) if n else 0 for k, n in zip(klens, lens)]
        fill = sum(min(k, W + sinks) for k in klens) * hkv * d * 4 if case["cache"] else 0
        return {"bytes": sum(lens) * hq * (d * 4 + 4) + sum(seen) * hkv * d * 4 + fill,
                "flops": 4 * d * hq * _pairs(lens, hist, W, sinks)}
    n = case["n"]
    rows = int(n * (0.9 + 0.05) * (W + sinks))      # one in ten sequences has just begun
    return {"bytes": rows * hkv * d * 4 + n * (hq * d * 4 + 2 * hkv * d * 4), "flops": 4 * d * hq * rows}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return dict(gdn_prefill=_exact_gdn, gdn_decode=_exact_gdn, rope=_exact_rope, window_prefill=_exact_window,
                window_decode=_exact_window_step)[case["op"]](s)


def _exact_gdn(s):
    """The recurrence, token by token: S <- a S; S <- S + k (b (v - S^T k))^T; o = S^T q."""
    c = s["case"]
    prefill = c["op"] == "gdn_prefill"
    rep = c["hv"] // c["hk"]
    q, k, v = (s[x].double() for x in "qkv")
    q = (q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt())
    k = (k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt())
    z, A, beta = s["z"].double(), s["A"].double(), s["beta"].double()
    a = torch.exp(-5 * torch.sigmoid(A.exp() * z) if c["gate"] == "bounded"
                  else -A.exp() * torch.logaddexp(z, torch.zeros_like(z)))
    if prefill:
        cu = s["cu_host"].tolist()
        lens = [cu[i + 1] - cu[i] for i in range(len(cu) - 1)]
        S = s["S0"].double() if s["S0"] is not None else torch.zeros(len(lens), c["hv"], D, D, dtype=torch.float64, device=q.device)
        order = sorted(range(len(lens)), key=lambda n: -lens[n])     # the sequences still running come first
        starts = torch.tensor([cu[n] for n in order], device=q.device)
        S = S[torch.tensor(order, device=q.device)]
        steps, running = max(lens), [sum(x > t for x in lens) for t in range(max(lens))]
    else:
        S, starts = s["state"].double()[s["slots"].long()], torch.arange(c["n"], device=q.device)
        steps, running = 1, [c["n"]]
    o = torch.zeros(v.shape, dtype=torch.float64, device=q.device)
    hv, hk = c["hv"], c["hk"]
    for t in range(steps):
        n = running[t]
        i = starts[:n] + t
        qi, ki = (x[i].view(n, hk, 1, D).expand(n, hk, rep, D).reshape(n, hv, D, 1) for x in (q, k))
        R = S[:n]
        R *= a[i][..., None, None]
        u = beta[i][..., None] * (v[i] - (ki.transpose(-1, -2) @ R).squeeze(-2))
        torch.baddbmm(R.flatten(0, 1), ki.flatten(0, 1), u.view(n * hv, 1, D), out=R.flatten(0, 1))
        o[i] = (qi.transpose(-1, -2) @ R).squeeze(-2)
    if prefill:
        back = torch.empty(len(lens), dtype=torch.int64, device=q.device)
        back[torch.tensor(order, device=q.device)] = torch.arange(len(lens), device=q.device)
        return {"o": o, "S": S[back]}
    state = s["state"].double()
    state[s["slots"].long()] = S
    return {"o": o, "state": state}


def _exact_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    j = torch.arange(half, device=s["q"].device)
    first, second = (j, j + half) if c["style"] == "half" else (2 * j, 2 * j + 1)
    w = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]
    res = {}
    for name, weight in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        t = torch.complex(y[..., first], y[..., second]) * w
        y[..., first], y[..., second] = t.real, t.imag
        res[name] = y
    return res


def _exact_window(s):
    c = s["case"]
    W, sinks, hq, hkv, d = c["window"], c["sinks"], c["hq"], c["hkv"], c["d"]
    lens, hist = _ints(c["lens"]), _ints(c["hist"])
    if 4 * d * hq * _pairs(lens, hist, W, sinks) > 6e12:
        return None
    cu, cuk = s["cu_host"].tolist(), s["cuk_host"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    step = 1024
    for n, (ln, h) in enumerate(zip(lens, hist)):
        for a in range(0, ln, step):
            b = min(ln, a + step)
            p = torch.arange(h + a, h + b, device=o.device)
            lo = max(0, h + a - W + 1)
            j = torch.cat([torch.arange(min(sinks, lo), device=o.device), torch.arange(lo, h + b, device=o.device)])
            see = (j <= p[:, None]) & ((j > p[:, None] - W) | (j < sinks))
            K, V = (s[x][cuk[n]:cuk[n + 1]][j].double() for x in "kv")
            for x in range(hq):
                y = x // (hq // hkv)
                t = (s["q"][cu[n] + a:cu[n] + b, x].double() @ K[:, y].T) / math.sqrt(d)
                t = t.masked_fill(~see, -math.inf)
                r = torch.logsumexp(t, -1)
                lse[cu[n] + a:cu[n] + b, x] = r
                o[cu[n] + a:cu[n] + b, x] = torch.exp(t - r[:, None]) @ V[:, y]
    out = {"o": o, "lse": lse}
    if c["cache"]:
        for name, x in (("kc", "k"), ("vc", "v")):
            new = s[name].double()
            for n in range(len(lens)):
                for p in range(cuk[n + 1] - cuk[n]):            # in order: later tokens overwrite the ring
                    if p < sinks or p >= cuk[n + 1] - cuk[n] - W:
                        new[s["slots"][n].long(), p if p < sinks else sinks + (p - sinks) % W] = s[x][cuk[n] + p].double()
            out[name] = new
    return out


def _exact_window_step(s):
    c = s["case"]
    W, sinks, hq, hkv, d = c["window"], c["sinks"], c["hq"], c["hkv"], c["d"]
    kc, vc = s["kc"].double(), s["vc"].double()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=kc.device)
    pos, slots = s["pos"].tolist(), s["slots"].tolist()
    for n, (p, i) in enumerate(zip(pos, slots)):
        here = p if p < sinks else sinks + (p - sinks) % W
        kc[i, here], vc[i, here] = s["k"][n].double(), s["v"][n].double()
        seen = [x for x in range(min(sinks, p + 1))] + list(range(max(sinks, p - W + 1), p + 1))
        rows = torch.tensor([x if x < sinks else sinks + (x - sinks) % W for x in seen], device=kc.device)
        K, V = kc[i, rows].transpose(0, 1), vc[i, rows].transpose(0, 1)
        t = s["q"][n].double().view(hkv, hq // hkv, d) @ K.transpose(-1, -2) / math.sqrt(d)
        o[n] = (torch.softmax(t, -1) @ V).reshape(hq, d)
    return {"o": o, "kc": kc, "vc": vc}
