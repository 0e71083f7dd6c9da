"""Plain 64-bit forms of the hybrid token mixers, and small input makers."""
import math

import torch


def silu_bf16(g, *shape):
    x = torch.randn(*shape, generator=g)
    return (x * torch.sigmoid(x)).to(torch.bfloat16)


def gdn_inputs(lens, Hk, Hv, seed=0, dtype=torch.bfloat16, z_mean=-3.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    d = dict(q=silu_bf16(g, T, Hk, 128), k=silu_bf16(g, T, Hk, 128), v=silu_bf16(g, T, Hv, 128),
             z=1.5 * torch.randn(T, Hv, generator=g) + z_mean, beta=torch.sigmoid(torch.randn(T, Hv, generator=g)),
             A=torch.log(1 + 7 * torch.rand(Hv, generator=g)), S0=0.1 * torch.randn(len(lens), Hv, 128, 128, generator=g))
    for n in "qkv":
        d[n] = d[n].to(dtype)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    return d, cu


def log_decay(z, A, gate, g_min=-5.0):
    z, e = z.double(), A.double().exp()
    return g_min * torch.sigmoid(e * z) if gate == "bounded" else -e * torch.logaddexp(z, torch.zeros_like(z))


def gdn_reference(q, k, v, z, beta, A, cu, S0=None, gate="softplus", scale=1.0, l2=True, g_min=-5.0):
    """The recurrence token by token: (o [T, Hv, 128], S_T [N, Hv, 128, 128])."""
    T, Hv = v.shape[0], v.shape[1]
    rep = Hv // q.shape[1]
    q, k, v, beta = q.double(), k.double(), v.double(), beta.double()
    if l2:
        q = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    a = log_decay(z, A, gate, g_min).exp()
    o = torch.zeros(T, Hv, 128, dtype=torch.float64)
    out = []
    cu = [int(x) for x in cu]
    for n in range(len(cu) - 1):
        S = S0[n].double().clone() if S0 is not None else torch.zeros(Hv, 128, 128, dtype=torch.float64)
        for t in range(cu[n], cu[n + 1]):
            S = S * a[t][:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            o[t] = scale * torch.einsum("hij,hi->hj", S, q[t])
        out.append(S)
    return o, torch.stack(out) if out else torch.zeros(0, Hv, 128, 128, dtype=torch.float64)


def rope_reference(x, w, cos, sin, pos, interleaved, eps=1e-6):
    """(y, |n_a| + |n_b|): the normalised and rotated rows, and the size that their rounding goes by."""
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    half = cos.shape[1]
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    c, s = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]
    size = y.abs()
    ya, yb = y[..., a], y[..., b]
    size[..., a] = size[..., b] = ya.abs() + yb.abs()
    y = y.clone()
    y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y, size


def visible(p, window, sinks):
    """Positions that the query at position p sees."""
    return list(range(min(sinks, max(0, p - window + 1)))) + list(range(max(0, p - window + 1), p + 1))


def window_reference(q, k, v, cu_q, cu_k, window, sinks, scale=None):
    """(o, lse, size) in 64 bits; size = the softmax-weighted sum of |v|."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, size = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.zeros(T, Hq, dtype=torch.float64)
    q, k, v = q.double(), k.double(), v.double()
    cu_q, cu_k = [int(x) for x in cu_q], [int(x) for x in cu_k]
    for n in range(len(cu_q) - 1):
        lk, lq = cu_k[n + 1] - cu_k[n], cu_q[n + 1] - cu_q[n]
        if lq == 0:
            continue
        p = torch.arange(lk - lq, lk)[:, None]
        j = torch.arange(lk)
        see = (j <= p) & ((j > p - window) | (j < sinks))
        K, V = (x[cu_k[n]:cu_k[n + 1]].repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        s = torch.einsum("qhd,khd->hqk", q[cu_q[n]:cu_q[n + 1]], K) * scale
        s = s.masked_fill(~see, -math.inf)
        r = torch.logsumexp(s, -1, keepdim=True)
        w = (s - r).exp()
        V = torch.where(see.any(0)[:, None, None], V, torch.zeros_like(V))    # rows that nothing sees
        o[cu_q[n]:cu_q[n + 1]] = torch.einsum("hqk,khd->qhd", w, V)
        size[cu_q[n]:cu_q[n + 1]] = torch.einsum("hqk,khd->qhd", w, V.abs())
        lse[cu_q[n]:cu_q[n + 1]] = r.squeeze(-1).T
    return o, lse, size


def check_window(got, ref, size, what=""):
    """Each weight is rounded to bf16 (half a step, 2^-8 of it) and so is the output;
    a quarter step more covers the scores' and the sums' float32 roundings."""
    bound = 2.0 ** -8 * 1.25 * size + 2.0 ** -8 * ref.abs() + 1e-30
    off = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got.float()).all(), what
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    n = b.norm().item()
    return (a - b).norm().item() / n if n else (a - b).norm().item()
