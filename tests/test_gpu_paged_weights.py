"""How many bits the one-token step keeps of its softmax weights.  Keys come in pairs whose scores are nearly alike and whose values
are each other's negative, so that outputs are small beside the sum of |weight value| and what the weights' rounding leaves stands above
the outputs' own rounding.

Bounds, relative to the softmax-weighted sum of |v| (``size``):
  weights: 2^-16 over bf16 pages (16 bits or more), 2^-11 over 8-bit ones (11 bits: half a step);
  scores: 128 products in 8 steps of float32 sums, each off by 2^-23 of partial sums that stay below scale sum |q k| log2 e, here below
  8 (asserted): 2^-17 of an exponent of two, 2^-17.5 of a weight, and as much of their sum: 2^-16.5;
  exponentials (2 units of 2^-23) and the sums over at most 64 keys (8 steps of 2^-23): below 2^-19;
and half a step of bf16, 2^-8, of the output itself."""
import math

import pytest
import torch

import paged_testutil
from paged_testutil import Cache, attention

BF = torch.bfloat16
WEIGHT = {"bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}
SUMS = 2.0 ** -16.5 + 2.0 ** -19
SHAPES = [([8, 16, 33, 64, 20, 2], 8, 2, 128, 16), ([16, 17, 48], 16, 1, 64, 32), ([31, 32, 12, 64], 3, 3, 128, 64)]


def _pairs(g, lens, hkv, d):
    """Keys and values of sequences: key 2i + 1 is key 2i but for one channel, value 2i + 1 the negative of value 2i."""
    K, V = [], []
    for n in lens:
        k = (0.4 * torch.randn(n, hkv, d, generator=g)).to(BF).float()
        v = torch.randn(n, hkv, d, generator=g).to(BF).float()
        m = n // 2 * 2
        k[1:m:2] = k[0:m:2]
        k[1:m:2, :, 0] = (k[1:m:2, :, 0] + 0.125).to(BF).float()
        v[1:m:2] = -v[0:m:2]
        if n % 2:
            v[-1] = 0
        K.append(k)
        V.append(v)
    return K, V


def _case(shape, kind):
    lens, hq, hkv, d, page = shape
    g = torch.Generator().manual_seed(51)
    K, V = _pairs(g, lens, hkv, d)
    c = Cache(K, V, page, kind, "cpu")
    q = torch.randn(len(lens), hq, d, generator=g).to(BF)
    for n, k in enumerate(c.host["k"]):
        partial = torch.einsum("hgd,lhd->hgl", q[n].double().abs().unflatten(0, (hkv, -1)), k.abs())
        assert partial.max() * d ** -0.5 * math.log2(math.e) < 8
    return c, q, attention(q, [1] * len(lens), c.host["k"], c.host["v"])


def _worst(o, ref, size, kind):
    """The largest error in units of its bound."""
    bound = (WEIGHT[kind] + SUMS) * size + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + 1e-30
    return ((o.double().cpu() - ref).abs() / bound).max().item()


def _model(c, q, bits):
    """The step with weights of ``bits`` bits, everything else in 64, outputs rounded to bf16."""
    out = []
    for n, (k, v) in enumerate(zip(c.host["k"], c.host["v"])):
        s = torch.einsum("hgd,lhd->hgl", q[n].double().unflatten(0, (k.shape[1], -1)), k) * q.shape[2] ** -0.5
        w = torch.exp(s - s.amax(-1, keepdim=True))
        m, e = torch.frexp(w)
        r = torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)
        out.append((torch.einsum("hgl,lhd->hgd", r, v) / w.sum(-1)[..., None]).flatten(0, 1))
    return torch.stack(out).to(BF)


@pytest.mark.parametrize("kind,enough,short", [("bf16", 16, 11), ("e4m3", 11, 8)])
def test_the_bound_tells_the_bits(kind, enough, short):
    """What the header promises meets the bound, weights of fewer bits do not: in every shape."""
    for shape in SHAPES:
        c, q, (ro, _, size) = _case(shape, kind)
        assert _worst(_model(c, q, enough), ro, size, kind) <= 1
        assert _worst(_model(c, q, short), ro, size, kind) > 1.5, shape


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [0, 40])                 # units whole, and cut where the tables have room for many tiles
@pytest.mark.parametrize("shape", SHAPES)
def test_step(kda_lib, cuda_dev, kind, wide, shape):
    import serving_kda_chunked_gated_gb300.kda as kda
    c, q, (ro, _, size) = _case(shape, kind)
    tables = torch.nn.functional.pad(c.tables, (0, wide), value=-1).to(cuda_dev)
    dev = lambda x: x.to(cuda_dev)                                                      # noqa: E731
    pages = [dev(c.k.view(torch.uint8)).view(c.k.dtype), dev(c.v.view(torch.uint8)).view(c.v.dtype)] if kind == "e4m3" else [dev(c.k), dev(c.v)]
    o = kda.paged_decode(dev(q), *pages, tables, dev(c.lens), **{n: dev(x) for n, x in c.scales.items()})
    assert torch.isfinite(o).all()
    worst = _worst(o, ro, size, kind)
    assert worst <= 1, f"{worst:.3f} of the bound"
