"""The example's decoder layer (examples/decoder_layer.py) against the same
steps in 64 bits, with the same roundings (8-bit operands, bf16 results).

An 8-bit code that falls on the other side of its rounding moves by 2^-3 at
most; that happens where a value lies within the error of its operands (bf16's
2^-8 relative) of the middle of two codes, so for less than 2^-8 / 2^-4 of them, each
by at most 2^-3: sqrt(2^-4) * 2^-3 = 2^-5 of a norm, and two such steps in a row
stay below 2^-4.  A wrong stride, slot or scale is an error of the norm's own size."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import bit_weight_only_03_amd as L  # noqa: E402
import decoder_layer as ex  # noqa: E402


def e4m3(x):
    K = x.shape[1]
    p = torch.nn.functional.pad(x, (0, -K % 128)).view(x.shape[0], -1, 128)
    s = p.abs().amax(2).clamp_min(2.0 ** -60) / 448
    q = (p / s[:, :, None]).float().to(ex.FP8).double()
    return (q * s[:, :, None]).reshape(x.shape[0], -1)[:, :K]


def values(weight):
    q, s = weight
    return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def norm(h, w):
    return h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("B,T,lens", [(1, 1, [30]), (2, 6, [75, 0]), (3, 20, [500, 64, 129])])
def test_layer_matches_its_steps(B, T, lens):
    hidden, q_heads, kv_heads, D, inner, page = 640, 8, 2, 64, 1040, 16
    g = torch.Generator(device="cuda").manual_seed(B)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bits = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)  # noqa: E731
    K = q_heads * D
    o = (bits(hidden, K // 8), (randn(K // 128, hidden) * 1e-2).half().view(torch.int16), bits(K // 128, hidden // 8))
    w = ex.Weights(hidden, q_heads, kv_heads, D, inner, (1 + 0.1 * randn(hidden)).to(ex.BF16), randn((q_heads + 2 * kv_heads) * D, hidden) * 0.05,
                   o, (1 + 0.1 * randn(hidden)).to(ex.BF16), randn(2 * inner, hidden) * 0.05, randn(hidden, inner) * 0.05)
    M, per = B * T, -(-(max(lens) + T) // page)
    layer = ex.Layer(w, B, T, B * per, page, max(lens))
    layer.k.normal_(generator=g)
    layer.v.normal_(generator=g)
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    parent = [int(torch.randint(-1, max(i, 1), (1,), generator=g, device="cuda")) if i else -1 for i in range(T)]
    row = []
    for i in range(T):
        row.append((row[parent[i]] if parent[i] >= 0 else 0) | 1 << i)
    mask = torch.tensor([row] * B, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    p = n[:, None].long() + torch.arange(T, device="cuda")
    slots = (table.gather(1, p // page).long() * page + p % page).view(-1)
    x = (2 * randn(M, hidden)).to(ex.BF16)
    h, y = layer(x, table, n, mask, slots)
    torch.cuda.synchronize()

    bf = lambda t: t.to(ex.BF16).double()  # noqa: E731
    qkv = bf(e4m3(norm(x.double(), w.norm1)) @ values(w.qkv).t())
    assert rel(layer.qkv, qkv) < 2.0 ** -5
    qkv = layer.qkv.double()                                           # the attention on what the layer itself had
    qw, kw = q_heads * D, kv_heads * D
    att = torch.zeros(M, q_heads, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        total = lens[b] + T
        at = torch.arange(total, device="cuda")
        rows = table[b, at // page].long() * page + at % page
        kk, vv = (c.view(-1, kv_heads, D)[rows].double().clone() for c in (layer.k, layer.v))
        assert torch.equal(kk[lens[b]:].reshape(T, -1), qkv[b * T:(b + 1) * T, qw:qw + kw])
        for i in range(T):
            see = torch.ones(total, dtype=torch.bool, device="cuda")
            see[lens[b]:] = torch.tensor([bool(row[i] >> j & 1) for j in range(T)], device="cuda")
            for hh in range(q_heads):
                a = kk[see, hh // (q_heads // kv_heads)] @ qkv[b * T + i, hh * D:(hh + 1) * D] * D ** -0.5
                att[b * T + i, hh] = torch.softmax(a, 0) @ vv[see, hh // (q_heads // kv_heads)]
    assert rel(layer.att, att.view(M, qw)) < 2.0 ** -7
    wo = torch.empty(K, hidden, device="cuda")
    L.w4a16_dequant(*w.o, wo, hidden, K, 128)
    assert rel(layer.o, layer.att.double() @ wo.double()) < 2.0 ** -7
    h64 = x.double() + layer.o.double()
    assert rel(h, h64) < 2.0 ** -8
    gu = bf(e4m3(norm(h64, w.norm2)) @ values(w.gate_up).t())
    assert rel(layer.gu, gu) < 2.0 ** -5
    gate, up = layer.gu.double().split(inner, 1)
    want = e4m3(gate * torch.sigmoid(gate) * up) @ values(w.down).t()
    assert rel(y, want) < 2.0 ** -5
    # The whole MLP from the 64-bit start.
    gate, up = gu.split(inner, 1)
    assert rel(y, e4m3(gate * torch.sigmoid(gate) * up) @ values(w.down).t()) < 2.0 ** -4


@pytest.mark.parametrize("B,T,lens", [(5, 16, [300, 12, 0, 77, 41]), (2, 40, [130, 5])])
def test_layer_with_more_rows_than_the_4_bit_product_takes_at_once(B, T, lens):
    test_layer_matches_its_steps(B, T, lens)
