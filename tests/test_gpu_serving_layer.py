"""The example's decoder layer (examples/decoder_layer.py) with rotary positions,
adapters beside its qkv product and a shared prefix, against the same steps in 64 bits.

Tolerances, of a norm.  The 8-bit products as in test_gpu_decoder_layer.py: 2^-5.  The
adapters' input and result, the sum's rounding and the rotation's are half a step of bf16 each,
4 * 2^-8 = 2^-6.  Attention on what the layer itself had: probabilities and result, 2 * 2^-8."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
sys.path.insert(0, os.path.join(ROOT, "tests"))

import bit_weight_only_03_amd as L  # noqa: E402
import decoder_layer as ex  # noqa: E402
from test_gpu_decoder_layer import e4m3, norm, rel, values  # noqa: E402

DEV = "cuda"
HIDDEN, HQ, HKV, D, INNER, PAGE, ROT, N_ADAPT, R = 640, 8, 2, 64, 1040, 16, 32, 3, 24
QW, KW = HQ * D, HKV * D


def bf(t):
    return t.to(ex.BF16).double()


class Run:
    """A layer for B requests of T drafts and everything a call takes, at maxima that set() stays within."""

    def __init__(self, B, T, max_len, max_prefix, seed):
        self.B, self.T, self.M, self.max_len, self.max_prefix = B, T, B * T, max_len, max_prefix
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        bits = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
        o = (bits(HIDDEN, QW // 8), (randn(QW // 128, HIDDEN) * 1e-2).half().view(torch.int16), bits(QW // 128, HIDDEN // 8))
        self.w = ex.Weights(HIDDEN, HQ, HKV, D, INNER, (1 + 0.1 * randn(HIDDEN)).to(ex.BF16), randn(QW + 2 * KW, HIDDEN) * 0.05, o,
                            (1 + 0.1 * randn(HIDDEN)).to(ex.BF16), randn(2 * INNER, HIDDEN) * 0.05, randn(HIDDEN, INNER) * 0.05)
        ranks = torch.tensor([R, 9, 16], dtype=torch.int32, device=DEV)
        a, b = randn(N_ADAPT, 3, R, HIDDEN) * HIDDEN ** -0.5, randn(N_ADAPT, QW + 2 * KW, R) * 0.3
        for i, r in enumerate(ranks.tolist()):
            a[i, :, r:], b[i, :, r:] = 0, 0
        self.adapters = ex.Adapters(a.to(ex.BF16), b.to(ex.BF16), ranks, torch.tensor([1.0, 0.5, 2.0], device=DEV))
        self.freq = ex.frequencies(ROT, 1e4, 4.0, 256.0)
        per, shared = -(-(max_len + T) // PAGE), -(-max_prefix // PAGE)
        self.layer = ex.Layer(self.w, B, T, B * per + shared, PAGE, max_len, self.freq, self.adapters, max_prefix)
        self.layer.k.normal_(generator=g)
        self.layer.v.normal_(generator=g)
        order = torch.randperm(B * per + shared, generator=g, device=DEV).to(torch.int32)
        self.table, self.pages = order[:B * per].view(B, per).contiguous(), order[B * per:].contiguous()
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        self.lens, self.length, self.positions, self.ids = i32(B), i32(1), i32(self.M), i32(self.M)
        self.mask, self.slots = torch.zeros(B, T, dtype=torch.int64, device=DEV), torch.zeros(self.M, dtype=torch.int64, device=DEV)
        self.x = torch.zeros(self.M, HIDDEN, dtype=ex.BF16, device=DEV)

    def set(self, lens, prefix, ids):
        """New lengths, adapters (of the requests), residual stream and tree of drafts, in place."""
        T, g = self.T, self.g
        row = []
        for i in range(T):
            p = int(torch.randint(-1, i, (1,), generator=g, device=DEV)) if i else -1
            row.append((row[p] if p >= 0 else 0) | 1 << i)
        depth = torch.tensor([bin(r).count("1") - 1 for r in row], device=DEV)
        self.row = row
        self.mask.copy_(torch.tensor([r - (1 << 64) if r >> 63 else r for r in row], device=DEV).expand(self.B, T))
        self.lens.copy_(torch.tensor(lens))
        self.length.fill_(prefix)
        self.ids.copy_(torch.tensor(ids, device=DEV).repeat_interleave(T))
        self.positions.copy_((prefix + self.lens[:, None] + depth).view(-1))
        at = self.lens[:, None].long() + torch.arange(T, device=DEV)
        self.slots.copy_((self.table.gather(1, at // PAGE).long() * PAGE + at % PAGE).view(-1))
        self.x.copy_(2 * torch.randn(self.M, HIDDEN, generator=g, device=DEV))

    def call(self):
        return self.layer(self.x, self.table, self.lens, self.mask, self.slots, self.positions, self.ids, (self.pages, self.length))

    def rotate(self, x):
        """x [M][heads][D] in 64 bits, halves."""
        angle = self.positions.double()[:, None] * self.freq.double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        u, v = x[..., :ROT // 2], x[..., ROT // 2:ROT]
        return torch.cat([u * c - v * s, v * c + u * s, x[..., ROT:]], 2)

    def check(self, h, y):
        w, M, T, layer, ad = self.w, self.M, self.T, self.layer, self.adapters
        n = norm(self.x.double(), w.norm1)
        qkv = bf(e4m3(n) @ values(w.qkv).t())
        for i in range(N_ADAPT):
            rows = (self.ids == i).nonzero()[:, 0]
            for p, (c0, c1) in enumerate(((0, QW), (QW, QW + KW), (QW + KW, QW + 2 * KW))):
                qkv[rows, c0:c1] += float(ad.scales[i]) * (n[rows] @ ad.a[i, p].double().t()) @ ad.b[i, c0:c1].double().t()
        tol = 2.0 ** -5 + 2.0 ** -6
        kc, vc = (c.view(-1, HKV, D) for c in (layer.k, layer.v))
        assert rel(layer.qkv[:, QW:], qkv[:, QW:]) < tol
        assert rel(layer.qkv[:, :QW].view(M, HQ, D), self.rotate(qkv[:, :QW].view(M, HQ, D))) < tol
        # The keys in the cache are the layer's own, rotated and rounded once (half a step, and sines' and products' 2^-20).
        mine = self.rotate(layer.qkv[:, QW:QW + KW].double().view(M, HKV, D))
        big = layer.qkv[:, QW:QW + KW].double().abs().amax()
        assert torch.all((kc[self.slots].double() - mine).abs() <= 2.0 ** -8 * mine.abs() + 2.0 ** -20 * big)
        assert torch.equal(vc[self.slots].reshape(M, KW), layer.qkv[:, QW + KW:])
        att = torch.zeros(M, HQ, D, dtype=torch.float64, device=DEV)
        P, q = int(self.length), layer.qkv[:, :QW].double().view(M, HQ, D)
        for b in range(self.B):
            total = int(self.lens[b]) + T
            at, sh = torch.arange(total, device=DEV), torch.arange(P, device=DEV)
            rows = torch.cat([self.pages[sh // PAGE].long() * PAGE + sh % PAGE, self.table[b, at // PAGE].long() * PAGE + at % PAGE])
            kk, vv = kc[rows].double(), vc[rows].double()
            for i in range(T):
                see = torch.ones(P + total, dtype=torch.bool, device=DEV)
                see[P + total - T:] = torch.tensor([bool(self.row[i] >> j & 1) for j in range(T)], device=DEV)
                for head in range(HQ):
                    a = kk[see, head * HKV // HQ] @ q[b * T + i, head] / math.sqrt(D)
                    att[b * T + i, head] = torch.softmax(a, 0) @ vv[see, head * HKV // HQ]
        assert rel(layer.att, att.view(M, QW)) < 2.0 ** -7
        wo = torch.empty(QW, HIDDEN, device=DEV)
        L.w4a16_dequant(*w.o, wo, HIDDEN, QW, 128)
        assert rel(layer.o, layer.att.double() @ wo.double()) < 2.0 ** -7
        h64 = self.x.double() + layer.o.double()
        assert rel(h, h64) < 2.0 ** -8
        gu = bf(e4m3(norm(h64, w.norm2)) @ values(w.gate_up).t())
        gate, up = gu.split(INNER, 1)
        assert rel(y, e4m3(gate * torch.sigmoid(gate) * up) @ values(w.down).t()) < 2.0 ** -4


@pytest.mark.parametrize("B,T,lens,prefix,ids", [
    (1, 1, [0], 0, [1]),                                     # the first token of a request that shares nothing
    (3, 1, [40, 0, 129], 500, [0, -1, 2]),
    (4, 6, [75, 0, 16, 3], 33, [2, 2, 0, 1]),
    (20, 4, [i * 7 % 90 for i in range(20)], 200, [i % 4 - 1 for i in range(20)]),
])
def test_layer_matches_its_steps(B, T, lens, prefix, ids):
    run = Run(B, T, max(lens), prefix, B)
    run.set(lens, prefix, ids)
    h, y = run.call()
    torch.cuda.synchronize()
    run.check(h, y)


def test_a_captured_layer_follows_its_inputs():
    # Lengths, prefix, adapters, tree and residual stream change between the replays.
    run = Run(5, 4, 100, 300, 9)
    stream = torch.cuda.Stream()
    run.set([0] * 5, 0, [0] * 5)
    run.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run.call()
    for lens, prefix, ids in (([100, 3, 64, 0, 15], 300, [0, 1, 2, -1, 0]), ([1, 2, 3, 4, 5], 17, [-1] * 5), ([99] * 5, 0, [2, 2, 2, 2, 1]), ([0] * 5, 299, [1, 0, 1, 0, 7])):
        run.set(lens, prefix, ids)
        graph.replay()
        torch.cuda.synchronize()
        run.check(run.layer.h, run.layer.y)
        got = [t.clone() for t in (run.layer.qkv, run.layer.att, run.layer.h, run.layer.y)]
        run.call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (run.layer.qkv, run.layer.att, run.layer.h, run.layer.y)))
