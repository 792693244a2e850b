"""GPU tests of the attention behind a shared prefix (include/prefix_attn.h)
against its definition in 64 bits on the CPU.

Tolerances.  u = 2^-24, ut the type's half step.  A score is an fp32 sum of D
products (error at most (D + 4) u times the sum of magnitudes, scale included); with
the exponential's argument rounded twice and 2^x good to a few u, a probability is
off by at most e = (D + 4) u S + 4 u (A + 4) of itself, S the largest sum of magnitudes
of a score and A the largest |score|.  Each enters the product with v rounded once more
(ut), sums over n keys are fp32 ((n + 64) u), and the quotient is rounded to the type.
All of it relative to the mean |v| under the probabilities."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
UT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


class Case:
    """What no position maps to holds NaN: it must never be seen."""

    def __init__(self, B, T, Hq, Hkv, D, page, dtype, P, lens, seed=0, heads_first=False, q_pad=0, mask=None, spare=2, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.Hq, self.Hkv, self.D, self.page, self.dtype, self.P = B, T, Hq, Hkv, D, page, dtype, P
        self.lens, self.heads_first, ty = torch.tensor(lens, dtype=torch.int32), heads_first, TYPES[dtype]
        self.max_len, self.common = max(lens), -(-P // page)
        per = -(-(self.max_len + T) // page)
        self.pages = self.common + B * per + spare
        shape = (self.pages, Hkv, page, D) if heads_first else (self.pages, page, Hkv, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=ty) for _ in range(2))
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.ptable, self.table = order[:self.common].clone(), order[self.common:self.common + B * per].view(B, per).clone()
        self.prefix = [torch.randn(P, Hkv, D, generator=g).to(ty) for _ in range(2)]
        self.dense = [[torch.randn(n + T, Hkv, D, generator=g).to(ty) for _ in range(2)] for n in lens]
        self.q = torch.randn(B * T, Hq * D + q_pad, generator=g).to(ty)
        self.scale = D ** -0.5 if scale is None else scale
        if mask is None:
            mask = np.zeros((B, T), dtype=np.uint64)
            for b in range(B):
                for i in range(T):
                    parent = int(torch.randint(-1, max(i, 1), (1,), generator=g)) if i else -1
                    mask[b, i] = (mask[b, parent] if parent >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
        self.mask = np.asarray(mask, dtype=np.uint64)
        self.store()

    def store(self):
        for table, (kd, vd) in [(self.ptable, self.prefix)] + [(self.table[b], self.dense[b]) for b in range(self.B)]:
            for c, d in ((self.k, kd), (self.v, vd)):
                for i in range(-(-d.shape[0] // self.page)):
                    part, p = d[i * self.page:(i + 1) * self.page], int(table[i])
                    if self.heads_first:
                        c[p, :, :part.shape[0]] = part.transpose(0, 1)
                    else:
                        c[p, :part.shape[0]] = part

    def to_gpu(self):
        self.g = dict(q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV), ptable=self.ptable.to(DEV), table=self.table.to(DEV), lens=self.lens.to(DEV),
                      plen=torch.tensor([self.P], dtype=torch.int32, device=DEV), mask=torch.from_numpy(self.mask.view(np.int64).copy()).to(DEV))
        return self

    def strides(self):
        s = self.k.stride()
        return (s[0], s[2], s[1]) if self.heads_first else (s[0], s[1], s[2])

    def run(self, max_len=None, max_prefix=None, work=None, lse=True, stream=None):
        if not hasattr(self, "g"):
            self.to_gpu()
        g, B, T, Hq, Hkv, D = self.g, self.B, self.T, self.Hq, self.Hkv, self.D
        max_len, max_prefix = self.max_len if max_len is None else max_len, self.P if max_prefix is None else max_prefix
        out = torch.full((B * T, Hq, D), float("nan"), dtype=TYPES[self.dtype], device=DEV)
        lse = torch.full((B * T, Hq), float("nan"), device=DEV) if lse else None
        need = L.prefix_attn_workspace_bytes(B, T, Hq, Hkv, D, max_prefix, max_len)
        if work is None:
            work = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)        # NaN
        ps, ts, hs = self.strides()
        L.prefix_attn(g["q"], self.q.stride(0), g["k"], g["v"], self.dtype, self.pages, self.page, ps, ts, hs, g["ptable"] if max_prefix else None,
                      g["plen"], max_prefix, g["table"], self.table.shape[1], g["lens"], max_len, g["mask"], self.scale, out, lse, B, T, Hq, Hkv, D,
                      work, work.numel(), stream)
        return out, lse

    def reference(self, requests=None):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits, of some requests."""
        B, T, Hq, D, G = self.B, self.T, self.Hq, self.D, self.Hq // self.Hkv
        requests = range(B) if requests is None else requests
        n = len(requests)
        out, tol = torch.zeros(n, T, Hq, D, dtype=torch.float64), torch.zeros(n, T, Hq, D, dtype=torch.float64)
        lse, ltol = torch.full((n, T, Hq), -math.inf, dtype=torch.float64), torch.zeros(n, T, Hq, dtype=torch.float64)
        for x, b in enumerate(requests):
            here = int(self.lens[b])
            k, v = (torch.cat([self.prefix[c][:self.P], self.dense[b][c]]).double() for c in range(2))
            for i in range(T):
                see = torch.ones(self.P + here + T, dtype=torch.bool)
                see[self.P + here:] = torch.tensor([bool(int(self.mask[b, i]) >> j & 1) for j in range(T)])
                at = see.nonzero()[:, 0]
                if not len(at):
                    continue
                for h in range(Hq):
                    q = self.q[b * T + i, h * D:(h + 1) * D].double()
                    kh, vh = k[at, h // G], v[at, h // G]
                    a = kh @ q * self.scale
                    mag = kh.abs() @ q.abs() * abs(self.scale)
                    p = torch.softmax(a, 0)
                    lse[x, i, h], o = torch.logsumexp(a, 0), p @ vh
                    e = (D + 4) * U * mag.max() + 4 * U * (a.abs().max() + 4) + (len(at) + 64) * U
                    out[x, i, h] = o
                    tol[x, i, h] = (UT[self.dtype] + 2 * e) * (p @ vh.abs()) + UT[self.dtype] * o.abs() + 2.0 ** -25
                    ltol[x, i, h] = e + 2 * U * lse[x, i, h].abs()
        return out, lse, tol, ltol

    def check(self, got, lse=None, requests=None):
        requests = list(range(self.B)) if requests is None else requests
        out, want_lse, tol, ltol = self.reference(requests)
        got = got.view(self.B, self.T, self.Hq, self.D)[requests].cpu().double()
        err = (got - out).abs()
        assert torch.all(err <= tol), (L.w4a16_last_variant(), float((err / tol).max()), (~(err <= tol)).nonzero()[:4].tolist())
        if lse is not None:
            lse = lse.view(self.B, self.T, self.Hq)[requests].cpu().double()
            none = torch.isinf(want_lse)
            assert torch.equal(lse[none], want_lse[none])
            assert torch.all((lse - want_lse)[~none].abs() <= ltol[~none])


CASES = [
    # B, T, Hq, Hkv, D, page, dtype, P, lens, heads_first, q_pad
    (1, 1, 1, 1, 64, 16, "bf16", 0, [0], False, 0),                 # one draft, nothing else
    (1, 1, 5, 1, 128, 16, "f16", 1, [0], False, 0),
    (2, 1, 8, 8, 128, 32, "f16", 33, [31, 33], False, 8),
    (3, 1, 40, 8, 128, 64, "bf16", 700, [70, 0, 64], False, 2048),
    (2, 1, 16, 2, 256, 16, "bf16", 515, [5, 130], True, 0),
    (2, 3, 10, 2, 64, 16, "f16", 64, [37, 5], False, 0),
    (4, 16, 10, 2, 128, 32, "bf16", 301, [300, 17, 0, 129], False, 0),   # 80 rows of a request
    (9, 8, 20, 4, 128, 64, "bf16", 2048, [1000, 3, 0, 77, 78, 79, 80, 0, 1], False, 0),
    (5, 13, 4, 2, 256, 128, "f16", 401, [41, 200, 0, 3, 127], False, 0),
    (2, 64, 2, 2, 64, 16, "f16", 100, [100, 0], False, 0),
    (3, 64, 8, 1, 128, 32, "bf16", 65, [65, 2, 31], False, 0),       # 512 rows of a request
    (1, 40, 6, 1, 256, 64, "bf16", 90, [90], True, 0),
    (33, 1, 3, 3, 64, 256, "bf16", 257, list(range(33)), False, 0),
    (70, 2, 4, 1, 128, 16, "f16", 1500, [i * 3 % 50 for i in range(70)], False, 0),   # 560 rows of the prefix
    (4, 1, 5, 1, 64, 32, "bf16", 6000, [10, 0, 600, 33], False, 0),
    (6, 2, 8, 2, 256, 64, "bf16", 3000, [30, 700, 1, 0, 2, 64], False, 0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,dtype,P,lens,heads_first,q_pad", CASES)
def test_matches_definition(B, T, Hq, Hkv, D, page, dtype, P, lens, heads_first, q_pad):
    c = Case(B, T, Hq, Hkv, D, page, dtype, P, lens, seed=T + Hq + D, heads_first=heads_first, q_pad=q_pad)
    out, lse = c.run()
    c.check(out, lse)
    again, _ = c.run(lse=False)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,T", [(1, 1), (5, 4)])
def test_every_form(dtype, D, G, T):
    # The bounds on the lengths choose the form: what it is for longer ones has to be right for these too.
    seen = set()
    for B in (2, 40):
        c = Case(B, T, 2 * G, 2, D, 16, dtype, 210, [(100, 0, 31, 32, 33, 64, 96)[i % 7] for i in range(B)], seed=D + G)
        c.ptable = torch.cat([c.ptable, torch.full((60000 // 16,), 10 ** 9, dtype=torch.int32)])     # clamped, never looked at
        wide = torch.full((B, 8192 // 16), -5, dtype=torch.int32)
        wide[:, :c.table.shape[1]] = c.table
        c.table = wide
        some = [0, 1] if B == 2 else [0, 1, 2, 3, 38, 39]
        want = c.reference(some)
        c.reference = lambda requests: want
        for max_prefix in (210, 700, 5000, 50000):
            for max_len in (100, 2000, 8000):
                out, lse = c.run(max_len=max_len, max_prefix=max_prefix)
                c.check(out, lse, some)
                seen.add(tuple(int(f.split("=")[1]) for f in L.w4a16_last_variant().split()[2:4]))
    assert any(sp == 0 for sp, so in seen) and any(sp > 1 for sp, so in seen), seen
    assert any(so > 1 for sp, so in seen) and any(so == 1 for sp, so in seen), seen


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(6, 2, 2, 128), (20, 2, 1, 64), (30, 4, 1, 128), (40, 1, 1, 256)])
@pytest.mark.parametrize("P,max_prefix", [(0, 0), (0, 3000), (50, 50), (50, 3000)])
def test_rows_that_see_nothing_and_values_that_are_not_seen(dtype, T, Hq, Hkv, D, P, max_prefix):
    # Request 0 has no context: its rows see the prefix and at most themselves, every
    # third nothing else.  Drafts that no row, or only their own row, sees hold NaN and infinities.
    B, lens = 2, [0, 45]
    mask = np.zeros((B, T), dtype=np.uint64)
    for i in range(T):
        if i % 3:
            mask[:, i] = np.uint64(1) << np.uint64(i)

    def case():
        c = Case(B, T, Hq, Hkv, D, 16, dtype, P, lens, seed=T, mask=mask)
        c.ptable = torch.cat([c.ptable, torch.zeros(200, dtype=torch.int32)])
        return c
    c = case()
    c.dense[0][0][0] = float("nan")                      # drafts 0, 3, .. are seen by nobody
    c.dense[0][1][3] = float("inf")
    c.dense[1][0][45] = float("inf")
    c.dense[1][1][48] = float("nan")
    c.store()
    out, lse = c.run(max_prefix=max_prefix)
    case().check(out, lse)                               # as if they were ordinary numbers
    if P == 0:
        assert torch.all(out.view(B, T, Hq, D)[0, ::3] == 0) and torch.all(torch.isneginf(lse.view(B, T, Hq)[0, ::3]))
    # A NaN and an infinity that only their own row sees change that row alone.
    c.dense[1][1][45 + 4, :, 7] = float("nan")
    c.dense[1][1][45 + 5, :, 9] = float("-inf")
    c.store()
    out2, lse2 = c.to_gpu().run(max_prefix=max_prefix)
    o, o2 = out.view(B, T, Hq, D).cpu().float(), out2.view(B, T, Hq, D).cpu().float()
    assert torch.all(torch.isnan(o2[1, 4, :, 7])) and torch.all(torch.isneginf(o2[1, 5, :, 9]))
    o2[1, 4, :, 7], o2[1, 5, :, 9] = o[1, 4, :, 7], o[1, 5, :, 9]
    assert torch.equal(o, o2)
    assert torch.equal(lse.cpu(), lse2.cpu())


@pytest.mark.parametrize("max_prefix", [70, 4000])
def test_nan_in_the_prefix_reaches_every_row(max_prefix):
    c = Case(3, 2, 2, 1, 64, 16, "bf16", 70, [5, 0, 40])
    c.ptable = torch.cat([c.ptable, torch.zeros(250, dtype=torch.int32)])
    c.prefix[1][10, 0, 5] = float("nan")
    c.store()
    o = c.run(max_prefix=max_prefix)[0].cpu().float()
    assert torch.all(torch.isnan(o[:, :, 5])) and torch.all(torch.isfinite(o[:, :, :5])) and torch.all(torch.isfinite(o[:, :, 6:]))
    c = Case(3, 2, 2, 1, 64, 16, "bf16", 70, [5, 0, 40])
    c.ptable = torch.cat([c.ptable, torch.zeros(250, dtype=torch.int32)])
    c.prefix[0][69] = float("nan")                       # the last key, in a tile that ends inside
    c.store()
    assert torch.all(torch.isnan(c.run(max_prefix=max_prefix)[0]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_prefix", [130, 5000])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_scales_and_scores_that_rise(dtype, max_prefix, scale):
    # Keys that grow with their position raise the running maximum in every tile; a large
    # scale leaves one key, the smallest steps stay below the slack of the maximum.
    c = Case(5, 3, 4, 2, 128, 32, dtype, 130, [40, 0, 64, 31, 33], scale=scale, seed=9)
    c.ptable = torch.cat([c.ptable, torch.zeros(200, dtype=torch.int32)])
    for kd in [c.prefix[0]] + [d[0] for d in c.dense]:
        kd *= torch.linspace(0.1, 1.0, kd.shape[0])[:, None, None].to(kd.dtype)
    c.store()
    out, lse = c.run(max_prefix=max_prefix)
    c.check(out, lse)


def test_lengths_past_their_bounds_are_cut():
    c = Case(3, 2, 4, 2, 64, 16, "bf16", 100, [50, 20, 0])
    want, _ = c.run()
    c.g["plen"].fill_(1000)                              # taken as max_prefix
    c.g["lens"][0] = 2 ** 31 - 1                         # taken as max_len
    c.g["lens"][2] = -7                                  # taken as 0
    assert torch.equal(c.run()[0], want)
    c.g["plen"].fill_(-3)
    short = Case(3, 2, 4, 2, 64, 16, "bf16", 100, [50, 20, 0])
    short.P = 0
    short.check(c.run(max_prefix=100)[0])


def test_many_requests_taken_in_several_runs():
    # Parts of more than 128 MiB: requests are taken in runs that share the workspace.
    B, T, Hq, Hkv, D, P = 300, 16, 32, 4, 256, 600
    c = Case(B, T, Hq, Hkv, D, 16, "bf16", P, [i % 40 for i in range(B)], spare=0)
    c.ptable = torch.cat([c.ptable, torch.zeros(2000, dtype=torch.int32)])
    need = L.prefix_attn_workspace_bytes(B, T, Hq, Hkv, D, 30000, c.max_len)
    assert need <= L.W4A16_WORKSPACE_HEAD_BYTES + (128 << 20)
    out, lse = c.run(max_prefix=30000)
    runs = L.w4a16_last_variant().split("requests=")[1]
    assert int(runs.split()[0]) < B, runs
    c.check(out, lse, [0, 1, 140, 299])


def test_cache_past_32_bits():
    # Page strides that put pages behind 4 GiB of elements.
    D, page = 64, 16
    c = Case(2, 1, 1, 1, D, page, "bf16", 20, [3, 17], spare=0)
    stride = (1 << 29) + 64                              # six pages: the last begin behind 2^31 elements
    big = [torch.zeros((c.pages - 1) * stride + page * D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for x, src in zip(big, (c.k, c.v)):
        for p in range(c.pages):
            x[p * stride:p * stride + page * D] = src[p].reshape(-1).to(DEV)
    c.to_gpu()
    for max_prefix in (20, 2000):
        out = torch.empty(2, 1, D, dtype=torch.bfloat16, device=DEV)
        table = torch.cat([c.g["ptable"], torch.zeros(200, dtype=torch.int32, device=DEV)])
        need = L.prefix_attn_workspace_bytes(2, 1, 1, 1, D, max_prefix, 17)
        work = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
        L.prefix_attn(c.g["q"], D, big[0], big[1], "bf16", c.pages, page, stride, D, D, table, c.g["plen"], max_prefix, c.g["table"],
                      c.table.shape[1], c.g["lens"], 17, c.g["mask"], c.scale, out, None, 2, 1, 1, 1, D, work, work.numel())
        c.check(out)


@pytest.mark.parametrize("P", [40, 3000])
def test_captured_and_replayed_with_other_lengths(P):
    c = Case(6, 2, 8, 2, 128, 32, "bf16", P, [200, 10, 0, 33, 64, 100], seed=3).to_gpu()
    need = L.prefix_attn_workspace_bytes(6, 2, 8, 2, 128, P, 200)
    work = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = c.run(work=work)
    torch.cuda.synchronize()
    c.check(*first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run(work=work)
    before = {}
    for lens, plen in (([200, 10, 0, 33, 64, 100], P), ([1, 199, 50, 0, 0, 7], P - 37), ([0, 0, 0, 0, 0, 0], 1)):
        c.g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        c.g["plen"].fill_(plen)
        eager, eager_lse = c.run()
        graph.replay()
        torch.cuda.synchronize()
        # by their bits: lengths past what a request has written reach what nothing was written to, NaN here
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)) and torch.equal(lse.view(torch.int32), eager_lse.view(torch.int32))
        before[plen] = out.clone()
    assert len(before) == 3 and not torch.equal(before[1], before[P])


def test_equals_the_tree_attention_without_a_prefix():
    # The same keys as one request's context: both are within their tolerances of one definition.
    P, n, T, Hq, Hkv, D, page = 96, 40, 5, 8, 2, 128, 32
    c = Case(1, T, Hq, Hkv, D, page, "f16", P, [n], seed=4)
    c.check(*c.run())
    whole = torch.cat([c.ptable, c.table[0]]).to(DEV)                  # the prefix ends with its page
    out = torch.empty(T, Hq, D, dtype=torch.float16, device=DEV)
    need = L.tree_attn_workspace_bytes(1, T, Hq, Hkv, D, P + n)
    work = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    ps, ts, hs = c.strides()
    L.tree_attn(c.g["q"], Hq * D, c.g["k"], c.g["v"], "f16", c.pages, page, ps, ts, hs, whole, whole.numel(),
                torch.tensor([P + n], dtype=torch.int32, device=DEV), P + n, c.g["mask"], c.scale, out, None, 1, T, Hq, Hkv, D, work, work.numel())
    c.check(out)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("P,lens", [(52003, [5, 40, 0]), (0, [70000]), (17, [66001, 3])])
def test_more_than_64_parts(D, dtype, P, lens):
    # One key/value head over a long axis: as many parts of the keys as the GPU has room for.
    c = Case(len(lens), 2, 2, 1, D, 64, dtype, P, lens, seed=D)
    out, lse = c.run()
    c.check(out, lse)
    sp, so = (int(f.split("=")[1]) for f in L.w4a16_last_variant().split()[2:4])
    assert sp + so > 64 or D == 256, (sp, so)
    # A prefix far shorter than its bound leaves most parts without a key.
    if P > 70:
        c.P, c.prefix, c.g["plen"][0] = 70, [t[:70] for t in c.prefix], 70
        out, lse = c.run(max_prefix=P)
        c.check(out, lse)
