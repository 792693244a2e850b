"""GPU tests of the draft-tree attention (include/tree_attn.h) against its
definition in 64 bits on the CPU.

Tolerances.  u = 2^-24, ut the type's unit roundoff.  A score is an fp32 sum of D
products (error at most (D + 4) u times the sum of magnitudes, scale included);
with the exponential's argument rounded twice and 2^x good to a few u, a
probability is off by at most e = (D + 4) u S + 4 u (A + 4) of itself, S the largest sum of
magnitudes of a score and A the largest |score|.  Each enters the product with
v rounded once more (ut), sums over keys are fp32 (n + 64 roundings at worst
between them, far fewer in the same sum), and the quotient is rounded to the
type.  All of it relative to the mean |v| under the probabilities."""
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
    def __init__(self, B, T, Hq, Hkv, D, page, dtype, lens, seed=0, heads_first=False, q_pad=0, mask=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.Hq, self.Hkv, self.D, self.page, self.dtype = B, T, Hq, Hkv, D, page, dtype
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.max_len = max(lens)
        per = -(-(self.max_len + T) // page)
        self.pages = B * per + spare
        shape = (self.pages, Hkv, page, D) if heads_first else (self.pages, page, Hkv, D)
        ty = TYPES[dtype]
        # what no position maps to holds NaN: it must never be seen
        self.k, self.v = (torch.full(shape, float("nan"), dtype=ty) for _ in range(2))
        self.table = torch.randperm(self.pages, generator=g)[:B * per].to(torch.int32).view(B, per)
        self.heads_first = heads_first
        self.dense = []
        for b in range(B):
            n = int(self.lens[b]) + T
            kd, vd = (torch.randn(n, Hkv, D, generator=g).to(ty) for _ in range(2))
            self.dense.append([kd, vd])
        self.q = torch.randn(B * T, Hq * D + q_pad, generator=g).to(ty)
        self.scale = D ** -0.5
        if mask is None:
            mask = np.zeros((B, T), dtype=np.uint64)
            for b in range(B):
                for i in range(T):
                    parent = int(torch.randint(-1, max(i, 1), (1,), generator=g)) if i else -1
                    mask[b, i] = (mask[b, parent] if parent >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
        self.mask = np.asarray(mask, dtype=np.uint64)
        self.store()

    def store(self):
        for b in range(self.B):
            for c, d in ((self.k, self.dense[b][0]), (self.v, self.dense[b][1])):
                for i in range(-(-d.shape[0] // self.page)):
                    part = d[i * self.page:(i + 1) * self.page]
                    p = int(self.table[b, i])
                    if self.heads_first:
                        c[p, :, :part.shape[0]] = part.transpose(0, 1)
                    else:
                        c[p, :part.shape[0]] = part

    def on_gpu(self):
        self.g = dict(q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV), table=self.table.to(DEV), lens=self.lens.to(DEV),
                      mask=torch.from_numpy(self.mask.view(np.int64).copy()).to(DEV))
        return self

    def strides(self):
        s = self.k.stride()
        return (s[0], s[2], s[1]) if self.heads_first else (s[0], s[1], s[2])

    def run(self, max_len=None, work=None, lse=True, stream=None, out=None, lse_out=None):
        if not hasattr(self, "g"):
            self.on_gpu()
        max_len = self.max_len if max_len is None else max_len
        out = torch.full((self.B * self.T, self.Hq, self.D), float("nan"), dtype=TYPES[self.dtype], device=DEV) if out is None else out
        if lse_out is None:
            lse_out = torch.full((self.B * self.T, self.Hq), float("nan"), device=DEV) if lse else None
        need = L.tree_attn_workspace_bytes(self.B, self.T, self.Hq, self.Hkv, self.D, max_len)
        if work is None:
            work = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
        ps, ts, hs = self.strides()
        L.tree_attn(self.g["q"], self.q.stride(0), self.g["k"], self.g["v"], self.dtype, self.pages, self.page, ps, ts, hs,
                    self.g["table"], self.table.shape[1], self.g["lens"], max_len, self.g["mask"], self.scale, out, lse_out,
                    self.B, self.T, self.Hq, self.Hkv, self.D, work, work.numel(), stream)
        return out, lse_out

    def sees(self, b):
        n = int(self.lens[b])
        s = torch.ones(self.T, n + self.T, dtype=torch.bool)
        for i in range(self.T):
            for j in range(self.T):
                s[i, n + j] = bool(int(self.mask[b, i]) >> j & 1)
        return s

    def reference(self):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
        B, T, Hq, D, G = self.B, self.T, self.Hq, self.D, self.Hq // self.Hkv
        out, tol = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.zeros(B, T, Hq, D, dtype=torch.float64)
        lse, ltol = torch.full((B, T, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, T, Hq, dtype=torch.float64)
        for b in range(B):
            s = self.sees(b)
            k, v = (x.double() for x in self.dense[b])
            for h in range(Hq):
                q = self.q[b * T:(b + 1) * T, h * D:(h + 1) * D].double()
                kh, vh = k[:, h // G], v[:, h // G]
                for i in range(T):
                    at = s[i].nonzero()[:, 0]
                    if not len(at):
                        continue
                    a = kh[at] @ q[i] * self.scale
                    mag = kh[at].abs() @ q[i].abs() * self.scale
                    lse[b, i, h] = torch.logsumexp(a, 0)
                    p = torch.softmax(a, 0)
                    o = p @ vh[at]
                    e = (D + 4) * U * mag.max() + 4 * U * (a.abs().max() + 4) + (len(at) + 64) * U
                    out[b, i, h] = o
                    tol[b, i, h] = (UT[self.dtype] + 2 * e) * (p @ vh[at].abs()) + UT[self.dtype] * o.abs() + 2.0 ** -25
                    ltol[b, i, h] = e + 2 * U * lse[b, i, h].abs()
        return tuple(x.view(B * T, Hq, *x.shape[3:]) for x in (out, lse, tol, ltol))

    def check(self, got, lse=None):
        out, want_lse, tol, ltol = self.reference()
        err = (got.cpu().double() - out).abs()
        assert torch.all(err <= tol), (L.w4a16_last_variant(), float((err / tol).max()), (err > tol).nonzero()[:4].tolist())
        if lse is not None:
            got_lse = lse.cpu().double()
            none = torch.isinf(want_lse)
            assert torch.equal(got_lse[none], want_lse[none])
            assert torch.all((got_lse - want_lse)[~none].abs() <= ltol[~none])


CASES = [
    # B, T, Hq, Hkv, D, page, dtype, lens, heads_first, q_pad
    (1, 1, 1, 1, 64, 16, "bf16", [0], False, 0),            # one draft, nothing else
    (1, 1, 5, 1, 128, 16, "bf16", [1], False, 0),
    (2, 1, 8, 8, 128, 32, "f16", [31, 33], False, 8),
    (3, 1, 40, 8, 128, 64, "bf16", [700, 0, 64], False, 2048),
    (1, 1, 16, 2, 256, 16, "bf16", [515], True, 0),
    (2, 3, 10, 2, 64, 1, "f16", [37, 5], False, 0),          # pages of one token
    (2, 7, 10, 2, 128, 8, "bf16", [95, 96], True, 16),       # pages shorter than a tile
    (4, 16, 10, 2, 128, 32, "bf16", [300, 17, 0, 129], False, 0),   # 80 rows
    (1, 8, 40, 8, 128, 64, "bf16", [1000], False, 0),        # 40 rows
    (1, 13, 4, 2, 256, 128, "f16", [401], False, 0),         # 26 rows
    (1, 64, 2, 2, 64, 16, "f16", [100], False, 0),
    (2, 64, 8, 1, 128, 32, "bf16", [65, 2], False, 0),       # 512 rows
    (1, 40, 6, 1, 256, 64, "bf16", [90], True, 0),           # 240 rows
    (1, 33, 3, 3, 64, 256, "bf16", [257], False, 0),
    (1, 2, 16, 1, 128, 16, "f16", [2500], False, 0),         # 32 rows
    (1, 4, 5, 1, 64, 32, "bf16", [6000], False, 0),          # split over the keys
    (1, 5, 20, 4, 256, 64, "f16", [3000], False, 0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,dtype,lens,heads_first,q_pad", CASES)
def test_matches_definition(B, T, Hq, Hkv, D, page, dtype, lens, heads_first, q_pad):
    c = Case(B, T, Hq, Hkv, D, page, dtype, lens, seed=T + Hq + D, heads_first=heads_first, q_pad=q_pad)
    out, lse = c.run()
    c.check(out, lse)
    again, _ = c.run(lse=False)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    # a looser bound on the lengths splits the keys otherwise
    if (c.max_len + 4096 + T) <= c.table.shape[1] * page:
        c.check(*c.run(max_len=c.max_len + 4096))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(6, 2, 2, 128), (20, 2, 1, 64), (30, 4, 1, 128), (40, 1, 1, 256), (9, 1, 1, 256)])
def test_rows_that_see_nothing_and_values_that_are_not_seen(dtype, T, Hq, Hkv, D):
    # Request 0 has no context: its rows see at most themselves, every third
    # nothing.  Request 1 has one.  Drafts that no row, or only their own row,
    # sees hold NaN and infinities in k and v.
    B = 2
    mask = np.zeros((B, T), dtype=np.uint64)
    for i in range(T):
        if i % 3:
            mask[:, i] = np.uint64(1) << np.uint64(i)
    c = Case(B, T, Hq, Hkv, D, 16, dtype, [0, 45], seed=T, mask=mask)
    c.dense[0][0][0] = float("nan")                      # drafts 0, 3, .. are seen by nobody
    c.dense[0][1][3] = float("inf")
    c.dense[1][0][45] = float("inf")
    c.dense[1][1][48] = float("nan")
    c.store()
    out, lse = c.run()
    ref = Case(B, T, Hq, Hkv, D, 16, dtype, [0, 45], seed=T, mask=mask)
    ref.check(out, lse)                                  # as if they were ordinary numbers
    empty = out.view(B, T, Hq, D)[0, ::3]
    assert torch.all(empty == 0) and torch.all(torch.isneginf(lse.view(B, T, Hq)[0, ::3]))
    # A NaN and an infinity that only their own row sees change that row alone.
    c.dense[1][1][45 + 4, :, 7] = float("nan")
    c.dense[1][1][45 + 5, :, 9] = float("-inf")
    c.store()
    out2, lse2 = Case.run(c.on_gpu())
    o, o2 = out.view(B, T, Hq, D).cpu().float(), out2.view(B, T, Hq, D).cpu().float()
    assert torch.all(torch.isnan(o2[1, 4, :, 7])) and torch.all(torch.isneginf(o2[1, 5, :, 9]))
    o2[1, 4, :, 7], o2[1, 5, :, 9] = o[1, 4, :, 7], o[1, 5, :, 9]
    # The finite columns of the two rows were summed with one value less in the
    # matrix unit's tile, nothing else: all as before.
    assert torch.equal(o, o2)
    assert torch.equal(lse.cpu(), lse2.cpu())


def test_infinite_scores_and_nan_in_the_context():
    c = Case(1, 2, 2, 1, 64, 16, "bf16", [70], mask=[[1, 3]])
    c.dense[0][1][10, 0, 5] = float("nan")               # every row sees the context
    c.store()
    out, _ = c.run()
    o = out.cpu().float()
    assert torch.all(torch.isnan(o[:, :, 5])) and torch.all(torch.isfinite(o[:, :, :5]))
    c = Case(1, 2, 2, 1, 64, 16, "bf16", [70], mask=[[1, 3]])
    c.dense[0][0][20] = float("nan")
    c.store()
    out, lse = c.run()
    assert torch.all(torch.isnan(out.float())) and torch.all(torch.isnan(lse))
    # A key far below the others (as a masked one is in other code) counts nothing.
    c = Case(1, 1, 2, 1, 64, 16, "bf16", [70], mask=[[1]])
    c.q[:] = 1.0
    c.dense[0][0][33] = -3e38
    c.store()
    out, lse = c.run()
    k, v = c.dense[0][0].double(), c.dense[0][1].double()
    a = k[:, 0].sum(1) * c.scale
    p = torch.softmax(a, 0)
    assert p[33] == 0 and torch.all((out.cpu().double()[0] - p @ v[:, 0]).abs() < 0.02)


def test_every_key_counts_once():
    # Equal scores and one-hot values: out = (how often a column's key is seen) / n,
    # over lengths around the tiles', splits' and pages' ends.
    for dtype, D, Hq, T, page in (("f16", 64, 1, 1, 16), ("bf16", 128, 5, 1, 32), ("f16", 128, 5, 16, 64), ("bf16", 256, 2, 20, 16)):
        for n in (1, 31, 32, 33, 63, 64, 127, 129, 255, 1000, 4095):
            mask = [[(1 << T) - 1] * T]
            c = Case(1, T, Hq, 1, D, page, dtype, [n], mask=mask)
            total = n + T
            c.dense[0][0][:] = 0
            v = torch.zeros(total, 1, D)
            v[torch.arange(total), 0, torch.arange(total) % D] = 1
            c.dense[0][1][:] = v
            c.store()
            out, lse = c.run()
            want = torch.bincount(torch.arange(total) % D, minlength=D).double() / total
            assert torch.all((out.cpu().double() - want).abs() <= 2 * UT[dtype] * want + 1e-12), (dtype, D, n)
            assert torch.all((lse.cpu().double() - math.log(total)).abs() <= 16 * U * (1 + math.log(total)))


def test_many_small_probabilities():
    # One key 16 above 40 000 others: each of those has 2^-23 of its
    # probability, all together 0.45 % of the sum, and their values are 100.
    n, D = 40000, 64
    for dtype in ("f16", "bf16"):
        c = Case(1, 1, 1, 1, D, 64, dtype, [n], mask=[[1]])
        c.q[:] = 0
        c.q[0, 0] = 1
        c.scale = 1.0
        k, v = c.dense[0]
        k[:] = 0
        k[:, 0, 0] = -16
        k[5, 0, 0] = 0
        v[:] = 100
        v[5] = 0
        c.store()
        out, lse = c.run()
        rest = n * math.exp(-16)
        want = 100 * rest / (1 + rest)
        assert torch.all((out.cpu().double() - want).abs() <= (2 * UT[dtype] + 64 * U) * want), (dtype, float(out[0, 0, 0]), want)
        assert abs(float(lse[0, 0]) - math.log1p(rest)) < 1e-5


def test_table_entries_and_lengths_out_of_range_stay_in_bounds():
    # Entries past a request's own pages hold anything; lens beyond max_len counts as max_len.
    c = Case(2, 2, 4, 2, 64, 16, "bf16", [40, 9])
    want, want_lse = c.run()
    t = torch.tensor([[-5], [10 ** 9]], dtype=torch.int32).expand(2, 3)
    c.table = torch.cat([c.table, t], 1).contiguous()
    c.on_gpu()
    out, lse = c.run()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    c.g["table"][0, 0] = 10 ** 9          # taken as the last page
    c.g["lens"][1] = 1 << 30              # taken as max_len
    c.run()
    c.g["lens"][1] = -3                   # taken as 0
    c.run()
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    # Pages more than 4 GiB from the start of the cache, and elements past 2^31.
    B, T, Hq, Hkv, D, page, n = 1, 3, 4, 2, 128, 16, 200
    c = Case(B, T, Hq, Hkv, D, page, "bf16", [n])
    per = page * Hkv * D
    far = (1 << 32) // per + 7            # element offset past 2^32
    big_k, big_v = (torch.empty((far + c.pages) * per, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    big_k[far * per:] = c.k.to(DEV).view(-1)
    big_v[far * per:] = c.v.to(DEV).view(-1)
    want, want_lse = c.run()
    c.g["k"], c.g["v"] = big_k, big_v
    c.g["table"] = c.g["table"] + far
    c.pages += far
    out, lse = c.run()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)


def test_graph_replays_with_other_lengths_and_a_shared_workspace():
    c = Case(2, 4, 10, 2, 128, 32, "bf16", [900, 300])
    d = Case(1, 1, 8, 8, 64, 16, "f16", [2000])
    need = max(L.tree_attn_workspace_bytes(x.B, x.T, x.Hq, x.Hkv, x.D, x.max_len) for x in (c, d))
    assert need > 0
    work = torch.zeros(need, dtype=torch.uint8, device=DEV)
    work[L.W4A16_WORKSPACE_HEAD_BYTES:].view(torch.float32).fill_(float("nan"))
    want = [x.run(work=work) for x in (c, d)]
    torch.cuda.synchronize()
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for x, (o, l) in zip((c, d), outs):
            x.run(work=work, stream=s, out=o, lse_out=l)
    for lens in ([900, 300], [1, 900], [0, 0], [900, 300]):
        c.g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        for o, l in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = c.run(work=work)
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0].view(torch.int16), eager[0].view(torch.int16)) and torch.equal(outs[0][1].view(torch.int32), eager[1].view(torch.int32))
        assert torch.equal(outs[1][0].view(torch.int16), want[1][0].view(torch.int16))
    assert torch.equal(outs[0][0].view(torch.int16), want[0][0].view(torch.int16))
    assert not work[:L.W4A16_WORKSPACE_HEAD_BYTES].any()


def test_parts_of_an_odd_number_of_rows_and_splits_are_aligned():
    # The sums of the parts are stored 16 bytes at a time: they have to begin the scratch (16-byte aligned), the pairs
    # (maximum in log2 units, sum) follow.  Joined from there they are the call's result.
    c = Case(1, 1, 5, 1, 128, 16, "bf16", [1200])
    need = L.tree_attn_workspace_bytes(1, 1, 5, 1, 128, 1200)
    work = torch.zeros(need, dtype=torch.uint8, device=DEV)
    out, lse = c.run(work=work)
    splits = int(dict(f.split("=") for f in L.w4a16_last_variant().split()[1:])["splits"])
    assert splits > 1 and (5 * splits) % 2 == 1
    parts = work[L.W4A16_WORKSPACE_HEAD_BYTES:].view(torch.float32)
    o = parts[:5 * splits * 128].view(5, splits, 128).cpu().double()
    m, l = parts[5 * splits * 128:][:5 * splits * 2].view(5, splits, 2).cpu().double().unbind(2)
    f = torch.exp2(m - m.amax(1, keepdim=True))
    want = (f[:, :, None] * o).sum(1) / (f * l).sum(1, keepdim=True)
    assert torch.all((out.cpu().double()[0] - want).abs() <= UT["bf16"] * want.abs() + 64 * U * (f[:, :, None] * o).abs().sum(1) / (f * l).sum(1, keepdim=True))
    c.check(out, lse)


def check_units(c, out, lse):
    """Case.check over the rows of a request and kv head at once (the same definition and tolerances, for larger cases)."""
    T, G, D = c.T, c.Hq // c.Hkv, c.D
    out = out.cpu().double().view(c.B, T, c.Hkv, G, D)
    lse = lse.cpu().double().view(c.B, T, c.Hkv, G)
    q = c.q[:, :c.Hq * D].double().view(c.B, T, c.Hkv, G, D)
    for b in range(c.B):
        sees = c.sees(b)[:, None, :].expand(T, G, -1).reshape(T * G, -1)
        some = sees.any(1)
        k, v = (x.double() for x in c.dense[b])
        for h in range(c.Hkv):
            rows = q[b, :, h].reshape(T * G, D)
            a = (rows @ k[:, h].t() * c.scale).masked_fill(~sees, -math.inf)
            mag = (rows.abs() @ k[:, h].abs().t() * c.scale).masked_fill(~sees, 0)
            want_lse = torch.logsumexp(a, 1)
            p = torch.exp(a - torch.where(some, want_lse, 0.0)[:, None])
            o = p @ v[:, h]
            e = (D + 4) * U * mag.amax(1) + 4 * U * (a.abs().masked_fill(~sees, 0).amax(1) + 4) + (sees.sum(1) + 64) * U
            tol = (UT[c.dtype] + 2 * e)[:, None] * (p @ v[:, h].abs()) + UT[c.dtype] * o.abs() + 2.0 ** -25
            err = (out[b, :, h].reshape(T * G, D) - o).abs()
            assert torch.all(err <= tol), (b, h, float((err / tol).max()), (err > tol).nonzero()[:4].tolist())
            got = lse[b, :, h].reshape(T * G)
            assert torch.all(out[b, :, h].reshape(T * G, D)[~some] == 0) and torch.all(torch.isneginf(got[~some]))
            assert torch.all(((got - want_lse).abs() <= e + 2 * U * want_lse.abs())[some])


# Every kernel, with the keys whole and split and with several blocks of rows, over enough tiles that each ring slot is
# filled again several times: 9 tiles a group of waves at least where a ring is four deep, 4 where it is two.
KERNELS = [
    # B, T, Hq, Hkv, D, len, page -> rows and key groups of a workgroup, split, blocks of rows
    (1, 1, 1, 1, 64, 700, 16, 16, 4, False, 1), (64, 1, 1, 1, 64, 4097, 64, 16, 4, True, 1), (1, 21, 1, 1, 64, 500, 32, 16, 4, False, 2),
    (96, 21, 3, 3, 64, 500, 16, 32, 4, False, 1), (32, 33, 1, 1, 64, 4097, 32, 32, 4, True, 2), (96, 33, 2, 2, 64, 500, 64, 32, 4, False, 2),
    (96, 33, 3, 3, 64, 700, 16, 64, 2, False, 1), (96, 33, 1, 1, 64, 4097, 32, 64, 2, True, 1), (96, 13, 10, 2, 64, 700, 8, 64, 2, False, 2),
    (96, 13, 15, 3, 64, 333, 16, 128, 1, False, 1), (48, 33, 9, 3, 64, 2100, 64, 128, 1, True, 1), (96, 21, 16, 2, 64, 333, 4, 128, 1, False, 2),
    (1, 5, 1, 1, 128, 700, 32, 16, 4, False, 1), (32, 1, 1, 1, 128, 4097, 16, 16, 4, True, 1), (1, 21, 1, 1, 128, 500, 64, 16, 4, False, 2),
    (48, 21, 3, 3, 128, 500, 8, 32, 4, False, 1), (16, 33, 1, 1, 128, 4097, 64, 32, 4, True, 2), (96, 33, 1, 1, 128, 500, 16, 32, 4, False, 2),
    (1, 8, 40, 8, 128, 8192, 64, 32, 4, True, 2), (1, 4, 40, 8, 128, 20000, 32, 32, 4, True, 1),
    (48, 33, 3, 3, 128, 700, 32, 64, 2, False, 1), (24, 33, 1, 1, 128, 6000, 64, 64, 2, True, 1), (96, 13, 5, 1, 128, 700, 16, 64, 2, False, 2),
    (96, 1, 3, 3, 128, 333, 2, 128, 1, False, 1), (32, 13, 5, 1, 128, 3000, 32, 128, 1, True, 1), (96, 21, 8, 1, 128, 333, 16, 128, 1, False, 2),
    (1, 1, 1, 1, 256, 333, 16, 16, 2, False, 1), (16, 1, 1, 1, 256, 4097, 32, 16, 2, True, 1), (1, 4, 5, 1, 256, 333, 64, 16, 2, False, 2),
    (48, 4, 15, 3, 256, 333, 8, 64, 1, False, 1), (24, 4, 5, 1, 256, 3000, 16, 64, 1, True, 1), (24, 21, 8, 1, 256, 333, 32, 64, 1, False, 3),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,n,page,rows,groups,split,row_blocks", KERNELS)
def test_each_kernel_over_many_tiles(dtype, B, T, Hq, Hkv, D, n, page, rows, groups, split, row_blocks):
    g = torch.Generator().manual_seed(n + B)
    # the first request has the whole length; of the others some have little or nothing: fewer tiles than splits
    lens = [n] + [int(torch.randint(0, n + 1, (1,), generator=g)) if b % 5 else b % 7 for b in range(1, B)]
    c = Case(B, T, Hq, Hkv, D, page, dtype, lens, seed=n)
    c.mask[B // 2, ::3] = 0                     # some rows see their context alone
    out, lse = c.run()
    ran = dict(f.split("=") for f in L.w4a16_last_variant().split()[1:])
    assert (int(ran["rows"]), int(ran["groups"]), int(ran["splits"]) > 1, int(ran["row_blocks"])) == (rows, groups, split, row_blocks), ran
    tiles = -(-(n + T) // 32)
    assert tiles // int(ran["splits"]) // groups >= (4 if rows <= 32 else 9), ran
    check_units(c, out, lse)


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,dtype,lens,heads_first,q_pad", CASES)
def test_a_looser_bound_on_the_lengths(B, T, Hq, Hkv, D, page, dtype, lens, heads_first, q_pad):
    # Planned for far longer contexts than there are: splits with no tiles, parts that have seen nothing.
    c = Case(B, T, Hq, Hkv, D, page, dtype, lens, seed=T + Hq + D, heads_first=heads_first, q_pad=q_pad)
    some_split = False
    for more in (4096, 60000):
        table = torch.full((B, -(-(c.max_len + more + T) // page)), 10 ** 9, dtype=torch.int32)   # past a request's pages: anything
        table[:, :c.table.shape[1]] = c.table[:, :table.shape[1]]
        wide = Case(B, T, Hq, Hkv, D, page, dtype, lens, seed=T + Hq + D, heads_first=heads_first, q_pad=q_pad)
        wide.table = table
        out, lse = wide.run(max_len=c.max_len + more)
        some_split |= "splits=1 " not in L.w4a16_last_variant()
        c.check(out, lse)
    assert some_split


def test_graph_replays_match_the_definition():
    # One capture, planned for 900 tokens, replayed for other lengths with the program's own calls between the replays.
    c = Case(2, 4, 10, 2, 128, 32, "bf16", [900, 900], seed=3)
    work = torch.zeros(L.tree_attn_workspace_bytes(2, 4, 10, 2, 128, 900), dtype=torch.uint8, device=DEV)
    assert work.numel() > L.W4A16_WORKSPACE_HEAD_BYTES
    c.run(work=work)
    torch.cuda.synchronize()
    out = torch.empty(8, 10, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(8, 10, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(work=work, stream=s, out=out, lse_out=lse)
    full = c.dense
    for lens in ([900, 900], [1, 900], [0, 0], [333, 31], [900, 2]):
        c.lens = torch.tensor(lens, dtype=torch.int32)
        c.dense = [[d[:n + 4] for d in full[b]] for b, n in enumerate(lens)]   # the drafts are what the cache holds after n
        c.g["lens"].copy_(c.lens)
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_units(c, out, lse)
        eager = c.run(work=work)
        torch.cuda.synchronize()
        assert torch.equal(eager[0].view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,n,page,rows,groups,split,row_blocks", [k for k in KERNELS if k[1] > 2])
def test_each_kernel_keeps_what_is_not_seen_out(dtype, B, T, Hq, Hkv, D, n, page, rows, groups, split, row_blocks):
    # Draft 1 is seen by nobody and holds NaN and infinities; then draft 0 has an infinity in one column of v, which
    # becomes the result's for the rows that see it and changes no bit of any other.
    c = Case(B, T, Hq, Hkv, D, page, dtype, [n if b % 3 == 0 else (7 * b) % 64 for b in range(B)], seed=n)
    c.mask &= ~np.uint64(2)
    want, want_lse = c.run()
    for b in range(B):
        k, v = c.dense[b]
        at = int(c.lens[b])
        k[at + 1], v[at + 1, :, ::2], v[at + 1, :, 1::2] = float("nan"), float("inf"), float("nan")
    c.store()
    out, lse = c.on_gpu().run()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    for b in range(B):
        c.dense[b][1][int(c.lens[b]), :, D - 3] = float("inf")
    c.store()
    out, lse = c.on_gpu().run()
    assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    sees = torch.from_numpy((c.mask & np.uint64(1)) != 0).view(B * T, 1).expand(B * T, Hq)
    out, want = out.cpu(), want.cpu()
    assert torch.all(out[..., D - 3][sees] == float("inf"))
    out[..., D - 3][sees] = want[..., D - 3][sees]
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
