"""GPU tests of rotary positions and the append to the paged cache
(include/rope_append.h) against the definition in 64 bits.

Tolerance.  u = 2^-24, ut the type's half step.  The fraction of a quarter turn
is rounded to fp32, times a rounded pi/2: the reduced angle (at most pi/4) is off
by at most 3 u; the 64-bit product before it by two roundings of |p f| 2^-53 in
radians.  The Taylor sums round their last steps (2 u) and leave out 2^-29, the
gain rounds once more: c and s are off by at most gain (6 u + 4 |p f| 2^-53).  The
rotation is a product and an fma: 2 u of (|x| + |y|) gain more, and the result
takes half a step of its type (fp16 has an absolute one of 2^-25 below 2^-14)."""
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
    def __init__(self, M, Hq, Hkv, D, rot, interleaved, page, dtype, pad=0, heads_first=False, far=5000, gain=1.0, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.M, self.Hq, self.Hkv, self.D, self.rot, self.interleaved, self.page, self.dtype = M, Hq, Hkv, D, rot, interleaved, page, dtype
        self.gain, self.pad, self.heads_first, ty = gain, pad, heads_first, TYPES[dtype]
        self.rows = torch.randn(M, (Hq + 2 * Hkv) * D + pad, generator=g).to(ty)
        self.pages = -(-M // page) + spare
        shape = (self.pages, Hkv, page, D) if heads_first else (self.pages, page, Hkv, D)
        self.k, self.v = (torch.randn(shape, generator=g).to(ty) for _ in range(2))
        self.slots = torch.randperm(self.pages * page, generator=g)[:M]
        self.positions = torch.randint(0, far + 1, (M,), generator=g, dtype=torch.int32)
        self.freq = torch.tensor(L.rope_frequencies(rot, 1e6, 4.0, 1000.0), dtype=torch.float32) if rot else None

    def to_gpu(self):
        self.g = {n: getattr(self, n).to(DEV) for n in ("rows", "k", "v", "slots", "positions")}
        self.g["freq"] = self.freq.to(DEV) if self.rot else None
        self.g["out"] = torch.full((self.M, self.Hq * self.D + 8), 7.0, dtype=TYPES[self.dtype], device=DEV)
        return self

    def strides(self):
        s = self.k.stride()
        return (s[0], s[2], s[1]) if self.heads_first else (s[0], s[1], s[2])

    def call(self, q=True, kv=True, in_place=False, stream=None):
        g, row, Hq, Hkv, D = self.g, self.g["rows"].stride(0), self.Hq, self.Hkv, self.D
        qkv = g["rows"]
        out = qkv if in_place else g["out"]
        L.rope_append(qkv if q else None, row, qkv[:, Hq * D:] if kv else None, row, qkv[:, (Hq + Hkv) * D:] if kv else None, row, self.dtype,
                      g["positions"] if self.rot else None, g["freq"], self.rot, self.interleaved, self.gain, out if q else None, out.stride(0),
                      g["k"] if kv else None, g["v"] if kv else None, self.pages, self.page, *self.strides(), g["slots"] if kv else None,
                      self.M, Hq, Hkv, D, stream)

    def rotated(self, x):
        """(values, tolerance) of x [M][heads][D] in 64 bits."""
        n, x = self.rot // 2, x.double()
        want, tol = x.clone(), torch.zeros_like(x)
        if n:
            first = torch.arange(n) if not self.interleaved else 2 * torch.arange(n)
            second = first + (n if not self.interleaved else 1)
            angle = self.positions.double()[:, None] * self.freq.double()
            c, s = (self.gain * f(angle)[:, None] for f in (torch.cos, torch.sin))
            u, v = x[..., first], x[..., second]
            want[..., first], want[..., second] = u * c - v * s, v * c + u * s
            e = (u.abs() + v.abs()) * abs(self.gain) * (8 * U + 4 * 2.0 ** -53 * angle.abs()[:, None])
            for at in (first, second):
                tol[..., at] = 1.01 * e + UT[self.dtype] * want[..., at].abs() + 2.0 ** -25
        return want, tol

    def check(self, out, k=True):
        M, Hq, Hkv, D = self.M, self.Hq, self.Hkv, self.D
        heads = self.rows[:, :(Hq + 2 * Hkv) * D].view(M, -1, D)
        if out is not None:
            want, tol = self.rotated(heads[:, :Hq])
            got = out[:, :Hq * D].cpu().double().view(M, Hq, D)
            assert torch.all((got - want).abs() <= tol), float(((got - want).abs() - tol).max())
        if k:
            want_k, tol_k = (self.k.double(), torch.zeros(self.k.shape, dtype=torch.float64))
            want_v = self.v.clone()
            rk, tk = self.rotated(heads[:, Hq:Hq + Hkv])
            for m, s in enumerate(self.slots.tolist()):
                if 0 <= s < self.pages * self.page:
                    p, i = divmod(s, self.page)
                    at = (p, slice(None), i) if self.heads_first else (p, i)
                    want_k[at], tol_k[at], want_v[at] = rk[m], tk[m], heads[m, Hq + Hkv:]
            assert torch.all((self.g["k"].cpu().double() - want_k).abs() <= tol_k)
            assert torch.equal(self.g["v"].cpu(), want_v)


CASES = [
    # M, Hq, Hkv, D, rot, interleaved, page, dtype, pad, heads_first
    (1, 40, 8, 128, 128, 0, 64, "bf16", 0, False),
    (1, 1, 1, 16, 16, 1, 1, "f16", 0, False),             # the least of everything
    (1, 1, 1, 16, 0, 0, 1, "bf16", 8, False),             # nothing rotated
    (7, 5, 1, 64, 64, 1, 16, "f16", 16, True),
    (37, 16, 2, 256, 64, 1, 16, "f16", 0, False),         # a quarter of the head
    (33, 6, 3, 80, 32, 0, 8, "bf16", 0, False),           # five threads a head
    (20, 3, 3, 112, 112, 0, 32, "f16", 24, True),
    (9, 12, 4, 96, 48, 1, 16, "bf16", 0, False),
    (3, 2, 1, 512, 512, 0, 4, "bf16", 0, False),
    (2, 64, 64, 256, 256, 0, 16, "bf16", 0, False),       # more heads than a workgroup's threads: 3 workgroups a token
    (300, 71, 1, 64, 32, 1, 128, "bf16", 0, False),
    (3001, 40, 8, 128, 128, 0, 64, "bf16", 0, False),     # four heads per thread
    (2500, 17, 5, 256, 128, 1, 16, "f16", 8, True),
    (300, 128, 65, 256, 96, 0, 64, "f16", 0, False),      # four heads per thread, two workgroups a token
]


@pytest.mark.parametrize("M,Hq,Hkv,D,rot,interleaved,page,dtype,pad,heads_first", CASES)
def test_matches_definition(M, Hq, Hkv, D, rot, interleaved, page, dtype, pad, heads_first):
    c = Case(M, Hq, Hkv, D, rot, interleaved, page, dtype, pad, heads_first, seed=M + D).to_gpu()
    c.call()
    c.check(c.g["out"])
    assert torch.all(c.g["out"][:, Hq * D:] == 7.0)                     # between the rows
    assert torch.equal(c.g["rows"].cpu(), c.rows)
    first = {n: c.g[n].clone() for n in ("out", "k", "v")}
    c.call()                                                            # the same again
    assert all(torch.equal(first[n], c.g[n]) for n in first)
    c.call(in_place=True)
    assert torch.equal(c.g["rows"][:, :Hq * D], first["out"][:, :Hq * D])
    assert torch.equal(c.g["rows"][:, Hq * D:].cpu(), c.rows[:, Hq * D:])


@pytest.mark.parametrize("far,gain", [(1 << 20, 1.0), ((1 << 31) - 1, 1.0), (1000, -0.25), (0, 1.5)])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_far_positions_and_gain(far, gain, interleaved):
    c = Case(50, 2, 1, 64, 64, interleaved, 16, "f16", gain=gain, seed=far % 97)
    c.positions = torch.linspace(0, far, 50, dtype=torch.float64).to(torch.int64).clamp(max=(1 << 31) - 1).to(torch.int32)
    c.positions[1::2] *= -1
    c.to_gpu().call()
    c.check(c.g["out"])


def test_slots_outside_append_nothing():
    c = Case(40, 4, 2, 64, 64, 0, 16, "bf16", seed=5)
    end = c.pages * c.page
    c.slots[::5] = -1
    c.slots[1], c.slots[2], c.slots[3], c.slots[4] = end, end + 7, -(1 << 62), (1 << 62) + 5
    c.slots[6] = (1 << 32) + 3
    c.to_gpu().call()
    c.check(c.g["out"])
    c = Case(6, 4, 2, 64, 64, 0, 16, "bf16", seed=6)
    c.slots[:] = -1
    c.to_gpu().call()
    c.check(c.g["out"])


def test_only_queries_or_only_keys():
    c = Case(11, 4, 2, 128, 64, 0, 16, "f16", seed=7).to_gpu()
    c.call(kv=False)
    c.check(c.g["out"], k=False)
    assert torch.equal(c.g["k"].cpu(), c.k) and torch.equal(c.g["v"].cpu(), c.v)
    c = Case(11, 4, 2, 128, 64, 1, 16, "f16", seed=8).to_gpu()
    c.call(q=False)
    c.check(None)
    assert torch.all(c.g["out"] == 7.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_what_is_not_rotated_keeps_its_bits(dtype):
    c = Case(5, 2, 1, 64, 32, 0, 16, dtype, seed=9)
    raw = c.rows.view(torch.int16)
    raw[:, 32:64] = torch.arange(0x7c00, 0x7c00 + 32, dtype=torch.int16)   # NaN payloads, infinities
    raw[:, -64:] = torch.arange(-64, 0, dtype=torch.int16)
    c.to_gpu().call()
    got = c.g["out"].view(torch.int16).cpu()
    assert torch.equal(got[:, 32:64], raw[:, 32:64])
    v = c.g["v"].view(torch.int16).cpu().view(-1, 64)
    assert torch.equal(v[c.slots], raw[:, -64:])


def test_infinity_and_nan_stay_in_their_pair():
    c = Case(3, 2, 1, 64, 64, 0, 16, "bf16", far=50, seed=10)
    c.positions += 1
    c.rows[0, 3], c.rows[1, 64 + 40] = float("nan"), float("inf")
    clean = Case(3, 2, 1, 64, 64, 0, 16, "bf16", far=50, seed=10)
    clean.positions += 1
    c.to_gpu().call()
    clean.to_gpu().call()
    a, b = c.g["out"].float().cpu(), clean.g["out"].float().cpu()
    odd = ~torch.isfinite(a)
    assert odd.nonzero().tolist() == [[0, 3], [0, 35], [1, 64 + 8], [1, 64 + 40]]
    assert torch.equal(a[~odd], b[~odd])


def test_cache_past_32_bits():
    # Page strides that put the last page behind 4 GiB of elements.
    D, page, Hkv = 64, 16, 1
    stride = (1 << 31) + 64
    c = Case(2, 1, Hkv, D, 64, 0, page, "bf16", seed=11)
    cache = torch.zeros(2 * stride + page * D, dtype=torch.bfloat16, device=DEV)
    c.to_gpu()
    c.slots = torch.tensor([2 * page + 3, page + 15])
    slots = c.slots.to(DEV)
    row = c.g["rows"].stride(0)
    other = torch.empty_like(cache)
    L.rope_append(None, 0, c.g["rows"][:, D:], row, c.g["rows"][:, 2 * D:], row, "bf16", c.g["positions"], c.g["freq"], 64, 0, 1.0, None, 0,
                  cache, other, 3, page, stride, D, D, slots, 2, 1, Hkv, D)
    want, tol = c.rotated(c.rows[:, D:2 * D].view(2, 1, D))
    for m, at in enumerate((2 * stride + 3 * D, stride + 15 * D)):
        assert torch.all((cache[at:at + D].cpu().double() - want[m, 0]).abs() <= tol[m, 0])
        assert torch.equal(other[at:at + D].cpu(), c.rows[m, 2 * D:3 * D])
    assert int((cache != 0).sum()) <= 2 * D


def test_captured_and_replayed_on_its_own_stream():
    c = Case(13, 8, 2, 128, 128, 0, 16, "bf16", seed=12).to_gpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()                                                    # the current stream
    torch.cuda.synchronize()
    want = {n: c.g[n].clone() for n in ("out", "k", "v")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for i in range(3):
        c.g["positions"] += 1                                       # read on the device at each replay
        c.positions += 1
        c.g["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check(c.g["out"])
        assert not torch.equal(c.g["out"][:, :64], want["out"][:, :64])
