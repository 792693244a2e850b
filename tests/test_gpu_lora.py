"""GPU tests of the low-rank adapters (include/lora.h) against their definition
in 64 bits.

Tolerance.  u = 2^-24, ut the result type's half step.  h is an fp32 sum of K exact
products: off by at most K u of their magnitudes, plus 16 u for the waves', slices' and scale's
roundings; of s h, 2^-16 (f32 result: 2^-21) of the row's largest element is left out of each;
the second product adds r (terms of) products and the base in fp32: (3 r + 4) u of their
magnitudes; and y takes half a step of its type (fp16 an absolute 2^-25)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": U}
NAN = float("nan")


class Case:
    """What a call must not look at holds NaN: columns past K and N, ranks past an adapter's, adapters that no row uses."""

    def __init__(self, M, K, cols, R, n, dtype, y, base="own", ids=None, ranks=None, scales=True, x_pad=0, y_pad=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        N, P, ty = sum(cols), len(cols), TYPES[dtype]
        self.M, self.N, self.K, self.R, self.n, self.cols, self.dtype, self.y, self.mode = M, N, K, R, n, cols, dtype, y, base
        self.ids = torch.randint(-1, n, (M,), generator=g, dtype=torch.int32) if ids is None else torch.tensor(ids, dtype=torch.int32)
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32)
        self.scales = torch.rand(n, generator=g) * 2 if scales else None
        self.x = torch.full((M, K + x_pad), NAN).to(ty)
        self.x[:, :K] = torch.randn(M, K, generator=g).to(ty)
        self.a = (torch.randn(n, P, R, K, generator=g) * K ** -0.5).to(ty)
        self.b = (torch.randn(n, N, R, generator=g) * 0.3).to(ty)
        for i in range(n):
            if i not in self.ids.tolist():
                self.a[i], self.b[i] = NAN, NAN
            r = self.rank(i)
            r8 = -(-r // 8) * 8
            self.a[i, :, r:], self.b[i, :, r:] = 0, 0
            self.a[i, :, r8:], self.b[i, :, r8:] = NAN, NAN
        self.base = torch.full((M, N + y_pad), NAN).to(TYPES[y])
        self.base[:, :N] = torch.randn(M, N, generator=g).to(TYPES[y])

    def rank(self, i):
        return self.R if self.ranks is None else min(max(int(self.ranks[i]), 0), self.R)

    def to_gpu(self):
        self.g = {k: None if getattr(self, k) is None else getattr(self, k).to(DEV) for k in ("x", "a", "b", "ranks", "scales", "ids", "base")}
        self.g["out"] = self.g["base"] if self.mode == "in place" else torch.full_like(self.g["base"], 9.0)
        need = L.lora_workspace_bytes(self.M, self.N, self.K, self.R, len(self.cols))
        self.work = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)      # NaN but for its head
        self.work[:L.W4A16_WORKSPACE_HEAD_BYTES] = 0
        return self

    def call(self, stream=None):
        g = self.g
        L.lora_add(g["x"], self.dtype, self.x.shape[1], g["a"], g["b"], g["ranks"], g["scales"], self.n, g["ids"], None if self.mode == "none" else g["base"],
                   g["out"], self.y, self.base.shape[1], self.cols if len(self.cols) > 1 else None, self.M, self.N, self.K, self.R, self.work,
                   self.work.numel() if self.work.numel() > 16 else 0, stream)
        return g["out"]

    def reference(self):
        M, N = self.M, self.N
        want = torch.zeros(M, N, dtype=torch.float64) if self.mode == "none" else self.base[:, :N].double()
        tol, left = want.abs() * 4 * U, 2.0 ** -16 if self.y != "f32" else 2.0 ** -21
        for i in range(self.n):
            rows, r, s = (self.ids == i).nonzero()[:, 0], self.rank(i), 1.0 if self.scales is None else float(self.scales[i])
            if not len(rows) or not r:
                continue
            x, first = self.x[rows, :self.K].double(), 0
            for p, width in enumerate(self.cols):
                a, b = self.a[i, p, :r].double(), self.b[i, first:first + width, :r].double()
                h, mag = s * x @ a.t(), s * x.abs() @ a.abs().t()
                off = (self.K + 16) * U * mag + left * h.abs().amax(1, keepdim=True)
                want[rows, first:first + width] += h @ b.t()
                tol[rows, first:first + width] += off @ b.abs().t() + (3 * r + 4) * U * (h.abs() @ b.abs().t())
                first += width
        return want, 1.01 * tol + UT[self.y] * want.abs() + (2.0 ** -25 if self.y == "f16" else 2.0 ** -140)

    def check(self, out):
        want, tol = self.reference()
        got = out[:, :self.N].cpu().double()
        err = (got - want).abs()
        assert torch.all(err <= tol), (L.w4a16_last_variant(), float((err / tol).nan_to_num(1e9).max()), (~(err <= tol)).nonzero()[:4].tolist())
        pad = out[:, self.N:].cpu()
        assert torch.all(torch.isnan(pad) if self.mode == "in place" else pad == 9.0)


CASES = [
    # M, K, cols, R, n, dtype, y, base, keywords
    (1, 8, [8], 8, 1, "bf16", "bf16", "own", dict(ids=[0])),                               # the least of everything
    (1, 5120, [5120, 1024, 1024], 16, 4, "bf16", "bf16", "own", dict(ids=[2])),
    (1, 512, [128, 64], 16, 3, "f16", "f16", "in place", dict(ids=[-1])),                  # a row without
    (5, 200, [72], 16, 3, "f16", "f32", "none", dict(ids=[2, 0, -1, 2, 7])),               # an adapter that is not there
    (16, 328, [64, 64, 64, 24], 24, 16, "bf16", "f32", "own", dict(ids=list(range(16)), x_pad=8, y_pad=16)),   # all different
    (37, 1000, [264], 40, 5, "bf16", "bf16", "in place", dict(ranks=[0, 3, 8, 40, 100], x_pad=24, y_pad=8)),
    (64, 640, [320, 104], 32, 48, "f16", "f16", "own", dict(ranks=[32, 16, 8] * 16)),
    (33, 96, [1032], 256, 3, "bf16", "f32", "own", dict(ranks=[256, 129, -5])),
    (20, 4096, [520], 128, 2, "f16", "bf16", "none", {}),                                  # two launches
    (11, 17384, [648], 64, 5, "bf16", "f32", "own", dict(ranks=[64, 32, 16, 60, 1])),
    (3, 100008, [72], 8, 2, "bf16", "f32", "in place", dict(ids=[1, 1, 0])),
    (530, 256, [136], 16, 7, "bf16", "bf16", "own", dict(y_pad=8)),                        # a workgroup takes all adapters of a tile
    (600, 2048, [192, 64], 104, 3, "f16", "f32", "in place", dict(ranks=[104, 50, 8])),
    (1100, 136, [64, 1000], 8, 4, "f16", "f16", "own", dict(ids=[i // 300 - 1 for i in range(1100)], scales=False)),
    (2, 4000, [128, 128, 64], 64, 2, "bf16", "bf16", "own", {}),                           # rows of a by three workgroups
    (70, 2000, [576], 128, 4, "f16", "f16", "own", dict(ranks=[128, 64, 7, 96])),
    (200, 328, [264], 64, 6, "bf16", "bf16", "own", dict(ranks=[64, 40, 33, 32, 8, 0])),   # a tile's adapters over several workgroups
    (65, 72, [8], 8, 20, "f16", "f32", "in place", {}),
    (520, 1000, [16384, 64], 32, 40, "bf16", "bf16", "own", dict(ids=[i // 5 % 41 - 1 for i in range(520)])),
    (700, 96, [512, 136], 48, 5, "f16", "f32", "in place", dict(ranks=[48, 41, 16, 5, 33])),
    (4100, 64, [2048, 520], 16, 3, "bf16", "bf16", "own", {}),                             # runs of row tiles, several adapters in each
    (3003, 72, [2048, 1032], 64, 4, "bf16", "f32", "own", dict(ids=[i // 100 % 5 - 1 for i in range(3003)])),
    (1300, 40, [1024], 256, 3, "bf16", "bf16", "none", dict(ranks=[256, 200, 65])),
]


@pytest.mark.parametrize("M,K,cols,R,n,dtype,y,base,kw", CASES)
def test_matches_definition(M, K, cols, R, n, dtype, y, base, kw):
    c = Case(M, K, cols, R, n, dtype, y, base, seed=M + K, **kw).to_gpu()
    out = c.call()
    c.check(out)
    assert torch.all(c.work[:L.W4A16_WORKSPACE_HEAD_BYTES][:16] == (0 if c.work.numel() > 16 else c.work[:16]))
    if base != "in place":
        again = out.clone()
        out.fill_(9.0)
        assert torch.equal(c.call()[:, :c.N], again[:, :c.N])


@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("K,R", [(72, 16), (4096, 64)])
def test_values_past_a_type_and_of_every_size(dtype, y, K, R):
    # h of a row from 2^-60 to 2^60 times the others': fp16's range does not bound it.
    c = Case(24, K, [72], R, 2, dtype, "f32", "none", ids=[i % 2 for i in range(24)], seed=3)
    c.y = "f32"
    c.scales = torch.tensor([2.0 ** 60, 2.0 ** -60])
    if dtype == "f16":
        c.x[:, :K] *= 2.0 ** 10
    out = c.to_gpu().call()
    c.check(out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,R", [(20, 200, 16), (20, 8192, 32), (520, 64, 8)])
def test_infinity_and_nan_stay_in_their_row(dtype, M, K, R):
    ids = [i % 3 - 1 for i in range(M)]
    clean = Case(M, K, [64, 40], R, 2, dtype, dtype, "own", ids=ids, seed=4)
    odd = Case(M, K, [64, 40], R, 2, dtype, dtype, "own", ids=ids, seed=4)
    odd.x[1, 5], odd.x[2, K - 1], odd.x[3, 0] = NAN, float("inf"), NAN
    odd.base[4, 7] = float("-inf")
    a, b = clean.to_gpu().call().cpu().float(), odd.to_gpu().call().cpu().float()
    assert torch.all(torch.isnan(b[1])) and not torch.any(torch.isfinite(b[2]))
    assert torch.equal(b[3], a[3])                                                          # row 3 has no adapter: x is not looked at
    assert torch.isneginf(b[4, 7])
    b[1], b[2], b[4, 7] = a[1], a[2], a[4, 7]
    assert torch.equal(a, b)


def test_an_infinite_sum_is_infinite():
    # One element of h infinite, the others ordinary, b positive: y is +infinity, not NaN.
    for dtype in ("f16", "bf16"):
        c = Case(3, 64, [64], 16, 1, dtype, "f32", "own", ids=[0, 0, 0], seed=5)
        c.x[1, 9] = float("inf")
        c.a[0, 0] = c.a[0, 0].abs()
        c.b = c.b.abs() + 0.01
        out = c.to_gpu().call().cpu()
        assert torch.all(torch.isposinf(out[1])) and torch.all(torch.isfinite(out[[0, 2]]))


def test_adapters_past_32_bits():
    # 9 adapters of 2^28 elements of a each: the last lies behind 4 GiB.
    K, R, n = 1 << 20, 256, 9
    a = torch.zeros(n, R, K, dtype=torch.bfloat16, device=DEV)
    b = torch.zeros(n, 64, R, dtype=torch.bfloat16, device=DEV)
    a[8, 255, K - 1], b[8, 63, 255] = 2.0, 3.0
    a[7, 255, K - 1] = 100.0
    x = torch.ones(2, K, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([8, 3], dtype=torch.int32, device=DEV)
    y = torch.empty(2, 64, device=DEV)
    need = L.lora_workspace_bytes(2, 64, K, R)
    work = torch.zeros(need, dtype=torch.uint8, device=DEV)
    L.lora_add(x, "bf16", K, a, b, None, None, n, ids, None, y, "f32", 64, None, 2, 64, K, R, work, need)
    want = torch.zeros(2, 64)
    want[0, 63] = 6.0
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,K,R", [(9, 256, 16), (9, 8192, 64)])
def test_captured_and_replayed_with_other_adapters(M, K, R):
    c = Case(M, K, [64, 200], R, 6, "bf16", "bf16", "own", ids=[i % 6 for i in range(M)], seed=6).to_gpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()
    torch.cuda.synchronize()
    c.check(c.g["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for i in range(3):
        c.ids = (c.ids + 2) % 7 - 1                                    # read on the device at each replay
        c.g["ids"].copy_(c.ids)
        c.g["out"].fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(c.g["out"])


def test_after_the_shared_projection():
    # The 4-bit product, then each row's adapter on its result, through one workspace.
    M, N, K, R, n = 7, 264, 1152, 16, 3
    g = torch.Generator().manual_seed(8)
    q = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 8), generator=g).to(torch.int32).to(DEV)
    s = (torch.rand(K // 128, N, generator=g) * 0.01).half().view(torch.int16).to(DEV)
    z = torch.randint(-2 ** 31, 2 ** 31 - 1, (K // 128, N // 8), generator=g).to(torch.int32).to(DEV)
    packed = [torch.empty(b, dtype=torch.uint8, device=DEV) for b in L.w4a16_packed_sizes(N, K, 128)]
    L.w4a16_pack(q, s, z, *packed, N, K, 128)
    w = torch.empty(K, N, device=DEV)
    L.w4a16_dequant(*packed, w, N, K, 128)
    c = Case(M, K, [N], R, n, "bf16", "f32", "in place", seed=8).to_gpu()
    need = max(L.w4a16_workspace_bytes(M, N, K, 128), L.lora_workspace_bytes(M, N, K, R), 16)
    c.work = torch.zeros(need, dtype=torch.uint8, device=DEV)
    L.w4a16_gemv(c.g["x"], "bf16", *packed, c.g["out"], "f32", M, N, K, 128, c.work, need)
    c.base = c.g["out"].cpu()
    product = c.x.double() @ w.cpu().double()
    assert float((c.base.double() - product).norm() / product.norm()) <= 1e-3
    c.call()
    want, tol = c.reference()
    assert torch.all((c.g["out"].cpu().double() - want).abs() <= tol)


@pytest.mark.parametrize("M,K,R", [(14, 200, 16), (40, 4000, 40), (130, 200, 24), (600, 72, 16), (600, 72, 72)])
def test_more_than_64_adapters(M, K, R):
    n = 200
    ids = [(i * 37 + 60) % (n + 1) - 1 for i in range(M)]
    c = Case(M, K, [136], R, n, "bf16", "bf16", "own", ids=ids, ranks=[i * 5 % (R + 1) for i in range(n)], seed=M).to_gpu()
    c.check(c.call())
