"""The rotary append, the adapters and the shared-prefix attention called side by side:
on two streams at once with a workspace each, and from two captured graphs that share one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402
from test_gpu_lora import Case as Lora  # noqa: E402
from test_gpu_prefix_attn import Case as Prefix  # noqa: E402

DEV = "cuda"


def bits(t):
    return t.contiguous().view(torch.uint8)


class Rope:
    """Rotation in place of a fused row's queries, keys and values appended."""

    def __init__(self, M, Hq, Hkv, D, seed):
        g = torch.Generator().manual_seed(seed)
        self.M, self.Hq, self.Hkv, self.D = M, Hq, Hkv, D
        self.qkv = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).bfloat16().to(DEV)
        self.k, self.v = (torch.zeros(M // 16 + 2, 16, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.slots = torch.randperm(self.k.shape[0] * 16, generator=g)[:M].to(DEV)
        self.positions = torch.randint(0, 100000, (M,), generator=g, dtype=torch.int32).to(DEV)
        self.freq = torch.tensor(L.rope_frequencies(D, 1e6), device=DEV)
        self.out = torch.zeros(M, Hq * D, dtype=torch.bfloat16, device=DEV)

    def call(self, stream=None):
        q, row, W = self.qkv, self.qkv.stride(0), self.Hq * self.D
        L.rope_append(q, row, q[:, W:], row, q[:, W + self.Hkv * self.D:], row, "bf16", self.positions, self.freq, self.D, False, 1.0, self.out, W,
                      self.k, self.v, self.k.shape[0], 16, *self.k.stride()[:3], self.slots, self.M, self.Hq, self.Hkv, self.D, stream)
        return self.out, self.k, self.v


def calls():
    """Two of each operator, of different forms: functions that call it on a stream and return what it wrote."""
    ropes = [Rope(40, 8, 2, 128, 1), Rope(900, 5, 1, 64, 2)]
    loras = [Lora(200, 2000, [128, 264], 64, 6, "bf16", "bf16", "own", seed=3).to_gpu(), Lora(5, 8192, [520], 16, 3, "f16", "f32", "own", seed=4).to_gpu()]
    prefixes = [Prefix(9, 4, 8, 2, 128, 16, "bf16", 2500, [100, 0, 7, 64, 31, 2, 5, 90, 33], seed=5).to_gpu(),
                Prefix(2, 1, 4, 4, 64, 32, "f16", 90, [700, 40], seed=6).to_gpu()]
    works = [torch.zeros(L.prefix_attn_workspace_bytes(c.B, c.T, c.Hq, c.Hkv, c.D, c.P, c.max_len) + 16, dtype=torch.uint8, device=DEV) for c in prefixes]
    pair = lambda x: [x[i] for i in range(2)]  # noqa: E731
    return pair([
        [lambda s=None, c=ropes[i]: c.call(s), lambda s=None, c=loras[i]: (c.call(s),), lambda s=None, c=prefixes[i], w=works[i]: c.run(work=w, stream=s)]
        for i in range(2)])


def test_two_streams_at_once():
    sides = calls()
    want = []
    for side in sides:
        want.append([[bits(t).clone() for t in f()] for f in side])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = [f(streams[i]) for f in sides[i]]
    torch.cuda.synchronize()
    for i in (0, 1):
        for a, b in zip(got[i], want[i]):
            assert all(torch.equal(bits(x), y) for x, y in zip(a, b))


def test_two_graphs_share_a_workspace():
    M, K, cols, R, n = 90, 4096, [256], 32, 5
    lora = Lora(M, K, cols, R, n, "bf16", "bf16", "own", seed=7).to_gpu()
    att = Prefix(6, 2, 8, 2, 64, 16, "bf16", 3000, [10, 0, 64, 200, 3, 77], seed=8).to_gpu()
    need = max(L.lora_workspace_bytes(M, sum(cols), K, R, 1), L.prefix_attn_workspace_bytes(att.B, att.T, att.Hq, att.Hkv, att.D, att.P, att.max_len))
    work = torch.zeros(need, dtype=torch.uint8, device=DEV)
    lora.work = work
    want = [bits(lora.call()).clone()] + [bits(t).clone() for t in att.run(work=work)]
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        y = lora.call()
    with torch.cuda.graph(second):
        out, lse = att.run(work=work)
    for i in range(4):
        y.fill_(9.0)
        out.fill_(9.0)
        lse.fill_(9.0)
        for graph in ((first, second) if i % 2 else (second, first)):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), b) for a, b in zip((y, out, lse), want))
        work[L.W4A16_WORKSPACE_HEAD_BYTES:].fill_(255)                   # NaN: nothing is kept from one call for the next
        torch.cuda.synchronize()
