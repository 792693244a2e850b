"""One decoder layer that verifies trees of drafted tokens, through the
library's 8-bit operators, its tree attention and its 4-bit product:

    norm + 8 bits -> qkv -> keys and values into the cache -> tree attention
    -> output projection (4-bit weights) -> residual + norm + 8 bits -> gate/up
    -> silu * up in 8 bits -> down

and, where they are given, rotary positions (rotated and put into the cache in one
pass), each request's low-rank adapter beside the qkv product, and a prefix that all
requests share.  The choice of accepted drafts is the caller's.

    python examples/decoder_layer.py [requests] [drafts] [context] [prefix]

runs a 27B-class layer (hidden 5120, 40 query and 8 key/value heads of 128,
17408 inner columns) on synthetic weights and prints its time from a captured graph; with a
prefix length (0: none) also positions and an adapter of rank 16 for each request.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_weight_only_03_amd as L  # noqa: E402

O_ROWS = 64     # rows the 4-bit product takes in a call
FP8 = torch.float8_e4m3fn
BF16 = torch.bfloat16


def blocks(n: int) -> int:
    return -(-n // 128)


def quantize_weight(w: torch.Tensor):
    """[N][K] values -> (e4m3 [N][K], scales [N/128][K/128])."""
    N, K = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128)).view(blocks(N), 128, blocks(K), 128)
    s = p.abs().amax((1, 3)).clamp_min(2.0 ** -60) / 448
    q = (p / s[:, None, :, None]).reshape(blocks(N) * 128, blocks(K) * 128)[:N, :K]
    return q.contiguous().to(FP8), s.contiguous()


class Weights:
    """A layer's weights as the library takes them.  o: (qweight, scales,
    zeros) of the 4-bit canonical format on the device, group 128."""

    def __init__(self, hidden, q_heads, kv_heads, D, inner, norm1, qkv, o, norm2, gate_up, down):
        self.hidden, self.q_heads, self.kv_heads, self.D, self.inner = hidden, q_heads, kv_heads, D, inner
        self.norm1, self.norm2 = norm1, norm2
        self.qkv, self.gate_up, self.down = quantize_weight(qkv), quantize_weight(gate_up), quantize_weight(down)
        N, K = hidden, q_heads * D
        sizes = L.w4a16_packed_sizes(N, K, 128)
        self.o = [torch.empty(n, dtype=torch.uint8, device=norm1.device) for n in sizes]
        L.w4a16_pack(*o, *self.o, N, K, 128)


class Adapters:
    """Low-rank adapters of the qkv product: a [n][3][R][hidden] (of q, k and v),
    b [n][qkv columns][R], ranks int32 [n] and scales fp32 [n] (or None), as include/lora.h takes them."""

    def __init__(self, a, b, ranks=None, scales=None):
        self.a, self.b, self.ranks, self.scales = a, b, ranks, scales
        self.n, self.R = b.shape[0], b.shape[2]


def frequencies(rot_dim: int, base: float = 1e6, factor: float = 1.0, original: float = 0.0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """The rotary frequencies as include/rope_append.h scales them, on the device."""
    return torch.tensor(L.rope_frequencies(rot_dim, base, factor, original, slow, fast), device=device)


class Layer:
    """Buffers for B requests with T drafts each over a paged cache, and the
    layer's calls.  Everything is allocated here, so that a call can be captured.
    rope: rotary frequencies, or None; adapters: Adapters, or None; max_prefix:
    the most tokens of a shared prefix, or None for a batch that shares nothing."""

    def __init__(self, w: Weights, B: int, T: int, pages: int, page: int, max_len: int, rope=None, adapters=None, max_prefix=None):
        self.w, self.B, self.T, self.M, self.page, self.max_len = w, B, T, B * T, page, max_len
        self.rope, self.adapters, self.max_prefix = rope, adapters, max_prefix
        dev, M = w.norm1.device, self.M
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        self.k = new(pages, page, w.kv_heads, w.D).zero_()
        self.v = torch.zeros_like(self.k)
        self.x8, self.xs = new(M, w.hidden, dtype=FP8), new(blocks(w.hidden), M, dtype=torch.float32)
        self.qkv = new(M, (w.q_heads + 2 * w.kv_heads) * w.D)
        self.att, self.o, self.h = new(M, w.q_heads * w.D), new(M, w.hidden), new(M, w.hidden)
        self.gu, self.a8 = new(M, 2 * w.inner), new(M, w.inner, dtype=FP8)
        self.as_, self.y = new(blocks(w.inner), M, dtype=torch.float32), new(M, w.hidden)
        n = max(L.w8a8_workspace_bytes(M, self.qkv.shape[1], w.hidden), L.w8a8_workspace_bytes(M, 2 * w.inner, w.hidden),
                L.w8a8_workspace_bytes(M, w.hidden, w.inner),
                *(L.w4a16_workspace_bytes(m, w.hidden, w.q_heads * w.D, 128) for m in self.o_rows()),
                L.tree_attn_workspace_bytes(B, T, w.q_heads, w.kv_heads, w.D, max_len))
        if adapters:
            self.xn = new(M, w.hidden)
            n = max(n, L.lora_workspace_bytes(M, self.qkv.shape[1], w.hidden, adapters.R, 3))
        if max_prefix is not None:
            n = max(n, L.prefix_attn_workspace_bytes(B, T, w.q_heads, w.kv_heads, w.D, max_prefix, max_len))
        self.work = torch.zeros(max(n, 16), dtype=torch.uint8, device=dev)   # its head has to start as zeros

    def o_rows(self):
        """The rows of each call of the output projection."""
        return [min(O_ROWS, self.M - m) for m in range(0, self.M, O_ROWS)]

    def product(self, x8, xs, weight, y):
        (q, s), (M, N) = weight, y.shape
        L.w8a8_gemm(x8, xs, q, s, y, "bf16", M, N, q.shape[1], self.work, self.work.numel())

    def append(self, positions, slots):
        """The new keys and values into the cache, rotated (as the queries are) where there are frequencies."""
        w, M = self.w, self.M
        qw, kw, ld = w.q_heads * w.D, w.kv_heads * w.D, self.qkv.stride(0)
        q, k, v = self.qkv, self.qkv[:, qw:], self.qkv[:, qw + kw:]
        if self.rope is None:
            self.k.view(-1, w.kv_heads, w.D)[slots] = k[:, :kw].view(M, w.kv_heads, w.D)
            self.v.view(-1, w.kv_heads, w.D)[slots] = v.view(M, w.kv_heads, w.D)
            return
        L.rope_append(q, ld, k, ld, v, ld, "bf16", positions, self.rope, 2 * self.rope.numel(), False, 1.0, q, ld, self.k, self.v,
                      self.k.shape[0], self.page, *self.k.stride()[:3], slots, M, w.q_heads, w.kv_heads, w.D)

    def attention(self, table, lens, mask, prefix):
        w, B, T = self.w, self.B, self.T
        cache = (self.qkv, self.qkv.stride(0), self.k, self.v, "bf16", self.k.shape[0], self.page, *self.k.stride()[:3])
        own = (table, table.shape[1], lens, self.max_len, mask, w.D ** -0.5, self.att, None, B, T, w.q_heads, w.kv_heads, w.D,
               self.work, self.work.numel())
        if self.max_prefix is None:
            L.tree_attn(*cache, *own)
        else:
            L.prefix_attn(*cache, *prefix, self.max_prefix, *own)

    def __call__(self, x, table, lens, mask, slots, positions=None, adapter=None, prefix=(None, None)):
        """x [M][hidden]: the residual stream.  table [B][pages], lens [B],
        mask [B][T] (uint64 bits as int64): see include/tree_attn.h.  slots
        [M]: page * page_size + offset of each draft's place in the cache.
        positions int32 [M] of a layer with rope; adapter int32 [M] of one with
        adapters; prefix (pages, length int32 [1]) of one with a prefix: see include/prefix_attn.h.
        Returns (residual stream after attention, this layer's output to add to it)."""
        w, M = self.w, self.M
        qw, kw = w.q_heads * w.D, w.kv_heads * w.D
        lora = self.adapters
        L.w8a8_rmsnorm_quant(x, "bf16", w.hidden, None, "bf16", None, w.norm1, "bf16", 1e-6, self.xn if lora else None, "bf16", self.x8, self.xs, M, w.hidden)
        self.product(self.x8, self.xs, w.qkv, self.qkv)
        if lora:
            L.lora_add(self.xn, "bf16", w.hidden, lora.a, lora.b, lora.ranks, lora.scales, lora.n, adapter, self.qkv, self.qkv, "bf16",
                       self.qkv.shape[1], [qw, kw, kw], M, self.qkv.shape[1], w.hidden, lora.R, self.work, self.work.numel())
        self.append(positions, slots)
        self.attention(table, lens, mask, prefix)
        for i, m in enumerate(self.o_rows()):
            L.w4a16_gemv(self.att[O_ROWS * i:], "bf16", *w.o, self.o[O_ROWS * i:], "bf16", m, w.hidden, qw, 128, self.work, self.work.numel())
        L.w8a8_rmsnorm_quant(self.o, "bf16", w.hidden, x, "bf16", self.h, w.norm2, "bf16", 1e-6, None, "bf16", self.x8, self.xs, M, w.hidden)
        self.product(self.x8, self.xs, w.gate_up, self.gu)
        L.w8a8_silu_mul_quant(self.gu, "bf16", 2 * w.inner, None, "bf16", self.a8, self.as_, M, w.inner)
        self.product(self.a8, self.as_, w.down, self.y)
        return self.h, self.y


def main():
    B, T, n, shared = (int(v) for v in (sys.argv[1:] + ["1", "8", "8192", "-1"][len(sys.argv) - 1:]))
    hidden, q_heads, kv_heads, D, inner, page = 5120, 40, 8, 128, 17408, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bits = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)  # noqa: E731
    o = (bits(hidden, q_heads * D // 8), (randn(q_heads * D // 128, hidden) * 1e-3).half().view(torch.int16), bits(q_heads * D // 128, hidden // 8))
    w = Weights(hidden, q_heads, kv_heads, D, inner, (1 + 0.1 * randn(hidden)).to(BF16), randn((q_heads + 2 * kv_heads) * D, hidden) * 0.02, o,
                (1 + 0.1 * randn(hidden)).to(BF16), randn(2 * inner, hidden) * 0.02, randn(hidden, inner) * 0.02)
    per, own = -(-(n + T) // page), max(shared, 0)
    options, inputs = {}, ()
    if shared >= 0:
        # The prefix's pages lie behind the requests' own.
        width, pages = (q_heads + 2 * kv_heads) * D, -(-shared // page)
        options = dict(rope=frequencies(D), max_prefix=shared,
                       adapters=Adapters((randn(B, 3, 16, hidden) * hidden ** -0.5).to(BF16), (randn(B, width, 16) * 0.1).to(BF16)))
        inputs = (shared + n + torch.arange(T, device="cuda", dtype=torch.int32).repeat(B),
                  torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(T),
                  (torch.arange(B * per, B * per + pages, device="cuda", dtype=torch.int32) if pages else None,
                   torch.full((1,), shared, device="cuda", dtype=torch.int32)))
    layer = Layer(w, B, T, B * per + -(-own // page), page, n, **options)
    layer.k.normal_(generator=g)
    layer.v.normal_(generator=g)
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    parent = [(i - 1) // 2 for i in range(T)]                         # a binary tree
    row = []
    for i in range(T):
        row.append((row[parent[i]] if i else 0) | 1 << i)
    mask = torch.tensor([[r - (1 << 64) if r >> 63 else r for r in row]] * B, device="cuda")
    p = n + torch.arange(T, device="cuda")
    slots = (table[:, p // page].long() * page + p % page).view(-1)
    x = (2 * randn(B * T, hidden)).to(BF16)
    call = lambda: layer(x, table, lens, mask, slots, *inputs)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(50):
        graph.replay()
    e.record()
    torch.cuda.synchronize()
    h, y = layer.h.float(), layer.y.float()
    print(f"{B} requests x {T} drafts over {n} tokens{f' behind {shared} shared' if shared >= 0 else ''}: {a.elapsed_time(e) / 50 * 1e3:.1f} us a layer; "
          f"residual rms {h.square().mean().sqrt():.3f}, output rms {y.square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
