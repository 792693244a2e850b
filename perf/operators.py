"""The operators of an 8-bit decoder layer that verifies drafted tokens: what is timed, on which sizes, and their plain forms.

  norm   h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; y in 8 bits with a scale for each 128 columns of a row
  gated  y = silu(gate) * up from the fused product's two halves, in 8 bits with the same scales
  gemm   y = x . w^T of two 8-bit operands: a scale for each 128 columns of a row of x, one for each 128 x 128 block of w
  tree   attention of a tree of drafted tokens over a paged cache: a draft sees its whole context and its ancestors

8 bits are OCP E4M3 (largest value 448).  Lengths 5120, 7168, 17408, 34816 are the 27B-class layer's of the benchmark."""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -60        # least magnitude a block's scale is made for
WORKSPACE = 128 << 20     # scratch a serving program sets aside once, zeroed once, for all of its calls
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # the residual and norm before qkv of one generated token: latency alone
        {"name": "norm one token", "op": "norm", "M": 1, "K": 5120, "dtype": "bf16", "add": True, "y": False},
        # drafts of several requests, a length that ends inside a block, the 16-bit norm wanted as well (for a 4-bit layer)
        {"name": "norm ragged", "op": "norm", "M": 37, "K": 4112, "dtype": "f16", "add": True, "y": True},
        # a long prompt: bound by memory
        {"name": "norm prompt", "op": "norm", "M": 8192, "K": 5120, "dtype": "bf16", "add": True, "y": False},
        # eight drafts between the gate/up and the down product
        {"name": "gated drafts", "op": "gated", "M": 8, "K": 17408, "dtype": "bf16", "y": False},
        # the same of a prompt
        {"name": "gated prompt", "op": "gated", "M": 4096, "K": 17408, "dtype": "bf16", "y": False},
        # qkv of one generated token: one read of the weights
        {"name": "gemm one token", "op": "gemm", "M": 1, "N": 7168, "K": 5120, "dtype": "bf16"},
        # down for eight drafts: few columns, a long sum
        {"name": "gemm drafts", "op": "gemm", "M": 8, "N": 5120, "K": 17408, "dtype": "bf16"},
        # a short prompt's chunk, sizes that end inside every tile
        {"name": "gemm ragged", "op": "gemm", "M": 100, "N": 5128, "K": 5136, "dtype": "f16"},
        # gate/up of a prompt: bound by the matrix units
        {"name": "gemm prompt", "op": "gemm", "M": 4096, "N": 34816, "K": 5120, "dtype": "bf16"},
        # one token over the longest context, no drafts beside it: one read of the cache
        {"name": "tree one token long", "op": "tree", "B": 1, "T": 1, "L": 150000, "Hq": 40, "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # four requests of different lengths, each with 16 drafts
        {"name": "tree drafts", "op": "tree", "B": 4, "T": 16, "L": 4097, "Hq": 40, "Hkv": 8, "D": 128, "page": 32, "dtype": "bf16"},
        # the widest tree, a head of its own for each query head, a short context
        {"name": "tree wide", "op": "tree", "B": 3, "T": 64, "L": 777, "Hq": 16, "Hkv": 16, "D": 64, "page": 16, "dtype": "f16"},
    ]


def spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "gated", "gemm", "gemm", "tree", "tree"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "norm":
        K = spread(rng, 64, 16384, 16)
        return {"op": op, "M": spread(rng, 1, min(16384, 8192 * 5120 // K)), "K": K, "dtype": dtype, "add": rng.random() < 0.8, "y": rng.random() < 0.3}
    if op == "gated":
        K = spread(rng, 64, 17408, 16)
        return {"op": op, "M": spread(rng, 1, min(16384, 4096 * 17408 // K)), "K": K, "dtype": dtype, "y": rng.random() < 0.2}
    if op == "gemm":
        N, K = spread(rng, 64, 34816, 8), spread(rng, 64, 17408, 16)
        return {"op": op, "M": spread(rng, 1, max(1, min(8192, 4096 * 34816 * 5120 // (N * K)))), "N": N, "K": K, "dtype": dtype}
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8, 8, 16))
    Hq = Hkv * rng.choice((1, 2, 4, 5, 5, 8))
    B, T = rng.choice((1, 1, 2, 3, 8, 16)), spread(rng, 1, 64)
    most = min(150000 * 1024 // (B * Hkv * D), 400_000_000 // (B * T * Hq), 150000)
    return {"op": op, "B": B, "T": T, "L": spread(rng, 1, max(1, most)), "Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice((16, 32, 64, 128)), "dtype": dtype}


def blocks(n):
    return -(-n // BLOCK)


def widen(s, rows, cols):
    """Scales of 128 x 128 blocks, one for each element."""
    return s.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    s["work"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    if case["op"] == "tree":
        return prepare_tree(s, g, normal)
    M, K, dtype = case["M"], case["K"], TYPES[case["dtype"]]
    if case["op"] == "gemm":
        N = case["N"]
        x = normal(M, K)
        x *= 1 + 20 * (torch.rand(K, generator=g, device="cuda") < 0.002)     # a few columns are large in every row
        xp = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(M, -1, BLOCK)
        xs = xp.abs().amax(2).clamp_min(FLOOR) / 448
        s["x"] = (xp / xs[:, :, None]).view(M, -1)[:, :K].contiguous().to(FP8)
        s["x_scales"] = xs.t().contiguous()
        w = normal(N, K) * 0.02
        wp = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK)).view(blocks(N), BLOCK, blocks(K), BLOCK)
        s["w_scales"] = wp.abs().amax((1, 3)).clamp_min(FLOOR) / 448
        s["w"] = (w / widen(s["w_scales"], N, K)).to(FP8)
        s["out"] = torch.empty(M, N, dtype=dtype, device="cuda")
        return s
    if case["op"] == "norm":
        s["x"] = normal(M, K).to(dtype)
        res = normal(M, K) * 2
        res *= 1 + 50 * (torch.rand(K, generator=g, device="cuda") < 0.002)
        s["residual"] = res.to(dtype) if case["add"] else None
        s["weight"] = (1 + 0.2 * normal(K)).to(dtype)
        s["h"] = torch.empty(M, K, dtype=dtype, device="cuda") if case["add"] else None
    else:
        s["x"] = (normal(M, 2 * K) * 1.5).to(dtype)
    s["y_out"] = torch.empty(M, K, dtype=dtype, device="cuda") if case["y"] else None
    s["q"] = torch.empty(M, K, dtype=FP8, device="cuda")
    s["scales"] = torch.empty(blocks(K), M, dtype=torch.float32, device="cuda")
    return s


def prepare_tree(s, g, normal):
    B, T, L, Hq, Hkv, D, page, dtype = (s[k] for k in ("B", "T", "L", "Hq", "Hkv", "D", "page", "dtype"))
    dtype = TYPES[dtype]
    pages = -(-(L + T) // page)
    s["q"] = normal(B * T, Hq, D).to(dtype)
    s["k"] = torch.empty(B * pages, page, Hkv, D, dtype=dtype, device="cuda").normal_(generator=g)
    s["v"] = torch.empty(B * pages, page, Hkv, D, dtype=dtype, device="cuda").normal_(generator=g)
    s["table"] = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    # the first request has the whole length, the others less, the last of several none where the length is short
    lens = torch.randint(L // 2, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = L
    if B > 2 and L < 1024:
        lens[-1] = 0
    s["lens"] = lens
    # a tree: each draft hangs on an earlier one, or starts a branch; one request in four leaves its last rows unused
    at = torch.arange(T, device="cuda")
    parent = (torch.rand(B, T, generator=g, device="cuda") * (at + 1)).long() - 1
    see = torch.zeros(B, T + 1, T, dtype=torch.bool, device="cuda")            # row T: a root's parent sees no draft
    for i in range(T):
        see[:, i] = see[torch.arange(B, device="cuda"), parent[:, i] % (T + 1)]
        see[:, i, i] = True
    see = see[:, :T]
    if B > 3:
        see[3::4, T - T // 4:] = False
    s["mask"] = (see.long() << at).sum(2)
    s["scale"] = D ** -0.5
    s["out"] = torch.empty(B * T, Hq, D, dtype=dtype, device="cuda")
    s["lse"] = torch.empty(B * T, Hq, dtype=torch.float32, device="cuda")
    return s


def run(s):
    if own:
        import bit_weight_only_03_amd as L
        dtype = s["dtype"]
        if s["op"] == "norm":
            L.w8a8_rmsnorm_quant(s["x"], dtype, s["K"], s["residual"], dtype, s["h"], s["weight"], dtype, 1e-6, s["y_out"], dtype, s["q"], s["scales"], s["M"], s["K"])
            return {"h": s["h"], "y": s["y_out"], "q": s["q"], "scales": s["scales"]}
        if s["op"] == "gated":
            L.w8a8_silu_mul_quant(s["x"], dtype, 2 * s["K"], s["y_out"], dtype, s["q"], s["scales"], s["M"], s["K"])
            return {"y": s["y_out"], "q": s["q"], "scales": s["scales"]}
        if s["op"] == "gemm":
            L.w8a8_gemm(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], dtype, s["M"], s["N"], s["K"], s["work"], WORKSPACE)
            return s["out"]
        kv = s["k"]
        L.tree_attn(s["q"], s["q"].stride(0), kv, s["v"], dtype, kv.shape[0], s["page"], kv.stride(0), kv.stride(1), kv.stride(2), s["table"], s["table"].shape[1],
                    s["lens"], s["L"], s["mask"], s["scale"], s["out"], s["lse"], s["B"], s["T"], s["Hq"], s["Hkv"], s["D"], s["work"], WORKSPACE)
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "norm":
        return plain_norm(s)
    if s["op"] == "gated":
        return plain_gated(s)
    return plain_gemm(s) if s["op"] == "gemm" else plain_tree(s)


def quantized(y):
    """(8-bit values, scales [blocks][rows]) of y in 32 bits."""
    M, K = y.shape
    b = torch.nn.functional.pad(y, (0, -K % BLOCK)).view(M, -1, BLOCK)
    s = b.abs().amax(2).clamp_min(FLOOR) / 448
    return (b / s[:, :, None]).view(M, -1)[:, :K].contiguous().to(FP8), s.t().contiguous()


def plain_norm(s):
    h = s["x"].float()
    if s["add"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    q, scales = quantized(y)
    return {"h": h.to(s["x"].dtype) if s["add"] else None, "y": y.to(s["x"].dtype) if s["y"] else None, "q": q, "scales": scales}


def plain_gated(s):
    gate, up = s["x"][:, :s["K"]].float(), s["x"][:, s["K"]:].float()
    y = gate / (1 + torch.exp(-gate)) * up
    q, scales = quantized(y)
    return {"y": y.to(s["x"].dtype) if s["y"] else None, "q": q, "scales": scales}


def plain_gemm(s):
    M, N, K = s["M"], s["N"], s["K"]
    x = s["x"].float() * s["x_scales"].t().repeat_interleave(BLOCK, 1)[:, :K]
    w = s["w"].float() * widen(s["w_scales"], N, K)
    return (x @ w.t()).to(s["out"].dtype)


def tree_sees(s, P):
    """[B, T, P]: whether draft i of request b sees the key at position p."""
    at, lens = torch.arange(P, device="cuda"), s["lens"].long()[:, None, None]
    bit = (s["mask"][:, :, None] >> (at - lens).clamp(0, 63)) & 1
    return (at < lens) | ((at >= lens) & (at < lens + s["T"]) & (bit == 1))


def plain_tree(s):
    B, T, Hq, Hkv, D = (s[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    P, G = s["L"] + T, Hq // Hkv
    k = s["k"][s["table"].long()].flatten(1, 2)[:, :P].permute(0, 2, 3, 1).float()          # [B, Hkv, D, P]
    v = s["v"][s["table"].long()].flatten(1, 2)[:, :P].transpose(1, 2).float()              # [B, Hkv, P, D]
    q = s["q"].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).float().reshape(B, Hkv, T * G, D)
    see = tree_sees(s, P)[:, None, :, None, :]
    a = (q @ k.contiguous() * s["scale"]).view(B, Hkv, T, G, P).masked_fill(~see, -math.inf)
    top = a.amax(4, keepdim=True).clamp_min(-1e30)                                          # finite where a row sees nothing
    a = torch.exp(a - top)
    total = a.sum(4, keepdim=True)
    o = (a.view(B, Hkv, T * G, P) @ v.contiguous()).view(B, Hkv, T, G, D) / total.clamp_min(1e-30)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B * T, Hq, D).to(s["out"].dtype), "lse": lse.permute(0, 2, 1, 3).reshape(B * T, Hq).contiguous()}


def work(case):
    if case["op"] == "norm":
        n, b = case["M"] * case["K"], 2 * case["K"] + 4 * case["M"] * blocks(case["K"])
        return {"bytes": n * (2 + (4 if case["add"] else 0) + (2 if case["y"] else 0) + 1) + b, "flops": 8 * n}
    if case["op"] == "gated":
        n = case["M"] * case["K"]
        return {"bytes": n * (4 + (2 if case["y"] else 0) + 1) + 4 * case["M"] * blocks(case["K"]), "flops": 10 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * M * blocks(K) + 4 * blocks(N) * blocks(K), "flops": 2 * M * N * K}
    B, T, Hq, Hkv, D, L = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "L"))
    keys = L + (B - 1) * L * 3 // 4 + B * T                   # the first request's length, the others' mean
    return {"bytes": 4 * keys * Hkv * D + 4 * B * T * Hq * D + 4 * B * T * Hq, "flops": 4 * keys * T * Hq * D}


def exact(case, seed):
    """The operators' definitions in 64 bits, before any rounding of an output to its type (an 8-bit value's is what its scale leaves of the result)."""
    s = prepare(case, seed)
    del s["work"]
    if case["op"] == "tree":
        return exact_tree(s)
    M, K = case["M"], case["K"]
    column = torch.arange(K, device="cuda") // BLOCK
    if case["op"] == "gemm":
        y, ws = torch.zeros(M, case["N"], dtype=torch.float64, device="cuda"), s["w_scales"].double()
        row = torch.arange(case["N"], device="cuda") // BLOCK
        for k in range(0, K, 16 * BLOCK):                      # a few blocks of the sum at a time
            c = column[k:k + 16 * BLOCK]
            y += (s["x"][:, k:k + 16 * BLOCK].double() * s["x_scales"].double()[c].t()) @ (s["w"][:, k:k + 16 * BLOCK].double() * ws[row][:, c]).t()
        return y
    if case["op"] == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = s["weight"].double() * h / ((h * h).sum(1, keepdim=True) / K + 1e-6).sqrt()
    else:
        gate, up = s["x"].double().split(K, 1)
        y = gate * torch.sigmoid(gate) * up
    scales = torch.stack([c.abs().amax(1).clamp_min(FLOOR) / 448 for c in y.split(BLOCK, 1)])
    got = {"y": y if case["y"] else None, "q": y / scales[column].t(), "scales": scales}
    if case["op"] == "norm":
        got["h"] = h if case["add"] else None
    return got


def exact_tree(s):
    B, T, Hq, Hkv, D = (s[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q, lens, bits = s["q"].view(B, T, Hq, D).double(), s["lens"].tolist(), s["mask"].tolist()
    for b in range(B):
        n = lens[b] + T
        see = torch.ones(T, n, dtype=torch.bool)
        see[:, lens[b]:] = torch.tensor([[bits[b][i] >> j & 1 for j in range(T)] for i in range(T)]).bool()
        hidden = ~see.cuda()
        some = see.any(1).cuda()
        k, v = (s[c][s["table"][b].long()].flatten(0, 1)[:n] for c in ("k", "v"))
        for h in range(Hq):
            a = (q[b, :, h] @ k[:, h * Hkv // Hq].double().t() * s["scale"]).masked_fill(hidden, -math.inf)
            lse[b, :, h] = torch.logsumexp(a, 1)
            o = torch.softmax(a, 1) @ v[:, h * Hkv // Hq].double()
            out[b, :, h] = torch.where(some[:, None], o, torch.zeros_like(o))
    return {"out": out.view(B * T, Hq, D), "lse": lse.view(B * T, Hq)}
