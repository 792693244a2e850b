"""GPU tests of the attention behind a shared prefix (include/prefix_attn.h) where values are not ordinary numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402
from test_gpu_prefix_attn import Case, UT  # noqa: E402

INF = float("inf")


def check_form(name):
    # parts of the prefix, 0: each request reads it; parts of the own keys
    sp, so = (int(f.split("=")[1]) for f in L.w4a16_last_variant().split()[2:4])
    assert {"each": sp == 0 and so == 1, "shared": sp > 0, "parts": so > 1}[name], (sp, so)


def case(D, dtype, P, lens, seed=0):
    c = Case(len(lens), 3, 4, 2, D, 16, dtype, P, lens, seed=seed)
    c.ptable = torch.cat([c.ptable, torch.zeros(400, dtype=torch.int32)])
    return c


# How the keys are divided: every request reads the prefix, one part; shared; own keys in parts.
SHAPES = {"each": (40, 40, [70, 0, 45]), "shared": (300, 5000, [70, 0, 45] * 14), "parts": (20, 20, [4000, 100, 9])}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", SHAPES)
def test_an_infinite_value_counts_however_small_its_probability(name, D, dtype):
    P, max_prefix, lens = SHAPES[name]

    def make():
        c = case(D, dtype, P, lens, seed=D)
        c.q.abs_().add_(0.5)
        for k in [c.prefix[0]] + [d[0] for d in c.dense]:          # the keys that will hold infinities: probabilities far below the least number
            k[3::8] = -60.0
        c.store()
        return c
    want, want_lse = make().run(max_prefix=max_prefix)
    check_form(name)
    c = make()
    # the prefix: +inf, -inf, both, NaN
    v = c.prefix[1]
    v[3, :, 5], v[11, :, 6] = INF, -INF
    v[3, :, 7], v[11, :, 7] = INF, -INF
    v[11, :, 8] = float("nan")
    # the first request's own context, each of its tiles' kinds (a whole one, one that ends with drafts)
    own = c.dense[0][1]
    own[11, :, 20], own[(lens[0] - 4) // 8 * 8 + 3, :, 21] = -INF, INF
    own[3, :, 5] = INF
    c.store()
    got, lse = c.run(max_prefix=max_prefix)
    shape = (c.B, c.T, c.Hq, D)
    g, w = got.view(shape).cpu().float(), want.view(shape).cpu().float()
    assert torch.all(torch.isposinf(g[..., 5])) and torch.all(torch.isneginf(g[..., 6]))
    assert torch.all(torch.isnan(g[..., 7])) and torch.all(torch.isnan(g[..., 8]))
    assert torch.all(torch.isneginf(g[0, ..., 20])) and torch.all(torch.isposinf(g[0, ..., 21]))
    g[..., 5:9] = w[..., 5:9]
    g[0, ..., 20:22] = w[0, ..., 20:22]
    assert torch.equal(g, w) and torch.equal(lse.cpu(), want_lse.cpu())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", SHAPES)
def test_a_draft_s_infinity_beside_a_far_larger_score(name, dtype):
    # A draft whose probability is below the least number, in a part or a wave of its own: seen by its own row alone.
    P, max_prefix, lens = SHAPES[name]
    c = case(128, dtype, P, lens, seed=3)
    c.q.abs_().add_(0.5)
    c.mask[:] = [1, 2, 4]
    for d in c.dense:
        d[0][-2] = -60.0
    c.store()
    want, _ = c.run(max_prefix=max_prefix)
    check_form(name)
    for d in c.dense:
        d[1][-2, :, 9] = -INF
    c.store()
    got, _ = c.to_gpu().run(max_prefix=max_prefix)
    g, w = (t.view(c.B, 3, 4, 128).cpu().float() for t in (got, want))
    assert torch.all(torch.isneginf(g[:, 1, :, 9]))
    g[:, 1, :, 9] = w[:, 1, :, 9]
    assert torch.equal(g, w)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", SHAPES)
def test_scores_whose_spacing_in_32_bits_is_large(name, D, dtype, sign):
    # Sums that are exact in 32 bits, multiples of 2^23 (f16) or 2^40 about 2^29 or 2^50: whatever the rounding of a score, the
    # largest takes all, and equal ones share.  out: the mean of the values at the largest scores, whose sum is fp32 and
    # which is rounded once (probabilities are 1); lse: the largest score, to two roundings and its factor's.
    P, max_prefix, lens = SHAPES[name]
    c = case(D, dtype, P, lens, seed=D + 1)
    top = 14 if dtype == "f16" else 20
    g = torch.Generator().manual_seed(7)
    c.scale = float(sign)
    c.q[:] = 2.0 ** top
    for k in [c.prefix[0]] + [d[0] for d in c.dense]:
        k.zero_()
        k[..., 0] = torch.randint(-40, 41, k.shape[:2], generator=g).to(k.dtype) * 2.0 ** (9 if dtype == "f16" else top)
        k[..., 1] = -(2.0 ** (15 if dtype == "f16" else 30))          # all scores far below zero, or far above
    c.store()
    out, lse = c.run(max_prefix=max_prefix)
    check_form(name)
    out, lse = out.view(c.B, c.T, c.Hq, D).cpu().double(), lse.view(c.B, c.T, c.Hq).cpu().double()
    for b in range(c.B):
        here = int(c.lens[b])
        k, v = (torch.cat([c.prefix[i], c.dense[b][i]]).double() for i in range(2))
        for i in range(c.T):
            see = torch.ones(P + here + c.T, dtype=torch.bool)
            see[P + here:] = torch.tensor([bool(int(c.mask[b, i]) >> j & 1) for j in range(c.T)])
            for h in range(c.Hq):
                a = (k[see, h // 2] @ c.q[b * c.T + i, h * D:(h + 1) * D].double()) * sign
                at = a == a.max()
                want = v[see, h // 2][at].mean(0)
                tol = 2 * UT[dtype] * v[see, h // 2][at].abs().mean(0) + 2.0 ** -24
                assert torch.all((out[b, i, h] - want).abs() <= tol), (L.w4a16_last_variant(), b, i, h)
                assert abs(lse[b, i, h] - a.max()) <= 2.0 ** -21 * a.max().abs()
