"""GPU tests of the forms of the attention behind a shared prefix (include/prefix_attn.h) against its definition in 64 bits:
which one is taken, replays with other lengths, and a workspace that a larger batch left."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402
from test_gpu_prefix_attn import DEV, Case  # noqa: E402


def splits():
    """Parts of the prefix (0: each request reads it) and of the own keys."""
    return tuple(int(f.split("=")[1]) for f in L.w4a16_last_variant().split()[2:4])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,P,shared", [(6, 7, 8, 2, 682, False), (6, 7, 8, 2, 10000, True), (44, 1, 10, 2, 690, False), (44, 1, 10, 2, 1522, True)])
def test_heads_of_256_share_a_long_prefix_alone(B, T, Hq, Hkv, P, shared, dtype):
    c = Case(B, T, Hq, Hkv, 256, 32, dtype, P, [(100, 0, 64, 33)[i % 4] for i in range(B)], seed=P)
    out, lse = c.run()
    assert (splits()[0] > 0) == shared, L.w4a16_last_variant()
    c.check(out, lse, [0, 1, 2, 3] if P < 5000 else [1, 2])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,shared", [(32, False), (6000, True)])
def test_a_prefix_of_one_tile_is_not_shared(D, P, shared):
    c = Case(64, 1, 4, 4, D, 16, "bf16", 32, [i % 40 for i in range(64)], seed=D)
    c.ptable = torch.cat([c.ptable, torch.zeros(400, dtype=torch.int32)])
    out, lse = c.run(max_prefix=P)
    assert (splits()[0] > 0) == shared, L.w4a16_last_variant()
    c.check(out, lse, [0, 1, 31, 33, 39])


# Bounds on the lengths: each request reads the prefix; shared, in parts; own keys in parts.
FORMS = {"each": (70, 200), "shared": (4000, 200), "parts": (40, 3000)}


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("name", FORMS)
def test_replays_with_other_lengths(name, D, dtype):
    # Every request has keys and values up to its bound; a replay takes some of them, its drafts behind those.
    P, longest = FORMS[name]
    B, T, Hq, Hkv = (40, 2, 4, 2) if name == "shared" else (5, 2, 4, 2)
    c = Case(B, T, Hq, Hkv, D, 16, dtype, P, [longest] * B, seed=D)
    whole_prefix, whole = c.prefix, c.dense
    need = L.prefix_attn_workspace_bytes(B, T, Hq, Hkv, D, P, longest)
    work = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)
    c.run(work=work)
    torch.cuda.synchronize()
    sp, so = splits()
    assert {"each": sp == 0 and so == 1, "shared": sp > 0, "parts": so > 1}[name], (sp, so)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run(work=work)
    some = [0, 1, 2, 3, B - 1]
    for plen, lens in ((P, [longest, 10, 0, 33, 199]), (0, [0, 1, 150, 32, 64]), (P - 33, [5, longest, 31, 0, longest - 1]), (1, [0] * 5)):
        c.P, c.lens = plen, torch.tensor([lens[i % 5] for i in range(B)], dtype=torch.int32)
        c.prefix = [t[:plen] for t in whole_prefix]
        c.dense = [[t[:int(n) + T] for t in whole[b]] for b, n in enumerate(c.lens)]
        c.g["lens"].copy_(c.lens)
        c.g["plen"].fill_(plen)
        out.fill_(9.0)
        lse.fill_(9.0)
        work.fill_(255)                                      # NaN: nothing is kept from one replay for the next
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, some)


def test_a_batch_that_shrinks_keeps_its_workspace():
    # The largest batch's workspace serves every smaller one, and nothing is written behind it.
    T, Hq, Hkv, D, P, n, most = 1, 40, 8, 128, 700, 500, 24
    need = L.prefix_attn_workspace_bytes(most, T, Hq, Hkv, D, P, n)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    room[need:] = 77
    c = Case(most, T, Hq, Hkv, D, 32, "bf16", P, [(n, 0, 33, 490)[i % 4] for i in range(most)], seed=1)
    whole = c.mask
    for B in (24, 17, 9, 5, 2, 1):
        c.B, c.mask, c.lens = B, np.ascontiguousarray(whole[:B]), c.lens[:B]
        for P_, n_ in ((P, n), (P // 3, n)):
            c.P, room[:need] = P_, 255
            c.to_gpu()
            c.g["work"] = room[:need]
            out, lse = c.run(max_len=n_, max_prefix=P_, work=c.g["work"])
            c.check(out, lse, [0, B - 1])
            assert torch.all(room[need:] == 77)
