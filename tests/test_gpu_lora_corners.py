"""GPU tests of the low-rank adapters (include/lora.h) where values are not ordinary numbers, in each of the kernels:
both products in one launch, the second product by tiles, the second product by runs of rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_03_amd as L  # noqa: E402
from test_gpu_lora import Case, TYPES  # noqa: E402

FORMS = {"one launch": (3, 64, 16), "by tiles": (40, 200, 16), "by tiles, more ranks": (20, 72, 104), "by runs": (70, 72, 16), "by runs, more ranks": (600, 72, 56)}


def form():
    f = dict(v.split("=") for v in L.w4a16_last_variant().split()[1:])
    return "one launch" if f["launches"] == "1" else "by tiles" if f["run"] == "0" else "by runs"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", FORMS)
def test_an_infinite_sum_of_any_rank_is_infinite(name, dtype):
    # A rank between two multiples of 8: the zeros behind it do not meet the infinity.
    M, K, R = FORMS[name]
    c = Case(M, K, [64, 40], R, 2, dtype, "f32", "own", ids=[i % 2 for i in range(M)], ranks=[R - 3, 1], seed=5)
    c.x[1, 9] = c.x[2, 9] = float("inf")
    c.a, c.b = c.a.abs(), torch.where(c.b != 0, c.b.abs() + 0.01, c.b)
    out = c.to_gpu().call().cpu()
    assert form() == name.split(",")[0]
    assert torch.all(torch.isposinf(out[1:3])) and torch.all(torch.isfinite(out[3:])) and torch.all(torch.isfinite(out[0]))


@pytest.mark.parametrize("y", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", FORMS)
def test_a_row_without_an_adapter_is_its_base(name, y):
    M, K, R = FORMS[name]
    c = Case(M, K, [64, 40], R, 2, "bf16" if y == "f32" else y, y, "own", ids=[i % 3 - 1 for i in range(M)], seed=6)
    c.base[:, ::3] = -0.0
    c.base[:, 1::3] = 0.0
    c.base[::3, 5] = torch.finfo(TYPES[y]).smallest_normal / 4
    c.base[::3, 8] = float("-inf")
    out = c.to_gpu().call().cpu()
    assert form() == name.split(",")[0]
    bits = torch.int32 if y == "f32" else torch.int16
    assert torch.equal(out[::3].contiguous().view(bits), c.base[::3].contiguous().view(bits))
