"""moe_grouped_gemm_int8 on bf16 rows with an infinity: no scale fits such a row (its own
quotients are not numbers), so its outputs are NaN, and no other row's change."""
import pytest
import torch

from test_gpu_int8 import B, make  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("values", [(INF,), (-INF,), (INF, -INF, float("nan"))], ids=str)
@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
def test_infinity_makes_its_row_nan(B, path, values):  # noqa: F811
    # the stream quantising by itself and behind a kernel, split tiles, whole tiles and the large ones
    for rows, E, N, Kd in ((1, 1, 264, 528), (2, 1, 264, 528), (20, 1, 264, 528), (130, 1, 1000, 5008),
                           (300, 1, 264, 528), (400, 3, 4104, 528)):
        d = make(rows, E, N, Kd, a="bf16", bias=True)
        d["w"][:, ::3] = 0                  # a weight of zero does not hide it
        _, packed = B.pack_int8(d["w"], path=path)
        clean, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], bias=d["bias"], path=path)
        hit = rows // 2
        for i, v in enumerate(values):
            d["a"][hit, 100 * i + 7] = v
        got, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], bias=d["bias"], path=path)
        rest = [r for r in range(rows) if r != hit]
        assert B.read_device_status(ws) == 0
        assert bool(torch.isnan(got[hit]).all())
        assert torch.equal(got[rest], clean[rest])


def test_the_largest_numbers_are_still_quantised(B):  # noqa: F811
    """The largest bf16 number is no infinity."""
    big = torch.finfo(torch.bfloat16).max
    for rows in (2, 20, 130):
        d = make(rows, 1, 1000, 5008, a="bf16")
        d["a"][1, 5] = -big
        d["ws"].fill_(1e-8)
        _, packed = B.pack_int8(d["w"], path="small")
        got, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path="small", out_dtype=torch.float32)
        scale = torch.tensor(big, device="cuda") / torch.full((), 127.0, device="cuda")
        want = ((-127.0 * d["w"][0, :, 5].float()) * 1e-8) * scale
        assert torch.equal(got[1], want)
