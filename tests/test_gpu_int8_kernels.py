"""Which kernels moe_grouped_gemm_int8's calls launch.  The ways are chosen by estimates
of time, so that the tests of a kernel could come to run another one unnoticed."""
import pytest
import torch

from test_gpu_int8 import KERNELS, TILES, B, make, reference  # noqa: F401

pytestmark = pytest.mark.gpu


def launches(B, d, path):  # noqa: F811
    """{kernel: CTAs} of one call."""
    _, packed = B.pack_int8(d["w"], path=path)
    B.profile_enable(True)
    try:
        B.profile_report()
        out, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], path=path)
        torch.cuda.synchronize()
        B.profile_report()
        grids = dict(B.LAST_GRIDS)
    finally:
        B.profile_enable(False)
    want = reference(d, torch.bfloat16)[0]
    assert torch.equal(out[:want.shape[0]], want)
    return grids


@pytest.mark.parametrize("kw,path,kernels", [
    (dict(rows=1, E=1, N=4096, Kd=7168, a="bf16"), "auto", {"int8_few"}),
    (dict(rows=1, E=1, N=4096, Kd=7168), "auto", {"int8_few"}),
    (dict(rows=16, E=1, N=4096, Kd=7168, a="bf16"), "auto", {"quant_rows_i8", "int8_few"}),
    (dict(rows=16, E=1, N=4096, Kd=7168), "auto", {"int8_few"}),
    (dict(rows=60, E=3, N=5000, Kd=400), "small", {"int8_tiles"}),
    (dict(rows=60, E=3, N=5000, Kd=400, a="bf16"), "small", {"rows_to_f16", "int8_tiles"}),
    (dict(rows=640, E=32, N=2048, Kd=2048), "auto", {"rows_to_f16", "gemm_linear_small"}),
    (dict(rows=512, E=1, N=7168, Kd=2048, a="bf16"), "auto", {"rows_to_f16", "gemm_linear_small"}),
    (dict(rows=2048, E=1, N=7168, Kd=2048, a="bf16"), "auto", {"rows_to_f16", "gemm_linear_pair"}),
    (dict(rows=9, E=1, N=520, Kd=528), "large", {"rows_to_f16", "gemm_linear"}),
    (dict(rows=9, E=1, N=520, Kd=528), "large_pair", {"rows_to_f16", "gemm_linear_pair"}),
], ids=lambda v: "-".join(f"{k}{x}" for k, x in v.items()) if isinstance(v, dict) else "")
def test_kernels_of_a_call(B, kw, path, kernels):  # noqa: F811
    assert set(launches(B, make(**kw), path)) == kernels


@pytest.mark.parametrize("kw,tile", [
    (dict(rows=64, E=1, N=7168, Kd=2048), 64), (dict(rows=64, E=1, N=4096, Kd=7168), 64),
    (dict(rows=37, E=1, N=1000, Kd=7184), 64), (dict(rows=128, E=1, N=4096, Kd=7168), 128),
    (dict(rows=127, E=1, N=1024, Kd=8192), 128),
], ids=lambda v: "-".join(f"{k}{x}" for k, x in v.items()) if isinstance(v, dict) else str(v))
def test_ctas_that_share_a_tile(B, kw, tile):  # noqa: F811
    """The calls that the tests of split tiles make have two CTAs a tile at least."""
    tiles = -(-kw["rows"] // tile) * -(-kw["N"] // 128)
    for a in ("int8", "bf16"):
        grids = launches(B, make(a=a, **kw), "small")
        assert set(grids) == {"int8_tiles"} | ({"rows_to_f16"} if a == "bf16" or tile == 128 else set())
        assert grids["int8_tiles"] >= 2 * tiles


def test_lists_of_the_tile_kernels_reach_them(B):  # noqa: F811
    """Among the calls that stand for the tile kernels are some of each, split and whole."""
    seen, split = [], 0
    for kw in KERNELS + [{k: v for k, v in c.items() if k != "bias"} for c in TILES]:
        d = make(**kw)
        grids = launches(B, d, "small")
        seen.append(frozenset(grids))
        tiles = sum(-(-n // 64) for n in torch.diff(d["off"].cpu()).tolist()) * -(-kw["N"] // 128)
        split += grids.get("int8_tiles", 0) > tiles
    assert sum(s == {"int8_tiles"} for s in seen) >= 4                  # int8 rows in tiles of 64
    assert sum(s == {"rows_to_f16", "int8_tiles"} for s in seen) >= 3   # images: tiles of 128, bf16 rows
    assert sum("gemm_linear_small" in s for s in seen) >= 2
    assert split >= 4
