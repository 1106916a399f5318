"""moe_add_rms_norm against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import load_binding

pytestmark = pytest.mark.gpu

FP32 = 64 * 2.0 ** -24     # sum of squares (at most 48 roundings on one path), rsqrt, two products


@pytest.fixture(scope="module")
def B():
    return load_binding()


def f64(t):
    return t.double().cpu().numpy()


def check(out, x, residual, w, eps):
    h, v = R.add_rms_norm(f64(x), None if residual is None else f64(residual), f64(w), eps)
    if "residual_out" in out:
        assert np.all(np.abs(f64(out["residual_out"]) - h) <= np.abs(h) * (2.0 ** -8 + FP32) + 2.0 ** -133)
    if "y" in out:
        assert np.all(np.abs(f64(out["y"]) - v) <= np.abs(v) * (2.0 ** -8 + FP32) + 2.0 ** -133)
    if "q" in out:
        q, s, u = R.quantise(v)
        got_s, got_q = f64(out["scales"]), out["q"].float().cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got_s - s) <= s * FP32)
        # a code is within half a step of the exact one's unrounded value
        assert np.all(np.abs(got_q - u) <= R.e4m3_step(u) * 0.5 + np.abs(u) * 2 * FP32)


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (2, 128), (3, 136), (5, 1000), (4, 2048),
                                 (7, 2056), (3, 4104), (2, 8192), (3, 8200), (2, 16384), (2, 16376),
                                 (700, 512), (2600, 264)])
@pytest.mark.parametrize("residual", [True, False])
def test_values(B, T, H, residual, w_dtype):
    g = torch.Generator(device="cuda").manual_seed(T * H)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    r = (4 * torch.randn(T, H, generator=g, device="cuda")).bfloat16() if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(w_dtype)
    out = B.add_rms_norm(x, w, residual=r, eps=1e-5)
    torch.cuda.synchronize()
    check(out, x, r, w, 1e-5)
    assert set(out) == {"y", "q", "scales"} | ({"residual_out"} if residual else set())


@pytest.mark.parametrize("keys", [("y",), ("q", "scales"), ("residual_out", "y"),
                                  ("residual_out", "q", "scales")])
def test_only_what_is_asked_for(B, keys):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(9, 328, generator=g, device="cuda").bfloat16()
    r = torch.randn(9, 328, generator=g, device="cuda").bfloat16()
    w = torch.ones(328, device="cuda")
    full = B.add_rms_norm(x, w, residual=r)
    out = {k: torch.empty_like(full[k]) for k in keys}
    B.add_rms_norm(x, w, residual=r, out=out)
    for k in keys:
        assert torch.equal(out[k].view(torch.uint8), full[k].view(torch.uint8))


def test_in_place(B):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(300, 520, generator=g, device="cuda").bfloat16()
    r = torch.randn(300, 520, generator=g, device="cuda").bfloat16()
    w = torch.randn(520, generator=g, device="cuda")
    full = B.add_rms_norm(x, w, residual=r)
    B.add_rms_norm(x, w, residual=r, out=dict(residual_out=r, y=x))
    assert torch.equal(r, full["residual_out"]) and torch.equal(x, full["y"])


def test_zero_small_and_large_rows(B):
    H = 264
    x = torch.zeros(6, H, device="cuda")
    x[1, 5] = 1.0
    x[2] = 1e-38
    x[3] = 3e18
    x[4, :128] = 0.0
    x[4, 128:] = torch.randn(H - 128, device="cuda")
    x[5] = torch.randn(H, device="cuda") * 1e-20
    x = x.bfloat16()
    w = torch.ones(H, device="cuda")
    out = B.add_rms_norm(x, w, eps=1e-6)
    torch.cuda.synchronize()
    check(out, x, None, w, 1e-6)
    assert (out["q"].float()[0] == 0).all() and (out["scales"][0] > 0).all()
    zero = B.add_rms_norm(torch.zeros(1, H, device="cuda").bfloat16(), w, eps=1e-12)
    assert (zero["y"] == 0).all()


def test_nan_stays_in_its_row(B):
    x = torch.randn(4, 512, device="cuda").bfloat16()
    clean = B.add_rms_norm(x, torch.ones(512, device="cuda"))
    x[2, 300] = float("nan")
    out = B.add_rms_norm(x, torch.ones(512, device="cuda"))
    assert torch.isnan(out["y"][2]).all() and torch.isnan(out["q"][2].float()).all()
    for t in (0, 1, 3):
        for k in out:
            assert torch.equal(out[k][t].view(torch.uint8), clean[k][t].view(torch.uint8))


def test_no_tokens(B):
    out = B.add_rms_norm(torch.empty(0, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda"))
    assert out["y"].shape == (0, 64) and out["scales"].shape == (0, 1)


def test_stores_stay_in_bounds(B):
    """Outputs between guard rows of a byte pattern."""
    for T, H in ((5, 136), (3, 8200), (1, 8)):
        g = torch.Generator(device="cuda").manual_seed(H)
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        r = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        full, out = {}, {}
        nb = R.blocks(H)
        for k, cols, dt in (("residual_out", H, torch.bfloat16), ("y", H, torch.bfloat16),
                            ("q", H, torch.uint8), ("scales", nb, torch.float32)):
            full[k] = torch.empty(T + 32, cols, dtype=dt, device="cuda")
            full[k].view(torch.uint8).fill_(0xA5)
            out[k] = full[k][16:16 + T]
        out["q"] = out["q"].view(torch.float8_e4m3fn)
        B.add_rms_norm(x, torch.ones(H, device="cuda"), residual=r, out=out)
        for k in full:
            b = full[k].view(torch.uint8)
            assert (b[:16] == 0xA5).all() and (b[16 + T:] == 0xA5).all(), k
