"""moe_block_norm against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import load_binding

pytestmark = pytest.mark.gpu

FP32 = 64 * 2.0 ** -24     # sum of squares (at most 48 roundings on one path), rsqrt, two products
F1 = 2.0 ** -24            # one fp32 rounding


@pytest.fixture(scope="module")
def B():
    return load_binding()


def f64(t):
    return t.double().cpu().numpy()


def formulas(x, residual, w, post, gate, act, rs, bs, eps):
    """h, v in 64 bits and bounds of what fp32 may be off them.  rs, bs: the fp32
    numbers that the call gets."""
    x, res = f64(x), f64(residual)
    T, H = x.shape
    a = x
    rel = 0.0                                       # of the branch, relative
    if post is not None:
        a = a / np.sqrt((a * a).sum(1, keepdims=True) / H + eps) * f64(post)
        rel = rel + FP32
    if gate is not None:
        g = np.repeat(f64(gate), T // gate.shape[0], 0)
        if act == "sigmoid":
            # the exponential's argument is rounded once (|g| 2^-24 of the result), exponential,
            # sum and reciprocal are within two units in the last place each
            rel = rel + (np.abs(g) + 2 * 2 * 2 + 1) * F1
            g = 1 / (1 + np.exp(-g))
        a = a * g
        rel = rel + F1
    branch, kept = bs * a, rs * res
    h = kept + branch
    dh = np.abs(branch) * (rel + 2 * F1) + np.abs(kept) * 2 * F1 + np.abs(h) * F1
    if w is None:
        return h, dh, None, None
    n2 = (h * h).sum(1, keepdims=True)
    r = 1 / np.sqrt(n2 / H + eps)
    v = h * r * f64(w)
    # the factor moves by at most the share of the row that dh is
    share = np.sqrt((dh * dh).sum(1, keepdims=True) / np.maximum(n2 + eps * H, 1e-300))
    dv = np.abs(f64(w)) * r * dh * (1 + FP32) + np.abs(v) * (FP32 + share)
    return h, dh, v, dv


def check(out, ref):
    h, dh, v, dv = ref
    tiny = 2.0 ** -133
    assert np.all(np.abs(f64(out["residual_out"]) - h) <= (np.abs(h) + dh) * 2.0 ** -8 + dh + tiny)
    if "y" in out:
        assert np.all(np.abs(f64(out["y"]) - v) <= (np.abs(v) + dv) * 2.0 ** -8 + dv + tiny)
    if "q" in out:
        q, s, u = R.quantise(v)
        nb = s.shape[1]
        wide = np.zeros((v.shape[0], nb * 128))
        wide[:, :v.shape[1]] = dv
        ds = wide.reshape(v.shape[0], nb, 128).max(2) / 448 + s * 4 * F1
        got_s, got_q = f64(out["scales"]), out["q"].float().cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got_s - s) <= ds)
        cols = np.arange(v.shape[1]) // 128
        du = dv / s[:, cols] + np.abs(u) * (ds / s)[:, cols] + np.abs(u) * 4 * F1
        # a code is within half a step of the exact one's unrounded value
        assert np.all(np.abs(got_q - u) <= R.e4m3_step(np.abs(u) + du) * 0.5 + du)


def make(T, H, gates, post, dtype, seed=0, stride=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    gate = None
    if gates:
        gate = randn(gates, stride or H).bfloat16()[:, :H] * 2
        if stride:
            buf = torch.zeros(gates, stride, device="cuda").bfloat16()
            buf[:, :H] = gate
            gate = buf[:, :H]
    return dict(x=(3 * randn(T, H)).bfloat16(), residual=(4 * randn(T, H)).bfloat16(),
                weight=(1 + 0.3 * randn(H)).to(dtype),
                post_weight=(1 + 0.3 * randn(H)).to(dtype) if post else None, gate=gate)


RS, BS = float(np.float32(0.9)), float(np.float32(0.4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T,H,gates,act", [
    (1, 8, 0, "none"), (1, 7168, 1, "none"), (2, 128, 2, "sigmoid"), (3, 136, 1, "sigmoid"),
    (6, 1000, 3, "none"), (4, 2048, 4, "none"), (7, 2056, 0, "none"), (7, 2056, 0, "sigmoid"), (3, 4104, 1, "none"),
    (4, 8192, 2, "sigmoid"), (3, 8200, 3, "none"), (2, 16384, 2, "sigmoid"), (500, 16376, 500, "none"),
    (700, 512, 7, "none"), (2600, 264, 2600, "sigmoid"), (2000, 7168, 1, "sigmoid")])
def test_values(B, T, H, gates, act, post, dtype):
    d = make(T, H, gates, post, dtype, seed=T + H)
    out = B.block_norm(**d, gate_act=act, residual_scale=0.9, branch_scale=0.4, eps=1e-5)
    torch.cuda.synchronize()
    assert set(out) == {"residual_out", "y", "q", "scales"}
    eps = float(np.float32(1e-5))
    check(out, formulas(d["x"], d["residual"], d["weight"], d["post_weight"], d["gate"], act, RS, BS, eps))


def test_strided_gate(B):
    """A gate that is a slice of a wider projection."""
    for T, H, gates, stride in ((12, 264, 4, 6 * 264), (5, 520, 5, 528), (3, 64, 1, 128)):
        d = make(T, H, gates, True, torch.bfloat16, stride=stride)
        whole = dict(d, gate=d["gate"].contiguous())
        a, b = B.block_norm(**d), B.block_norm(**whole)
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


def test_is_the_residual_norm_without_gate_and_post_norm(B):
    """Factors of 1 and nothing else: add_rms_norm's results."""
    d = make(33, 1032, 0, False, torch.float32)
    a = B.block_norm(**d, eps=1e-6)
    b = B.add_rms_norm(d["x"], d["weight"], residual=d["residual"], eps=1e-6)
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("keys", [(), ("y",), ("q", "scales")])
def test_only_what_is_asked_for(B, keys):
    d = make(9, 328, 3, True, torch.float32)
    full = B.block_norm(**d)
    out = {k: torch.empty_like(full[k]) for k in ("residual_out",) + keys}
    B.block_norm(**d, out=out)
    for k in out:
        assert torch.equal(out[k].view(torch.uint8), full[k].view(torch.uint8))
    alone = B.block_norm(**dict(d, weight=None))
    assert set(alone) == {"residual_out"}
    assert torch.equal(alone["residual_out"], full["residual_out"])


def test_in_place(B):
    d = make(900, 520, 900, True, torch.float32)
    full = B.block_norm(**d)
    B.block_norm(**d, out=dict(residual_out=d["residual"], y=d["x"]))
    assert torch.equal(d["residual"], full["residual_out"]) and torch.equal(d["x"], full["y"])


def test_zero_small_and_large_rows(B):
    H = 264
    x = torch.zeros(6, H, device="cuda")
    res = torch.zeros(6, H, device="cuda")
    x[1, 5] = 1.0
    x[2] = 1e-30
    x[3] = 3e18                       # squares past fp32's range, before both norms
    res[3] = 2e18
    x[4, 128:] = torch.randn(H - 128, device="cuda")
    res[5] = torch.randn(H, device="cuda") * 1e-20
    d = dict(x=x.bfloat16(), residual=res.bfloat16(), weight=torch.ones(H, device="cuda"),
             post_weight=torch.full((H,), 2.0, device="cuda"))
    eps = float(np.float32(1e-6))
    for post in (True, False):
        e = d if post else dict(d, post_weight=None)
        out = B.block_norm(**e, eps=1e-6)
        torch.cuda.synchronize()
        check(out, formulas(d["x"], d["residual"], d["weight"], e["post_weight"], None, "none", 1.0, 1.0, eps))
        assert (out["q"].float()[0] == 0).all() and (out["scales"][0] > 0).all()


def test_nan_and_infinity_stay_in_their_rows(B):
    d = make(5, 512, 5, True, torch.float32)
    clean = B.block_norm(**d)
    d["x"][2, 300] = float("nan")
    d["gate"][3, 7] = float("inf")
    out = B.block_norm(**d)
    assert torch.isnan(out["y"][2]).all() and torch.isinf(out["residual_out"][3, 7])
    for t in (0, 1, 4):
        for k in out:
            assert torch.equal(out[k][t].view(torch.uint8), clean[k][t].view(torch.uint8))


def test_no_tokens(B):
    e = torch.empty(0, 64, device="cuda").bfloat16()
    out = B.block_norm(e, e, torch.ones(64, device="cuda"), gate=e)
    assert out["y"].shape == (0, 64) and out["scales"].shape == (0, 1)


def test_stores_stay_in_bounds(B):
    """Outputs between guard rows of a byte pattern."""
    for T, H in ((5, 136), (3, 8200), (1, 8)):
        d = make(T, H, T, True, torch.float32)
        full, out = {}, {}
        for k, cols, dt in (("residual_out", H, torch.bfloat16), ("y", H, torch.bfloat16),
                            ("q", H, torch.uint8), ("scales", R.blocks(H), torch.float32)):
            full[k] = torch.empty(T + 32, cols, dtype=dt, device="cuda")
            full[k].view(torch.uint8).fill_(0xA5)
            out[k] = full[k][16:16 + T]
        out["q"] = out["q"].view(torch.float8_e4m3fn)
        B.block_norm(**d, out=out)
        for k in full:
            b = full[k].view(torch.uint8)
            assert (b[:16] == 0xA5).all() and (b[16 + T:] == 0xA5).all(), k
