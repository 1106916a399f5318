"""The fp8 MoE block of examples/ against 64 bits: norm, router, dispatch,
experts and combine together, as a model calls them."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import load_binding

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "fp8_moe_block.py")


@pytest.fixture(scope="module")
def ex():
    load_binding()
    spec = importlib.util.spec_from_file_location("fp8_moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.double().cpu().numpy()


def weights64(q, s):
    return f64(q.float()) * R.expand(R.expand(f64(s), q.shape[1], 1), q.shape[2], 2)


@pytest.mark.parametrize("T,H,E,K,N,groups,topk_groups,masked", [
    (1, 256, 8, 2, 256, 1, 1, False),
    (37, 400, 16, 4, 512, 4, 2, True),
    (200, 1024, 32, 6, 256, 8, 3, False),
])
def test_block(ex, T, H, E, K, N, groups, topk_groups, masked):
    block = ex.random_block(H, E, K, N, groups, topk_groups, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    residual = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
        x[mask == 0] = float("nan")           # padding holds anything
    st = {}
    out = block(x, residual, mask=mask, stages=st)
    torch.cuda.synchronize()
    live = np.ones(T, bool) if mask is None else mask.cpu().numpy() != 0

    h, v = R.add_rms_norm(f64(x)[live], f64(residual)[live], f64(block.norm_weight), 1e-6)
    q, s, _ = R.quantise(v)
    ids = st["routes"]["expert_ids"].cpu().numpy()
    assert (ids[~live] == -1).all()
    key, score, _ = R.gate_keys(f64(st["logits"]), f64(block.bias), None if mask is None else mask.cpu().numpy(),
                                "sigmoid", groups, topk_groups, "top2")
    # the chosen experts' keys are the largest ones (equal to within fp32's rounding of a score)
    want = -np.sort(-key, axis=1)[live, :K]
    got = np.take_along_axis(key, np.maximum(ids, 0), 1)[live]
    assert np.all(np.abs(got - want) <= 4e-6)
    w1, w2 = weights64(block.w1, block.w1_scales), weights64(block.w2, block.w2_scales)
    ref = h.copy()
    rows = q * R.expand(s, H, 1)
    wsum = np.take_along_axis(score, np.maximum(ids, 0), 1)[live]
    w = wsum / (wsum.sum(1, keepdims=True) + 1e-20) * 2.5
    for i, t in enumerate(np.flatnonzero(live)):
        for k in range(K):
            e = ids[t, k]
            y, _ = R.ffn(rows[i:i + 1], np.array([0, 1]), w1[e:e + 1], w2[e:e + 1])
            ref[i] += w[i, k] * y[0]
    got = f64(out)[live]
    # bf16 of y, of the residual and of the sum (2^-9 rms each), codes that
    # rounded the other way
    assert np.linalg.norm(got - ref) <= 6e-3 * np.linalg.norm(ref)
    assert np.abs(got - ref).max() <= 0.05 * np.abs(ref).max()


def test_example_runs():
    r = subprocess.run([sys.executable, PATH, "--tokens", "5", "--hidden", "512", "--experts", "16",
                        "--topk", "4", "--ffn", "256"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us per call" in r.stdout
