"""The int8 block of examples/ against its formulas in 64 bits: projection,
boundary norms, router and experts together, as a model calls them, for a few
tokens and for many, in a captured graph and on two streams."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_block.py")


@pytest.fixture(scope="module")
def ex():
    load_binding()
    spec = importlib.util.spec_from_file_location("int8_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(T, A, H, seed, masked=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, A, generator=g, device="cuda").bfloat16()
    residual = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
        mask[0] = 1
        x[mask == 0] = float("nan")           # padding holds anything
    return x, residual, mask


def rms(v, w):
    return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()


def codes(v):
    s = v.abs().amax(-1, keepdim=True) / 127
    return torch.where(s > 0, torch.round(v / s.clamp(min=1e-300)), 0.0) * s


@pytest.mark.parametrize("T,H,A,E,K,N,masked", [
    (1, 256, 512, 8, 2, 256, False),
    (9, 1040, 528, 16, 4, 512, True),
    (200, 1024, 1024, 32, 6, 512, True),
])
def test_block(ex, T, H, A, E, K, N, masked):
    raw = {}
    block = ex.random_block(H, A, E, K, N, seed=T, stages=raw)
    x, residual, mask = inputs(T, A, H, T, masked)
    st = {}
    out, nxt = block(x, residual, mask=mask, stages=st)
    torch.cuda.synchronize()
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    o = codes(x[live].double()) @ (raw["o_proj"][0].double() * block.o_scale[0].double()[:, None]).T
    h = residual[live].double() + torch.sigmoid(block.gate.double()) * rms(o, block.post_weight)
    y = rms(h, block.weight)
    ids, probs = st["routes"]["expert_ids"], st["routes"]["expert_scales"].double()
    assert (ids[~live] == -1).all()
    # the routes that the kernels made go into the reference: they may hang on a rounding
    p = torch.softmax(st["logits"][live].double(), 1).gather(1, ids[live].long())
    assert bool(((probs[live] - p / p.sum(1, keepdim=True)).abs() < 1e-5).all())
    w1 = raw["w1"].double() * block.scale1.double()[:, :, None]
    w2 = raw["w2"].double() * block.scale2.double()[:, :, None]
    q1 = codes(y)
    ref = h.clone()
    for i, t in enumerate(torch.nonzero(live)[:, 0].tolist()):
        for k in range(K):
            e = int(ids[t, k])
            a = w1[e] @ q1[i]
            q2 = codes((a[:N // 2] * torch.sigmoid(a[:N // 2]) * a[N // 2:])[None])[0]
            ref[i] += probs[t, k] * (w2[e] @ q2)
    # bf16 of the projection, both norms' sides, the experts' rows and sums (each 2^-9 rms
    # or less of a part), and the int8 codes that they move
    for got, want in ((out, ref), (nxt, rms(ref, block.next_weight))):
        got = got[live].double()
        assert (got - want).norm() <= 1e-2 * want.norm()
        assert (got - want).abs().max() <= 0.05 * want.abs().max()


def test_few_and_many_tokens_agree(ex, monkeypatch):
    """The same tokens through either layer: the same bits."""
    block = ex.random_block(512, 512, 16, 4, 512, seed=5)
    x, residual, mask = inputs(30, 512, 512, 5, True)
    few = block(x, residual, mask=mask)
    monkeypatch.setattr(ex, "FEW_ROUTES", 0)
    many = block(x, residual, mask=mask)
    live = mask != 0
    for a, b in zip(few, many):
        assert torch.equal(a[live].view(torch.int16), b[live].view(torch.int16))


@pytest.mark.parametrize("T", [1, 40, 200])
def test_captured_graph(ex, T):
    """Captured once, replayed on other inputs: the same as called."""
    block = ex.random_block(512, 512, 16, 4, 512, seed=1)
    static = inputs(T, 512, 512, 0)[:2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            block(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(*static)
    for seed in (1, 2, 3):
        new = inputs(T, 512, 512, seed)[:2]
        want = [v.clone() for v in block(*new)]
        for s, n in zip(static, new):
            s.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_two_streams(ex):
    """Many calls of the same length in flight on two streams."""
    block = ex.random_block(512, 512, 16, 4, 512, seed=2)
    args = [inputs(24, 512, 512, s)[:2] for s in range(2)]
    want = [[v.clone() for v in block(*a)] for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    busy = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(4):
                torch.mm(busy, busy)
    got = [[], []]
    for _ in range(30):
        for s, a, g in zip(streams, args, got):
            with torch.cuda.stream(s):
                g.append(block(*a))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for out in g:
            for a, b in zip(out, w):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_example_runs():
    r = subprocess.run([sys.executable, PATH, "--tokens", "130", "--hidden", "512", "--experts", "16",
                        "--topk", "4", "--ffn", "256"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("us per call") == 2
