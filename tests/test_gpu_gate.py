"""moe_gate against the formulas in 64 bits: scores, bias, groups, ties, closed
experts, inactive tokens, strides, one token to many."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import dev, load_binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    return load_binding()


def run(B, logits, K, **kw):
    kw = dict(score="sigmoid", groups=1, topk_groups=1, group_score="max", renormalize=True,
              scale=1.0, bias=None, mask=None) | kw
    ref = R.gate(logits.float().cpu().numpy().astype(np.float64),
                 None if kw["bias"] is None else kw["bias"].cpu().numpy().astype(np.float64),
                 None if kw["mask"] is None else kw["mask"].cpu().numpy(), K, kw["score"],
                 kw["groups"], kw["topk_groups"], kw["group_score"], kw["renormalize"], kw["scale"])
    out = B.gate(logits, K, **kw)
    torch.cuda.synchronize()
    return out, ref


def check(out, ref, span=0.0):
    """ids and mask equal; weights within 2^-24 of their size per rounding: the
    exp's argument (as large as `span`), exp 2, the sum and its reciprocal 12,
    the products 3."""
    ids, w, on = ref
    np.testing.assert_array_equal(out["expert_ids"].cpu().numpy(), ids)
    np.testing.assert_array_equal(out["route_mask"].cpu().numpy(), on)
    got = out["expert_scales"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w) <= np.abs(w) * (span + 18) * 2.0 ** -24 + 2.0 ** -126)


def logits_without_near_ties(T, E, K, seed, dtype, bias, **kw):
    g = np.random.default_rng(seed)
    out = np.empty((T, E), np.float32)
    todo = np.arange(T)
    while todo.size:
        l = torch.from_numpy(g.normal(0, 1.5, (todo.size, E)).astype(np.float32)).to(dtype)
        out[todo] = l.float().numpy()
        key, _, gv = R.gate_keys(out[todo].astype(np.float64), bias, None, kw["score"],
                                 kw["groups"], kw["topk_groups"], kw["group_score"])
        bad = R.near_ties(-np.sort(-key, axis=1)[:, :K + 1])
        if gv is not None:
            bad |= R.near_ties(-np.sort(-gv, axis=1)[:, :kw["topk_groups"] + 1])
        todo = todo[bad]
    return torch.from_numpy(out).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K,groups,topk_groups,group_score,bias", [
    (1, 256, 8, 8, 4, "top2", True),
    (1, 1, 1, 1, 1, "max", False),
    (3, 5, 5, 1, 1, "max", True),             # every expert chosen
    (17, 31, 3, 1, 1, "max", False),
    (33, 33, 16, 3, 2, "top2", True),
    (65, 64, 6, 8, 3, "max", False),
    (200, 160, 6, 8, 3, "max", False),
    (129, 72, 7, 9, 1, "top2", True),         # the K experts from one group
    (64, 1000, 16, 20, 7, "max", True),
    (64, 1024, 8, 1024, 9, "top2", False),    # groups of one expert
    (40, 1024, 16, 512, 100, "top2", True),
    (1000, 128, 8, 1, 1, "max", True),
    (2500, 256, 8, 8, 4, "top2", True),
    (700, 96, 8, 4, 4, "top2", False),        # every group stays
    (500, 384, 8, 1, 1, "max", True),
    (300, 512, 12, 16, 4, "top2", True),      # 32 neighbours in a group
    (300, 128, 4, 16, 5, "max", True),        # groups of 8
    (300, 40, 4, 20, 5, "top2", False),       # groups of 2
])
def test_choice_and_weights(B, T, E, K, groups, topk_groups, group_score, bias, score, dtype):
    g = np.random.default_rng(E * 1000 + T)
    b = (0.2 * g.normal(size=E)).astype(np.float32) if bias else None
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score)
    l = logits_without_near_ties(T, E, K, T + E, dtype, None if b is None else b.astype(np.float64), **kw)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        out, ref = run(B, l, K, bias=dev(b), renormalize=renorm, scale=scale, **kw)
        check(out, ref, span=24.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("E,K,groups,topk_groups,group_score", [
    (1000, 16, 20, 7, "top2"),                # groups that begin and end inside the lanes' runs
    (660, 5, 20, 3, "top2"),                  # the last lanes without experts
    (999, 16, 3, 1, "max"),                   # a group over eleven lanes; rows not 16-byte aligned
    (900, 12, 30, 6, "top2"),                 # runs of 30
    (800, 10, 100, 4, "top2"),                # groups shorter than a run
    (513, 16, 1, 1, "max"),
    (1024, 3, 16, 2, "max"),
])
def test_many_experts_and_masked_tokens(B, E, K, groups, topk_groups, group_score, score, bias, dtype):
    T = 90
    g = np.random.default_rng(E + groups)
    b = (0.2 * g.normal(size=E)).astype(np.float32) if bias else None
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score)
    l = logits_without_near_ties(T, E, K, E, dtype, None if b is None else b.astype(np.float64), **kw)
    m = (g.random(T) < 0.7).astype(np.uint8)
    l[torch.from_numpy(m == 0).cuda()] = float("nan")
    out, ref = run(B, l, K, bias=dev(b), mask=dev(m), **kw)
    check(out, ref, span=24.0)


@pytest.mark.parametrize("E,groups,topk_groups", [(64, 1, 1), (256, 8, 3), (512, 1, 1), (1000, 20, 4)])
def test_zeros_of_both_signs_are_equal(B, E, groups, topk_groups):
    """Many equal keys, 0 and -0 among them, in the order of the experts."""
    g = np.random.default_rng(E)
    l = g.choice(np.float32([-0.0, 0.0, 0.0, -1.0]), (200, E))
    l[100:] = g.choice(np.float32([-3.0, -2.0, -1.0]), (100, E))
    l[100:, g.permutation(E)[:6]] = g.choice(np.float32([-0.0, 0.0]), (100, 6))
    for score in ("softmax", "sigmoid"):
        out, ref = run(B, dev(l), 8, score=score, groups=groups, topk_groups=topk_groups)
        check(out, ref)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,topk_groups,group_score", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_ties_go_to_the_lowest_index(B, score, groups, topk_groups, group_score):
    g = np.random.default_rng(0)
    l = torch.from_numpy(g.integers(0, 3, (300, 64)).astype(np.float32)).cuda()   # three values only
    out, ref = run(B, l, 9, score=score, groups=groups, topk_groups=topk_groups,
                   group_score=group_score)
    check(out, ref)
    out, ref = run(B, torch.zeros(5, 64, device="cuda"), 9, score=score, groups=groups,
                   topk_groups=topk_groups, group_score=group_score)
    check(out, ref)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_closed_experts_and_empty_rows(B, score, groups, topk_groups):
    """-inf, NaN and the types' lowest values close an expert; a row of nothing
    else, and a row with fewer open experts than K, leave routes over."""
    g = np.random.default_rng(3)
    E, K, T = 32, 6, 64
    low = [-np.inf, np.nan, np.finfo(np.float32).min, float(torch.finfo(torch.bfloat16).min)]
    l = g.integers(-8, 8, (T, E)).astype(np.float32) / 2
    closed = g.random((T, E)) < np.linspace(0, 1, T)[:, None]
    l[closed] = g.choice(low, closed.sum())
    bias = (g.integers(0, 4, E) / 4).astype(np.float32)        # lifts a score of 0 above open ones
    out, ref = run(B, dev(l), K, score=score, groups=groups, topk_groups=topk_groups,
                   group_score="top2", bias=dev(bias))
    assert (ref[0][-1] == -1).all() and (ref[0] == -1).any(1).sum() > 4
    check(out, ref, span=16.0)
    assert not torch.isnan(out["expert_scales"]).any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_infinite_and_extreme_logits(B, score):
    l = torch.zeros(4, 40, device="cuda")
    l[0, 7] = float("inf")
    l[0, 21] = float("inf")
    l[1, 3] = 3e38
    l[2] = -1e29
    l[3] = torch.arange(40, device="cuda") * 100.0 - 2000.0
    out, ref = run(B, l, 4, score=score)
    ids = out["expert_ids"].cpu().numpy()
    if score == "softmax":
        np.testing.assert_array_equal(ids[0, :2], [7, 21])
        np.testing.assert_allclose(out["expert_scales"][0].cpu().numpy(), [0.5, 0.5, 0, 0], atol=1e-7)
        np.testing.assert_array_equal(ids[3, 0], 39)
    assert torch.isfinite(out["expert_scales"]).all()
    np.testing.assert_array_equal(ids[2], [0, 1, 2, 3])        # open, all equal


def test_inactive_tokens_and_nan_padding(B):
    g = np.random.default_rng(5)
    l = g.integers(-6, 6, (50, 24)).astype(np.float32)
    m = (g.random(50) < 0.6).astype(np.uint8)
    m[7] = 255
    l[m == 0] = np.nan
    for score in ("softmax", "sigmoid"):
        out, ref = run(B, dev(l), 4, mask=dev(m), score=score)
        check(out, ref, span=12.0)
        assert (out["expert_ids"].cpu().numpy()[m == 0] == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_unaligned_logits(B, dtype):
    """A column slice of a wider matrix, starting at an odd element."""
    g = torch.Generator().manual_seed(1)
    wide = torch.randint(-20, 20, (70, 205), generator=g).to(dtype).cuda()
    part = wide[:, 3:3 + 128]
    out = B.gate(part, 8, score="sigmoid", groups=8, topk_groups=2, group_score="top2")
    same = B.gate(part.contiguous(), 8, score="sigmoid", groups=8, topk_groups=2, group_score="top2")
    for k in out:
        assert torch.equal(out[k], same[k])


def test_no_tokens_and_no_route_mask(B):
    e = B.gate(torch.empty(0, 16, device="cuda"), 4)
    assert e["expert_ids"].shape == (0, 4)
    l = torch.randn(10, 16, device="cuda")
    full = B.gate(l, 4)
    out = {k: torch.empty_like(full[k]) for k in ("expert_ids", "expert_scales")}
    B.gate(l, 4, out=out)
    assert all(torch.equal(out[k], full[k]) for k in out)


def test_another_stream_and_repeats(B):
    l = torch.randn(3000, 256, device="cuda")
    a = B.gate(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = B.gate(l, 8)
    c = B.gate(l, 8, stream=s)
    s.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])


def test_feeds_dispatch(B):
    """Routes left over are inactive in the dispatch under the route mask."""
    l = torch.randn(32, 8, device="cuda")
    l[:, 2:] = -float("inf")
    r = B.gate(l, 4)
    x = torch.randn(32, 64, device="cuda").bfloat16()
    d = B.dispatch(x, r["expert_ids"], 8, 1, mask=r["route_mask"])
    torch.cuda.synchronize()
    assert B.read_device_status(d["workspace"]) == 0
    assert d["expert_token_nums"].tolist() == [32, 32, 0, 0, 0, 0, 0, 0]
