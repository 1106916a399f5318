"""moe_gate's order where fp32 scores saturate: the keys are scores in fp32, so
logits whose scores are the same number tie, whatever the logits are, and the
lower index comes first, with a bias and without one.

The reference rounds 64-bit scores to fp32.  The logits are such that any fp32
evaluation within a few units in the last place agrees with it: sigmoids of 18
and more are 1 (1 - 2^-25.97 rounds to 1), exponentials of -110 and less and
sigmoids of -110 and less are 0, and the others lie far apart."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import dev, load_binding

pytestmark = pytest.mark.gpu

MAX32 = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def B():
    return load_binding()


def reference(logits, bias, K, score, groups, topk_groups, group_score):
    """(ids, weights) from keys in fp32."""
    l = logits.astype(np.float64)
    key, s, _ = R.gate_keys(l, None, None, score, 1, 1, "max")
    key, s = key.astype(np.float32), s.astype(np.float32).astype(np.float64)
    if bias is not None:
        key = key + bias
    T, E = key.shape
    if groups > 1:
        per = -np.sort(-key.reshape(T, groups, -1), axis=2)
        gv = per[:, :, 0].copy()
        if group_score == "top2" and per.shape[2] > 1:
            gv = np.where(per[:, :, 1] > -np.inf, per[:, :, 0] + per[:, :, 1], gv)
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, np.argsort(-gv, axis=1, kind="stable")[:, :topk_groups], True, axis=1)
        key = np.where(np.repeat(keep, E // groups, 1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    on = np.take_along_axis(key, ids, 1) > -np.inf
    w = np.where(on, np.take_along_axis(s, ids, 1), 0.0)
    return np.where(on, ids, -1), w / (w.sum(1, keepdims=True) + 1e-20)


def check(B, logits, K, score, groups=1, topk_groups=1, group_score="max", bias=None):
    t = logits if isinstance(logits, torch.Tensor) else dev(np.float32(logits))
    out = B.gate(t, K, bias=dev(bias), score=score, groups=groups, topk_groups=topk_groups,
                 group_score=group_score)
    ids, w = reference(t.float().cpu().numpy(), bias, K, score, groups, topk_groups, group_score)
    np.testing.assert_array_equal(out["expert_ids"].cpu().numpy(), ids)
    # a weight: the exponential's argument (at most 16 here), exponential,
    # sum and quotients, 2^-24 of its size each
    got = out["expert_scales"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w) <= w * 40 * 2.0 ** -24 + 2.0 ** -126)
    return out


HIGH = [18.0, 20.0, 25.0, 40.0, 100.0, 1e4, MAX32, np.inf]
LOW = [-110.0, -120.0, -300.0, -1e4, -1e29]
CLOSED = [-np.inf, np.nan, -MAX32, -1e30]
# no two scores, nor sums of two, are equal or near
MID = np.array([-4.0, -3.25, -2.25, -1.125, 0.3125, 0.875, 1.75, 2.625, 3.5])


def test_the_values_are_far_apart():
    for f in (lambda v: 1.0 / (1.0 + np.exp(-v)), np.exp):
        s = np.concatenate([[0.0, 1.0], f(MID)])
        sums = np.sort(np.concatenate([s, (s[:, None] + s)[np.triu_indices(s.size)]]))
        gaps = np.diff(sums)
        assert gaps[gaps > 1e-12].min() > 1e-4


def rows(score, T, E, seed):
    """Rows of few to many saturated logits among some that are not, some closed."""
    g = np.random.default_rng(seed)
    l = g.choice(MID, (T, E))
    high = HIGH if score == "sigmoid" else [0.0]
    for t in range(T):
        u = g.random(E)
        share = g.choice([0.0, 0.02, 0.1, 0.6])
        l[t] = np.where(u < share, g.choice(high, E), l[t])
        share = g.choice([0.0, 0.3, 0.97])
        l[t] = np.where(g.random(E) < share, g.choice(LOW, E), l[t])
        l[t] = np.where(g.random(E) < 0.05, g.choice(CLOSED, E), l[t])
    return l


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K,groups,topk_groups,group_score", [
    (5, 3, 1, 1, "max"),
    (40, 4, 1, 1, "max"),
    (128, 8, 8, 3, "max"),
    (256, 8, 1, 1, "max"),
    (256, 8, 8, 4, "top2"),
    (333, 16, 1, 1, "max"),
    (512, 12, 16, 4, "max"),
    (660, 5, 20, 3, "top2"),
    (1000, 16, 20, 7, "max"),
    (1024, 8, 512, 40, "top2"),
    (1024, 16, 1, 1, "max"),
])
def test_saturated_scores_tie(B, E, K, groups, topk_groups, group_score, dtype, score):
    l = torch.from_numpy(np.float32(rows(score, 200, E, E + K))).to(dtype).cuda()
    kw = dict(groups=groups, topk_groups=topk_groups, group_score=group_score)
    a = check(B, l, K, score, **kw)
    b = check(B, l, K, score, bias=np.zeros(E, np.float32), **kw)
    assert torch.equal(a["expert_ids"], b["expert_ids"])


def test_the_rows_of_the_extreme_logits(B):
    """Logits up to 1900 and down to -2000: sigmoids of all the large ones are
    1; exponentials of all but the first two are 0 (the second is 2^-144)."""
    l = np.zeros((2, 40))
    l[1] = np.arange(40) * 100.0 - 2000.0
    out = check(B, l, 4, "sigmoid")
    np.testing.assert_array_equal(out["expert_ids"][1].cpu().numpy(), [21, 22, 23, 24])
    out = B.gate(dev(np.float32(l)), 4, score="softmax")
    np.testing.assert_array_equal(out["expert_ids"].cpu().numpy(), [[0, 1, 2, 3], [39, 38, 0, 1]])
    np.testing.assert_array_equal(out["expert_scales"][1].cpu().numpy() > 0.5, [True, False, False, False])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [8, 256, 900])
def test_infinity_is_the_largest_number(B, E, score):
    """+inf and the largest finite number are equal."""
    l = np.zeros((3, E))
    l[:, 2] = MAX32
    l[:, 5] = np.inf
    l[1, [2, 5]] = l[1, [5, 2]]
    l[2, 7] = MAX32
    check(B, l, 2, score)
    check(B, l, 2, score, bias=np.zeros(E, np.float32))


@pytest.mark.parametrize("E", [64, 256, 600])
def test_scores_near_one(B, E):
    """Between 12 and 17 the sigmoids are 1 minus a few multiples of 2^-24:
    the kernel's choice has to be in the order of the 64-bit scores up to that
    spacing (two roundings of 1 + e and the quotient, a unit each way)."""
    g = np.random.default_rng(E)
    l = np.float32(g.uniform(11.0, 17.0, (300, E)))
    ids = B.gate(dev(l), 8, score="sigmoid")["expert_ids"].cpu().numpy()
    s = 1.0 / (1.0 + np.exp(-l.astype(np.float64)))
    want = -np.sort(-s, axis=1)[:, :8]
    got = np.take_along_axis(s, ids, 1)
    assert np.all(np.abs(got - want) <= 4 * 2.0 ** -24)
    # equal to the bit: 1 + e in fp32 decides, the lower index first
    for t in range(300):
        assert len(set(ids[t])) == 8
        e = np.exp(-l[t].astype(np.float64))
        d = np.float32(1.0) + np.float32(e)
        sure = np.abs(e * 2.0 ** 23 - np.floor(e * 2.0 ** 23) - 0.5) > 1e-4 * (1 + e * 2.0 ** 23)
        order = [i for i in ids[t] if sure[i]]
        for a, b in zip(order, order[1:]):
            assert d[a] < d[b] or (d[a] == d[b] and a < b)
