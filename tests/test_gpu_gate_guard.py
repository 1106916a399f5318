"""moe_gate's stores stay in its outputs: guard rows of a byte pattern around
them, at one token, a last block that is not full, and every form of the run
(vectors, shared memory, groups, left-over routes)."""
import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu

PAD, PATTERN = 16, 0xA5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,kw", [
    (1, 1, 1, {}),
    (1, 256, 8, dict(score="sigmoid", groups=8, topk_groups=4, group_score="top2")),
    (5, 33, 16, {}),
    (7, 40, 3, dict(score="sigmoid")),
    (127, 160, 6, dict(groups=8, topk_groups=3)),
    (130, 999, 16, dict(groups=3, topk_groups=1)),
    (9, 1024, 16, dict(score="sigmoid", groups=512, topk_groups=100)),
])
@pytest.mark.parametrize("closed", [0.0, 0.97, 1.0])
def test_stores_stay_in_bounds(T, E, K, kw, dtype, closed):
    B = load_binding()
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = torch.randn(T, E, generator=g, device="cuda").to(dtype)
    l[torch.rand(T, E, generator=g, device="cuda") < closed] = -float("inf")
    want = B.gate(l, K, **kw)
    full, out = {}, {}
    for k, dt in (("expert_ids", torch.int32), ("expert_scales", torch.float32), ("route_mask", torch.uint8)):
        full[k] = torch.empty(T + 2 * PAD, K, dtype=dt, device="cuda")
        full[k].view(torch.uint8).fill_(PATTERN)
        out[k] = full[k][PAD:PAD + T]
    B.gate(l, K, out=out, **kw)
    for k in full:
        b = full[k].view(torch.uint8)
        assert bool((b[:PAD] == PATTERN).all()) and bool((b[PAD + T:] == PATTERN).all()), k
        assert torch.equal(out[k], want[k]), k
