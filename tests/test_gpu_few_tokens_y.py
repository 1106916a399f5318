"""moe_layer_few_tokens with the experts' outputs in fp32 up to the weighted sum: within
what one rounding leaves of the formulas in 64 bits, which rounded outputs exceed."""
import pytest
import torch

from test_gpu_few_tokens import B, codes64, make  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(B, d, **kw):  # noqa: F811
    got, ws = B.layer_few_tokens(d["shape"], d["x"], d["ids"], d["probs"], d["p1"], d["s1"], d["p2"], d["s2"],
                                 mask=d["mask"], shared=d["shared"], **kw)
    torch.cuda.synchronize()
    assert B.read_device_status(ws) == 0
    return got


def formulas(d, kw):
    """The output in 64 bits, and what may lie between it and fp32 sums rounded once to bf16."""
    E, Z, K, T, Nh = kw["E"], kw.get("Z", 0), kw["K"], kw["T"], kw["N"] // 2
    on = torch.ones(T, K) if d["mask"] is None else d["mask"].view(T, -1).expand(T, K)
    out = torch.zeros(T, kw["H"], dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for t in range(T):
        # the first codes as fp32's division gives them (quotients of bf16 numbers can be ties)
        x = d["x"][t].float()
        s1 = x.abs().amax() / torch.full((), 127.0, device=DEV)
        q1 = torch.round(x / s1).double()
        for k in range(K):
            e, p = int(d["ids"][t, k]), float(d["probs"][t, k])
            if not int(on[t, k]) or E <= e < E + Z:
                continue
            if e >= E:
                y, err = x.double(), 0.0
            else:
                h = (d["w1"][e].double() @ q1) * d["s1"][e].double() * s1.double()
                q2, s2, near = codes64(h[:Nh] * torch.special.expit(h[:Nh]) * h[Nh:])
                y = (d["w2"][e].double() @ q2) * d["s2"][e].double() * s2
                # codes that fp32 could move by one; s2 and two products in fp32
                err = d["w2"][e].double().abs() @ near.double() * d["s2"][e].double() * s2 * 1.01 + y.abs() * 2.0 ** -19
            out[t] += p * y
            # p * y and each addition to the sum round in fp32: 2 + K steps of 2^-24 of a term at most
            tol[t] += abs(p) * (err + y.abs() * (K + 2) * 2.0 ** -24)
    if d["shared"] is not None:
        out += d["shared"].double()
        tol += (out.abs() + d["shared"].double().abs()) * 2.0 ** -24
    # the one rounding to bf16, of a value that is `tol` away
    return out, tol + (out.abs() + tol) * 2.0 ** -8 + 1e-9


CASES = [dict(T=1, H=256, E=8, K=8, N=256), dict(T=1, H=2048, E=12, K=8, N=512, shared=True),
         dict(T=3, H=1040, E=5, K=3, N=768, Z=1, C=1, path="auto"), dict(T=9, H=512, E=9, K=4, N=512, mask=2, shared=True),
         dict(T=40, H=272, E=3, K=3, N=256, mask=1)]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: f"T{c['T']}-H{c['H']}")
def test_against_64_bits(B, kw):  # noqa: F811
    d = make(B, seed=11, **kw)
    ref, tol = formulas(d, kw)
    got, rounded = layer(B, d, y_dtype=torch.float32), layer(B, d)
    assert bool(((got.double() - ref).abs() <= tol).all())
    # what the choice is for: experts' outputs that were rounded come out further away
    assert bool(((rounded.double() - ref).abs() > tol).any())
    assert float((got.double() - ref).norm()) < float((rounded.double() - ref).norm())


def test_same_bits_whatever_the_memory_held(B):  # noqa: F811
    for kw in (dict(T=2, H=1040, E=11, K=5, N=768), dict(T=37, H=336, E=4, K=4, N=512, mask=2, shared=True)):
        d = make(B, **kw)
        want = layer(B, d, y_dtype=torch.float32)
        size = B.layer_few_tokens_workspace_size(d["shape"])
        for fill in (0, 0x7f, 0xff):
            ws = torch.full((size + 1024,), fill, dtype=torch.uint8, device=DEV)
            ws = ws[-ws.data_ptr() % 1024:][:size]
            out = torch.empty_like(want).view(torch.uint8).fill_(fill).view(torch.bfloat16)
            for _ in range(3):
                layer(B, d, y_dtype=torch.float32, ws=ws, out=out)
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_one_route_is_rounded_once_either_way(B):  # noqa: F811
    """A single route of weight 1 has nothing between its product and the output."""
    d = make(B, T=5, H=512, E=4, K=1, N=512)
    assert bool((d["probs"] == 1.0).all())
    assert torch.equal(layer(B, d, y_dtype=torch.float32).view(torch.int16), layer(B, d).view(torch.int16))
