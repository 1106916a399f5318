"""moe_layer_few_tokens: bit for bit moe_layer's output, and within derived
bounds of the layer's formulas in 64 bits."""
import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    return load_binding()


def make(B, T, H, E, K, N, Z=0, C=0, mask=0, shared=False, path="small", ids="distinct", seed=0,
         extreme=False):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*s):
        return torch.rand(*s, generator=g, device=DEV)

    def randn(*s):
        return torch.randn(*s, generator=g, device=DEV)

    def int8(*s):
        w = torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device=DEV)
        if extreme:      # every product at its largest, signs mostly the same
            w = torch.where(rand(*s) < 0.9, torch.full_like(w, 127), torch.full_like(w, -128))
        return w

    total = E + Z + C
    if ids == "distinct":
        i = torch.argsort(rand(T, total), dim=1)[:, :K]
    elif ids == "any":                       # repeats within a token, and ids of no expert
        i = torch.randint(-1, total + 1, (T, K), generator=g, device=DEV)
    else:
        i = torch.full((T, K), int(ids), device=DEV)
    m = None
    if mask == 1:
        m = (rand(T) < 0.7).to(torch.uint8)
    elif mask == 2:
        m = (rand(T, K) < 0.7).to(torch.uint8)
    elif mask == "none left":
        mask, m = 1, torch.zeros(T, dtype=torch.uint8, device=DEV)
    x = randn(T, H).bfloat16()
    if extreme:
        x = torch.where(rand(T, H) < 0.9, 1.0, 0.5).bfloat16()
    d = dict(x=x, ids=i.int().contiguous(), probs=torch.softmax(randn(T, K), 1), mask=m,
             shared=randn(T, H).bfloat16() if shared else None, w1=int8(E, N, H),
             s1=1e-3 + 9e-3 * rand(E, N), w2=int8(E, H, N // 2), s2=1e-3 + 9e-3 * rand(E, H))
    if extreme:
        d["s1"].fill_(1e-6)
    d["shape"] = B.make_shape(T, 1, H, E, K, N, mask_kind=mask, has_shared=shared, zero_experts=Z,
                              copy_experts=C, ffn_path=path)
    (d["o1"], d["p1"]), (d["o2"], d["p2"]) = B.pack_weights(d["shape"], d["w1"], d["w2"])
    return d


def both(B, d, **kw):
    a = (d["shape"], d["x"], d["ids"], d["probs"], d["p1"], d["s1"], d["p2"], d["s2"])
    ref, wr = B.layer(*a, mask=d["mask"], shared=d["shared"])
    got, ws = B.layer_few_tokens(*a, mask=d["mask"], shared=d["shared"], **kw)
    torch.cuda.synchronize()
    return got, ws, ref, wr


CASES = [
    dict(T=1, H=16, E=1, K=1, N=256),
    dict(T=1, H=128, E=8, K=2, N=256),
    dict(T=1, H=2048, E=128, K=8, N=1536, shared=True),
    dict(T=1, H=7168, E=16, K=8, N=4096),
    dict(T=1, H=8192, E=3, K=2, N=8192),
    dict(T=2, H=144, E=1024, K=16, N=512, mask=2),
    dict(T=3, H=1040, E=5, K=3, N=768, path="auto", Z=1, C=1, shared=True),
    dict(T=5, H=2000, E=9, K=4, N=2816, mask=1, shared=True),
    dict(T=7, H=80, E=4, K=4, N=256, ids="any", Z=2, C=2),
    dict(T=8, H=7168, E=12, K=8, N=1024, mask=1, shared=True),
    dict(T=17, H=336, E=6, K=2, N=256, ids="2"),             # 34 routes of one expert
    dict(T=31, H=2000, E=64, K=6, N=2816, Z=2, C=1, mask=2),
    dict(T=32, H=4096, E=40, K=16, N=512),                   # all 512 routes
    dict(T=512, H=272, E=7, K=1, N=256, shared=True),
    dict(T=512, H=8192, E=130, K=1, N=256),
    dict(T=64, H=1024, E=128, K=8, N=2048, ids="any", C=1),
    dict(T=4, H=256, E=8, K=2, N=256, mask="none left", shared=True),
    dict(T=4, H=256, E=8, K=2, N=256, mask="none left"),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_same_as_the_layer(B, kw):
    d = make(B, **kw)
    got, ws, ref, wr = both(B, d)
    assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    assert B.read_device_status(ws) == B.read_device_status(wr)


def test_sums_are_exact(B):
    """Products of 127 * 127 and 127 * -128 that all add up: the fp32 sums of
    1024 of them come to just under 2^24, the totals far beyond it."""
    for H, N in ((8192, 512), (1024, 8192)):
        d = make(B, T=2, H=H, E=2, K=1, N=N, extreme=True)
        got, _, ref, _ = both(B, d)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))


def codes64(v):
    s = v.abs().amax() / 127.0
    r = v / s if float(s) else torch.zeros_like(v)
    q = torch.round(r)
    # codes that an error of a few units in the last place of fp32 could move
    return q, s, ((r - r.floor() - 0.5).abs() < 1e-4)


@pytest.mark.parametrize("kw", [
    dict(T=1, H=256, E=4, K=2, N=256, shared=True),
    dict(T=3, H=1040, E=5, K=3, N=768, Z=1, C=1),
    dict(T=9, H=512, E=4, K=4, N=512, mask=2, shared=True),
], ids=lambda c: f"T{c['T']}")
def test_against_64_bits(B, kw):
    d = make(B, seed=3, **kw)
    got, _, _, _ = both(B, d)
    E, Z, K, T, Nh = kw["E"], kw.get("Z", 0), kw["K"], kw["T"], kw["N"] // 2
    on = torch.ones(T, K) if d["mask"] is None else d["mask"].view(T, -1).expand(T, K)
    for t in range(T):
        x = d["x"][t].double()
        out = torch.zeros_like(x)
        tol = torch.zeros_like(x)
        # the first codes are defined by fp32's division, of values that are exact:
        # a quotient of bf16 numbers can be a tie in 64 bits (half the maximum is
        # 63.5 scales), which only fp32's rounding of the scale decides
        s1 = d["x"][t].float().abs().amax() / torch.full((), 127.0, device=DEV)
        q1 = torch.round(d["x"][t].float() / s1).double()
        s1 = s1.double()
        for k in range(K):
            e, p = int(d["ids"][t, k]), float(d["probs"][t, k])
            if not int(on[t, k]) or E <= e < E + Z:
                continue
            if e >= E:
                out += p * x
                tol += abs(p) * x.abs() * 2.0 ** -22
                continue
            h = (d["w1"][e].double() @ q1) * d["s1"][e].double() * s1
            gate = h[:Nh] * torch.special.expit(h[:Nh]) * h[Nh:]
            q2, s2, near = codes64(gate)
            y = (d["w2"][e].double() @ q2) * d["s2"][e].double() * s2
            moved = d["w2"][e].double().abs() @ near.double() * d["s2"][e].double() * s2
            out += p * y
            # a moved code, y's rounding to bf16, and fp32's few roundings in scale and product
            tol += abs(p) * (moved * 1.01 + y.abs() * (2.0 ** -8 + 2.0 ** -19))
        if d["shared"] is not None:
            out += d["shared"][t].double()
        tol += out.abs() * 2.0 ** -8 + tol * 2.0 ** -7 + 1e-9
        assert bool(((got[t].double() - out).abs() <= tol).all())


def test_empty(B):
    s = B.make_shape(0, 1, 128, 4, 2, 256, ffn_path="small")
    d = make(B, T=1, H=128, E=4, K=2, N=256)
    out, _ = B.layer_few_tokens(s, d["x"][:0], d["ids"][:0], d["probs"][:0], d["p1"], d["s1"], d["p2"],
                                d["s2"])
    assert out.shape == (0, 128)


def test_repeats_and_poisoned_memory(B):
    """The same bits every time, whatever the workspace and the output held."""
    d = make(B, T=6, H=1040, E=11, K=5, N=768, mask=2, shared=True)
    got, ws, ref, _ = both(B, d)
    for fill in (0, 0x7f, 0xff):
        ws.fill_(fill)
        out = torch.empty_like(got).view(torch.uint8).fill_(fill).view(torch.bfloat16)
        for _ in range(3):
            B.layer_few_tokens(d["shape"], d["x"], d["ids"], d["probs"], d["p1"], d["s1"], d["p2"], d["s2"],
                               mask=d["mask"], shared=d["shared"], ws=ws, out=out)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
        assert B.read_device_status(ws) == 0


def test_crowded_experts_many_times(B):
    """Experts with more than eight routes: every CTA has to put the same routes
    into the same block of eight."""
    for seed in range(20):
        d = make(B, T=33 + seed, H=384, E=40, K=1 + seed % 4, N=256, ids=str(seed), seed=seed)
        got, _, ref, _ = both(B, d)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16)), seed


def test_stores_stay_in_bounds(B):
    """Output and workspace between guard bytes, on both ways through the kernels."""
    for kw in (dict(T=1, H=272, E=5, K=3, N=256), dict(T=37, H=2000, E=9, K=4, N=768, mask=2, shared=True)):
        d = make(B, **kw)
        _, _, ref, _ = both(B, d)
        T, H = kw["T"], kw["H"]
        whole = torch.full(((T + 32) * H,), 0x5A5A, dtype=torch.int16, device=DEV)
        out = whole[16 * H:(16 + T) * H].view(torch.bfloat16).view(T, H)
        need = B.layer_few_tokens_workspace_size(d["shape"])
        owner = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        at = (-owner.data_ptr()) % 1024 + 1024
        B.layer_few_tokens(d["shape"], d["x"], d["ids"], d["probs"], d["p1"], d["s1"], d["p2"], d["s2"],
                           mask=d["mask"], shared=d["shared"], ws=owner[at:at + need], out=out)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
        assert bool((whole[:16 * H] == 0x5A5A).all()) and bool((whole[(16 + T) * H:] == 0x5A5A).all())
        assert bool((owner[:at] == 0xA5).all()) and bool((owner[at + need:] == 0xA5).all())


def test_nan_and_infinity_stay_in_their_tokens(B):
    for T, K, N in ((4, 2, 256), (40, 4, 2816)):
        d = make(B, T=T, H=512, E=6, K=K, N=N)
        clean, _, _, _ = both(B, d)
        d["x"][1, 7] = float("nan")
        d["x"][3, 9] = float("inf")
        d["probs"][2, 0] = float("nan")
        got, _, ref, _ = both(B, d)
        rest = [t for t in range(T) if t not in (1, 2, 3)]
        assert torch.equal(got[rest].view(torch.int16), clean[rest].view(torch.int16))
        assert bool(torch.isnan(got[2]).all())
        same = torch.isnan(got) & torch.isnan(ref) | (got == ref)
        assert bool(same.all())


def test_output_in_the_shared_buffer(B):
    for T in (1, 20):
        d = make(B, T=T, H=1024, E=6, K=3, N=512, shared=True)
        _, _, ref, _ = both(B, d)
        out, _ = B.layer_few_tokens(d["shape"], d["x"], d["ids"], d["probs"], d["p1"], d["s1"], d["p2"],
                                    d["s2"], shared=d["shared"], out=d["shared"])
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


def test_weights_past_32_bits(B):
    """Experts whose weights begin beyond 2^32 bytes of the packed buffer."""
    E, H, N = 200, 7168, 4096
    g = torch.Generator(device=DEV).manual_seed(9)
    s1 = 1e-3 + 9e-3 * torch.rand(E, N, generator=g, device=DEV)
    s2 = 1e-3 + 9e-3 * torch.rand(E, H, generator=g, device=DEV)
    w1 = torch.randint(-127, 128, (E, N, H), generator=g, dtype=torch.int8, device=DEV)
    w2 = torch.randint(-127, 128, (E, H, N // 2), generator=g, dtype=torch.int8, device=DEV)
    for T in (1, 3):
        shape = B.make_shape(T, 1, H, E, 4, N, ffn_path="small")
        (o1, p1), (o2, p2) = B.pack_weights(shape, w1, w2)
        x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        ids = (E - 1 - torch.arange(4 * T, device=DEV).view(T, 4)).int()
        probs = torch.full((T, 4), 0.25, device=DEV)
        ref, _ = B.layer(shape, x, ids, probs, p1, s1, p2, s2)
        got, _ = B.layer_few_tokens(shape, x, ids, probs, p1, s1, p2, s2)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
