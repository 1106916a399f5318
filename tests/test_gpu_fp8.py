"""moe_grouped_gemm_fp8 and moe_grouped_ffn_fp8 against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_ref as R
from gpu_util import load_binding

pytestmark = pytest.mark.gpu

PATHS = ["large", "large_pair", "small"]


@pytest.fixture(scope="module")
def B():
    return load_binding()


def codes(g, *shape):
    """e4m3 codes over the format's whole range, zeros and subnormals included."""
    v = torch.randn(*shape, generator=g, device="cuda") * 110.0
    small = torch.rand(*shape, generator=g, device="cuda") < 0.1
    return torch.where(small, v * 1e-4, v).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(g, typical, *shape):
    return typical * torch.exp(0.5 * torch.randn(*shape, generator=g, device="cuda"))


def values(q, *axes_scales):
    v = q.float().cpu().numpy().astype(np.float64)
    for axes, s in axes_scales:
        f = s.cpu().numpy().astype(np.float64)
        for ax in axes:
            f = R.expand(f, v.shape[ax], ax)
        v = v * f
    return v


def gemm_case(counts, N, Kd, seed, spare=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + spare
    return dict(off=off, a=codes(g, rows, Kd), sa=scales(g, 0.01, rows, R.blocks(Kd)),
                w=codes(g, E, N, Kd), sw=scales(g, 1e-4, E, R.blocks(N), R.blocks(Kd)))


def gemm_ref(c):
    return R.product(values(c["a"], ((1,), c["sa"])), c["off"],
                     values(c["w"], ((1, 2), c["sw"])))


RAGGED = [1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0]


@pytest.mark.parametrize("path", PATHS + ["auto"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,Kd", [
    ([1], 8, 16),
    ([1], 128, 128),
    ([3], 4096, 1024),
    ([0, 130, 257], 256, 64),
    ([129, 0, 0, 64, 1], 264, 2064),          # N and K end inside a block
    (RAGGED, 136, 80),
    ([700, 333, 1024, 17, 256, 0, 90, 511], 512, 640),
    ([8] * 40 + [0] * 8 + [3] * 16, 384, 1152),
    ([300], 1000, 1456),
    ([0, 0, 5], 392, 144),
    ([0, 0, 0], 64, 64),                      # no rows at all
])
def test_product(B, counts, N, Kd, out_dtype, path):
    c = gemm_case(counts, N, Kd, N + Kd)
    R0 = int(c["off"][-1])
    out = torch.full((c["a"].shape[0], N), 7.0, dtype=out_dtype, device="cuda")
    _, ws = B.grouped_gemm_fp8(torch.from_numpy(c["off"]).cuda(), c["a"], c["sa"], c["w"], c["sw"],
                               out=out, path=path)
    torch.cuda.synchronize()
    assert B.read_device_status(ws) == 0
    ref, mag = gemm_ref(c)
    bound = R.product_bound(mag, Kd) + (np.abs(ref) * 2.0 ** -8 if out_dtype == torch.bfloat16 else 0)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref)[:R0] <= bound[:R0] + 1e-30)
    assert np.all(got[R0:] == 7.0)            # rows past the last expert's


@pytest.mark.parametrize("path", PATHS)
def test_product_has_fp32_sums(B, path):
    """Cancelling blocks: a wide sum that a narrower accumulator would lose."""
    Kd, N, rows = 1024, 128, 40
    g = torch.Generator(device="cuda").manual_seed(0)
    a = torch.zeros(rows, Kd)
    a[:, :1024:2] = 448.0
    a[:, 1:1024:2] = -448.0
    a[:, 1023] = -448.0 + 32.0
    w = torch.ones(1, N, Kd) * 448.0
    ones = torch.ones
    out, _ = B.grouped_gemm_fp8(torch.tensor([0, rows], dtype=torch.int32).cuda(),
                                a.to(torch.float8_e4m3fn).cuda(), ones(rows, 8).cuda(),
                                w.to(torch.float8_e4m3fn).cuda(), ones(1, 1, 8).cuda(),
                                out_dtype=torch.float32, path=path)
    assert (out == 32.0 * 448.0).all()


def test_product_repeats_and_streams(B):
    c = gemm_case([40, 300, 0, 7], 264, 528, 9)
    off = torch.from_numpy(c["off"]).cuda()
    for path in PATHS:
        a, ws = B.grouped_gemm_fp8(off, c["a"], c["sa"], c["w"], c["sw"], path=path)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        b, _ = B.grouped_gemm_fp8(off, c["a"], c["sa"], c["w"], c["sw"], path=path, stream=s)
        d, _ = B.grouped_gemm_fp8(off, c["a"], c["sa"], c["w"], c["sw"], path=path, ws=ws)
        torch.cuda.synchronize()
        n = int(c["off"][-1])
        assert torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16))
        assert torch.equal(a[:n].view(torch.int16), d[:n].view(torch.int16))


def test_nan_and_zero_scales_stay_in_their_rows(B):
    c = gemm_case([20, 30], 136, 272, 4, spare=0)
    off = torch.from_numpy(c["off"]).cuda()
    for path in PATHS:
        clean, _ = B.grouped_gemm_fp8(off, c["a"], c["sa"], c["w"], c["sw"], path=path)
        a, sa = c["a"].clone(), c["sa"].clone()
        a.view(torch.uint8)[3, 200] = 0x7F            # the NaN code
        sa[25] = 0.0
        got, _ = B.grouped_gemm_fp8(off, a, sa, c["w"], c["sw"], path=path)
        assert torch.isnan(got[3]).all() and (got[25] == 0).all()
        keep = [r for r in range(50) if r not in (3, 25)]
        assert torch.equal(got[keep], clean[keep])


def ffn_case(B, T, P, H, E, K, N, seed, mask_p=1.0, ffn_path="auto"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].int()
    mask = None
    if mask_p < 1:
        mask = (torch.rand(T, K, generator=g, device="cuda") < mask_p).to(torch.uint8)
    d = B.dispatch(None, ids, E, P, mask=mask, with_rows=False)
    return dict(shape=B.make_shape(T, P, H, E, K, N, ffn_path=ffn_path), d=d,
                x=codes(g, T, H), xs=scales(g, 0.01, T, R.blocks(H)),
                w1=codes(g, E, N, H), s1=scales(g, 2e-4, E, N // 128, R.blocks(H)),
                w2=codes(g, E, H, N // 2), s2=scales(g, 2e-4, E, R.blocks(H), N // 256))


def ffn_check(B, c, y):
    P = c["shape"].num_partitions
    M = c["shape"].num_tokens // P
    off = c["d"]["expert_offsets"].cpu().numpy()
    n = int(off[-1])
    as_ = c["d"]["assist"][:n].cpu().numpy()
    tok = as_[:, 0] * M + as_[:, 1]
    ref, bound = R.ffn(values(c["x"], ((1,), c["xs"]))[tok], off, values(c["w1"], ((1, 2), c["s1"])),
                       values(c["w2"], ((1, 2), c["s2"])))
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got[:n] - ref) <= bound)
    assert np.linalg.norm(got[:n] - ref) <= 4e-3 * max(np.linalg.norm(ref), 1e-30)
    assert np.all(got[n:] == 7.0)


@pytest.mark.parametrize("path", PATHS + ["auto"])
@pytest.mark.parametrize("T,P,H,E,K,N,mask_p", [
    (1, 1, 128, 8, 2, 256, 1.0),
    (16, 2, 128, 8, 2, 256, 1.0),
    (45, 3, 272, 9, 3, 512, 0.7),             # H ends inside a block, routes masked
    (300, 1, 400, 5, 2, 768, 1.0),
    (64, 4, 1024, 64, 8, 256, 0.9),
    (700, 1, 256, 4, 4, 1024, 1.0),           # every expert takes every token
    (20, 1, 144, 6, 2, 256, 0.0),             # every route masked: nothing to do
])
def test_ffn(B, T, P, H, E, K, N, mask_p, path):
    c = ffn_case(B, T, P, H, E, K, N, T + H, mask_p, path)
    y = torch.full((T * K, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _, ws = B.grouped_ffn_fp8(c["shape"], c["x"], c["xs"], c["d"]["expert_offsets"], c["w1"],
                              c["s1"], c["w2"], c["s2"], assist=c["d"]["assist"], y=y)
    torch.cuda.synchronize()
    assert B.read_device_status(ws) == 0
    ffn_check(B, c, y)


@pytest.mark.parametrize("path", PATHS)
def test_ffn_on_rows_equals_ffn_on_tokens(B, path):
    c = ffn_case(B, 60, 2, 272, 6, 3, 512, 1, 0.8, path)
    n = int(c["d"]["expert_offsets"][-1])
    as_ = c["d"]["assist"][:n].long()
    tok = as_[:, 0] * 30 + as_[:, 1]
    rows = torch.zeros(180, 272, dtype=torch.uint8, device="cuda")
    rs = torch.zeros(180, 3, device="cuda")
    rows[:n] = c["x"].view(torch.uint8)[tok]
    rs[:n] = c["xs"][tok]
    args = (c["d"]["expert_offsets"], c["w1"], c["s1"], c["w2"], c["s2"])
    a, _ = B.grouped_ffn_fp8(c["shape"], c["x"], c["xs"], *args, assist=c["d"]["assist"])
    b, _ = B.grouped_ffn_fp8(c["shape"], rows.view(torch.float8_e4m3fn), rs, *args)
    assert torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16))


@pytest.mark.parametrize("E,K,P,mask_p,skew", [
    (5, 2, 1, 1.0, 0.0),
    (5, 2, 4, 0.3, 0.0),                      # most routes masked
    (40, 3, 2, 0.9, 0.95),                    # almost every token's first route to one expert
    (1, 1, 1, 1.0, 0.0),
    (700, 2, 5, 1.0, 0.0),                    # fewer rows per expert than a segment's
    (6, 2, 1, 0.0, 0.0),                      # no rows
])
def test_ffn_on_many_tokens_takes_every_row(B, E, K, P, mask_p, skew):
    """More tokens than are copied in the rows' own order: the same rows, bit for bit."""
    T, H, N = 4700, 7168, 256
    g = torch.Generator(device="cuda").manual_seed(E + K)
    score = torch.rand(T, E, generator=g, device="cuda")
    score[:, E // 2] += (torch.rand(T, generator=g, device="cuda") < skew).float()
    ids = score.argsort(1, descending=True)[:, :K].int().contiguous()
    mask = (torch.rand(T, K, generator=g, device="cuda") < mask_p).to(torch.uint8)
    d = B.dispatch(None, ids, E, P, mask=mask, with_rows=False)
    x, xs = codes(g, T, H), scales(g, 0.01, T, H // 128)
    w = (codes(g, E, N, H), scales(g, 2e-4, E, 2, H // 128), codes(g, E, H, N // 2),
         scales(g, 2e-4, E, H // 128, 1))
    shape = B.make_shape(T, P, H, E, K, N)
    n = int(d["expert_offsets"][-1])
    assert n == int(mask.sum())
    as_ = d["assist"][:n].long()
    tok = as_[:, 0] * (T // P) + as_[:, 1]
    rows = torch.zeros(T * K, H, dtype=torch.uint8, device="cuda")
    rs = torch.zeros(T * K, H // 128, device="cuda")
    rows[:n] = x.view(torch.uint8)[tok]
    rs[:n] = xs[tok]
    y = torch.full((T * K, H), 7.0, dtype=torch.bfloat16, device="cuda")
    a, ws = B.grouped_ffn_fp8(shape, x, xs, d["expert_offsets"], *w, assist=d["assist"], y=y)
    b, _ = B.grouped_ffn_fp8(shape, rows.view(torch.float8_e4m3fn), rs, d["expert_offsets"], *w)
    torch.cuda.synchronize()
    assert B.read_device_status(ws) == 0
    assert torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16))
    assert bool((a[n:] == 7.0).all())


def test_ffn_no_tokens(B):
    s = B.make_shape(0, 1, 128, 4, 2, 256)
    z = torch.zeros
    f8 = torch.float8_e4m3fn
    y, _ = B.grouped_ffn_fp8(s, z(0, 128, device="cuda").to(f8), z(0, 1, device="cuda"),
                             z(5, dtype=torch.int32, device="cuda"),
                             z(4, 256, 128, device="cuda").to(f8), z(4, 2, 1, device="cuda"),
                             z(4, 128, 128, device="cuda").to(f8), z(4, 1, 1, device="cuda"))
    assert y.shape == (0, 128)
