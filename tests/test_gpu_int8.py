"""moe_grouped_gemm_int8: bit for bit its definition (an exact integer sum and
single fp32 operations), and within derived bounds of 64 bits, on every kernel."""
import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    return load_binding()


def make(rows, E, N, Kd, a="int8", bias=False, counts=None, seed=0, extreme=False):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*s):
        return torch.rand(*s, generator=g, device=DEV)

    def int8(*s):
        w = torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device=DEV)
        if extreme:
            w = torch.where(rand(*s) < 0.95, torch.full_like(w, -128), torch.full_like(w, 127))
        return w

    if counts is None:
        pick = torch.randint(0, E, (rows,), generator=g, device=DEV)
        counts = torch.bincount(pick, minlength=E).tolist()
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    d = dict(off=off.to(DEV), w=int8(E, N, Kd), ws=1e-4 + 9e-4 * rand(E, N),
             bias=torch.randn(E, N, generator=g, device=DEV) if bias else None)
    if a == "int8":
        d["a"], d["as_"] = int8(rows, Kd), 0.01 + 0.02 * rand(rows)
    else:
        d["a"], d["as_"] = torch.randn(rows, Kd, generator=g, device=DEV).bfloat16(), None
    return d


def codes(d):
    if d["as_"] is not None:
        return d["a"].double(), d["as_"]
    x = d["a"].float()
    s = x.abs().amax(1) / torch.full((), 127.0, device=DEV)
    q = torch.where(s[:, None] > 0, torch.round(x / torch.where(s > 0, s, 1.0)[:, None]), 0.0)
    return q.clamp(-127, 127).double(), s


def reference(d, dtype):
    """The definition in the precision it is defined in, and in 64 bits."""
    q, s = codes(d)
    off = d["off"].tolist()
    R = off[-1]
    out = torch.empty(R, d["w"].shape[1], device=DEV)
    out64 = out.double()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        acc = q[lo:hi] @ d["w"][e].double().T                    # exact: below 2^53
        v = (acc.float() * d["ws"][e]) * s[lo:hi, None]
        v64 = acc * d["ws"][e].double() * s[lo:hi, None].double()
        if d["bias"] is not None:
            v, v64 = v + d["bias"][e], v64 + d["bias"][e].double()
        out[lo:hi], out64[lo:hi] = v, v64
    return out.to(dtype), out64


def check(B, d, path, dtype, **kw):
    _, packed = B.pack_int8(d["w"], path=path)
    rows, N = d["a"].shape[0], d["w"].shape[1]
    out = torch.full((rows, N), 7.0, dtype=dtype, device=DEV)
    got, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], bias=d["bias"],
                                  out=out, path=path, **kw)
    torch.cuda.synchronize()
    assert B.read_device_status(ws) == 0
    ref, ref64 = reference(d, dtype)
    R = ref.shape[0]
    assert torch.equal(got[:R], ref)
    assert bool((got[R:] == 7.0).all())
    # three roundings of the product and one of the sum with the bias, then bf16's
    prod = (ref64 if d["bias"] is None else ref64 - torch.repeat_interleave(
        d["bias"], torch.diff(d["off"]).long(), 0).double()).abs()
    tol = prod * 3.01 * 2.0 ** -24 + ref64.abs() * 1.01 * 2.0 ** -24
    if dtype is torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + ref64.abs() * 2.0 ** -8
    assert bool(((got[:R].double() - ref64).abs() <= tol + 1e-30).all())


@pytest.mark.parametrize("path", ["auto", "small", "large", "large_pair"])
@pytest.mark.parametrize("kw", [
    dict(rows=1, E=1, N=8, Kd=16),
    dict(rows=1, E=1, N=4096, Kd=7168, a="bf16"),
    dict(rows=2, E=1, N=1000, Kd=1456, a="bf16", bias=True),
    dict(rows=5, E=1, N=264, Kd=4112, a="bf16"),
    dict(rows=8, E=1, N=520, Kd=8192, a="bf16"),
    dict(rows=9, E=1, N=520, Kd=8208, a="bf16"),
    dict(rows=7, E=1, N=72, Kd=144),
    dict(rows=17, E=1, N=1040, Kd=2048, bias=True),
    dict(rows=31, E=2, N=136, Kd=272, a="bf16"),
    dict(rows=33, E=1, N=4096, Kd=1024),
    dict(rows=64, E=1, N=7168, Kd=2048),
    dict(rows=100, E=3, N=392, Kd=5008, a="bf16", bias=True),
    dict(rows=130, E=1, N=256, Kd=16384, a="bf16"),
    dict(rows=300, E=40, N=136, Kd=400),
    dict(rows=257, E=1, N=1000, Kd=1456, bias=True),
    dict(rows=600, E=3, N=4104, Kd=528, a="bf16"),
], ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_definition(B, path, kw):
    for dtype in (torch.bfloat16, torch.float32):
        check(B, make(**kw), path, dtype)


@pytest.mark.parametrize("counts", [[0, 0, 0], [0, 5, 0], [1, 0, 9], [33, 2, 0], [0, 0, 140]], ids=str)
@pytest.mark.parametrize("path", ["auto", "small", "large", "large_pair"])
def test_empty_groups_and_rows_behind_the_last(B, path, counts):
    for a in ("int8", "bf16"):
        check(B, make(sum(counts) + 3, 3, 200, 336, a=a, counts=counts, bias=True), path, torch.float32)


@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
@pytest.mark.parametrize("rows", [1, 4, 6, 12, 30, 64, 128])
def test_sums_are_exact(B, path, rows):
    """Nearly every product is (-128) * (-128): sums of 1024 of them are just
    under 2^24, the whole ones far beyond it."""
    check(B, make(rows, 1, 136, 8192, extreme=True), path, torch.float32)


def test_zero_rows_and_special_values(B):
    d = make(6, 1, 64, 128, a="bf16")
    d["a"][1] = 0.0
    d["a"][2] = 0.0
    d["a"][2, 5] = 3e38
    d["a"][3] *= 1e-38
    for path in ("small", "large_pair"):
        check(B, d, path, torch.float32)


def test_no_rows(B):
    d = make(0, 2, 64, 128)
    _, packed = B.pack_int8(d["w"])
    out, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"])
    assert out.shape == (0, 64)


def test_split_tiles_many_times(B):
    """The CTAs that share a tile's inner dimension meet at a counter that every
    call clears: the same bits whatever the workspace held."""
    d = make(64, 1, 1024, 4096)
    _, packed = B.pack_int8(d["w"], path="small")
    ref, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], path="small")
    want, _ = reference(d, torch.bfloat16)
    assert torch.equal(ref, want)
    for fill in (0, 1, 0xff):
        ws.fill_(fill)
        for _ in range(20):
            got, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], ws=ws,
                                         path="small")
        assert torch.equal(got, want)


def test_stores_stay_in_bounds(B):
    """Output and workspace between guard bytes, on every kernel."""
    for rows, N, Kd, path in ((3, 200, 336, "small"), (20, 200, 336, "small"), (130, 1000, 5008, "small"),
                              (300, 1000, 528, "large_pair"), (300, 1000, 528, "large")):
        for dtype in (torch.float32, torch.bfloat16):
            d = make(rows, 1, N, Kd)
            _, packed = B.pack_int8(d["w"], path=path)
            ref, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], path=path,
                                          out_dtype=dtype)
            size = torch.finfo(dtype).bits // 8
            whole = torch.full(((rows + 32) * N * size,), 0x5A, dtype=torch.uint8, device=DEV)
            out = whole[16 * N * size:(16 + rows) * N * size].view(dtype).view(rows, N)
            need = ws.numel()
            owner = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
            at = (-owner.data_ptr()) % 1024 + 1024
            B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], path=path, out=out,
                                ws=owner[at:at + need])
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
            assert bool((whole[:16 * N * size] == 0x5A).all()) and bool((whole[(16 + rows) * N * size:] == 0x5A).all())
            assert bool((owner[:at] == 0xA5).all()) and bool((owner[at + need:] == 0xA5).all())


def test_weights_past_32_bits(B):
    """Groups whose weights begin beyond 2^32 bytes, on every kernel."""
    E, N, Kd = 40, 8192, 16384
    w = torch.randint(-127, 128, (E, N, Kd), dtype=torch.int8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    ws = 1e-4 + 9e-4 * torch.rand(E, N, generator=g, device=DEV)
    for rows, path in ((3, "small"), (400, "small"), (300, "large_pair"), (300, "large")):
        _, packed = B.pack_int8(w, path=path)
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[E] = rows                              # all rows in the last group
        a = torch.randint(-127, 128, (rows, Kd), generator=g, dtype=torch.int8, device=DEV)
        s = 0.01 + 0.02 * torch.rand(rows, generator=g, device=DEV)
        got, _ = B.grouped_gemm_int8(off, a, packed, ws, a_scales=s, path=path, out_dtype=torch.float32)
        acc = a.double() @ w[E - 1].double().T
        assert torch.equal(got, (acc.float() * ws[E - 1]) * s[:, None])
        del packed


@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
def test_nan_makes_its_row_nan(B, path):
    for rows in (2, 8, 20, 300):
        d = make(rows, 1, 264, 528, a="bf16")
        _, packed = B.pack_int8(d["w"], path=path)
        clean, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path=path)
        d["a"][rows // 2, 100] = float("nan")
        got, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path=path)
        rest = [r for r in range(rows) if r != rows // 2]
        assert bool(torch.isnan(got[rows // 2]).all())
        assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
def test_first_group_begins_behind_the_first_row(B, path):
    """Rows before expert_offsets[0] belong to no group: not read, not written."""
    for rows, a in ((5, "bf16"), (5, "int8"), (30, "bf16"), (300, "int8")):
        d = make(rows, 1, 200, 336, a=a)
        want, _ = reference(d, torch.float32)
        d["off"][0] = 2
        _, packed = B.pack_int8(d["w"], path=path)
        out = torch.full((rows, 200), 7.0, device=DEV)
        B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], out=out, path=path)
        assert torch.equal(out[2:], want[2:])
        assert bool((out[:2] == 7.0).all())


@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
def test_offsets_that_are_not_ascending(B, path):
    """Groups end at the last offset, and begin where the ones before them end, whatever is given."""
    for rows, N, Kd, a in ((30, 200, 336, "int8"), (130, 1000, 5008, "int8"), (130, 1000, 5008, "bf16")):
        d = make(rows, 40, N, Kd, a=a)
        _, packed = B.pack_int8(d["w"], path=path)
        up = d["off"].cpu()
        for bad in (up + torch.arange(41) * 1000, up - 1000, up.flip(0), torch.where(torch.arange(41) % 2 == 0, up, rows - up),
                    torch.where(torch.arange(41) < 40, torch.full_like(up, 2 ** 31 - 1), torch.full_like(up, rows - 3)),
                    torch.where(torch.arange(41) < 40, torch.full_like(up, -2 ** 31), torch.full_like(up, 2 ** 31 - 1))):
            last = int(bad[-1].clamp(0, rows))
            meant = bad.clamp(0, last).cummax(0).values
            out = [torch.full((rows, N), 7.0, device=DEV) for _ in range(2)]
            for off, o in zip((bad, meant), out):
                _, ws = B.grouped_gemm_int8(off.to(DEV, torch.int32), d["a"], packed, d["ws"], a_scales=d["as_"], out=o,
                                            path=path)
                assert B.read_device_status(ws) == 0
            assert torch.equal(*out)
            assert bool((out[0][last:] == 7.0).all()) and bool((out[0][:int(meant[0])] == 7.0).all())


@pytest.mark.parametrize("path", ["small", "large", "large_pair"])
@pytest.mark.parametrize("rows", [2, 6, 20])
def test_deepest_sums_fit_32_bits(B, path, rows):
    Kd = 131056
    w = torch.full((1, 8, Kd), -128, dtype=torch.int8, device=DEV)
    w[0, 1] = 127
    a = torch.full((rows, Kd), -128, dtype=torch.int8, device=DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    one = torch.ones(1, 8, device=DEV)
    out, _ = B.grouped_gemm_int8(off, a, B.pack_int8(w, path=path)[1], one, a_scales=torch.ones(rows, device=DEV),
                                 out_dtype=torch.float32, path=path)
    want = torch.full((rows, 8), float(Kd * 16384), device=DEV)      # fp32 rounds it once, as the definition does
    want[:, 1] = -float(Kd * 128 * 127)
    assert torch.equal(out, want)


# Products large enough for the tile kernel of the small path, with and without a
# split inner dimension, at widths and depths that end inside a tile.
TILES = [dict(rows=130, E=1, N=1000, Kd=5008, bias=True), dict(rows=64, E=1, N=520, Kd=16400, a="bf16"),
         dict(rows=65, E=1, N=1032, Kd=8208), dict(rows=200, E=3, N=1000, Kd=2512, bias=True),
         dict(rows=500, E=40, N=392, Kd=2608, a="bf16"), dict(rows=17, E=1, N=8200, Kd=4000),
         dict(rows=300, E=3, N=264, Kd=7168, counts=[0, 290, 7], a="bf16")]


@pytest.mark.parametrize("kw", TILES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_tiles(B, kw):
    assert kw["rows"] * kw["N"] * kw["Kd"] > 4.8e8 and kw["rows"] > 8 * kw["E"]
    for path in ("small", "auto"):
        for dtype in (torch.bfloat16, torch.float32):
            check(B, make(**kw), path, dtype)


# Each kernel for tiles, on whole and on split inner dimensions, with more tiles than the GPU
# takes at once (groups much larger than the others), and rows that end anywhere in a tile.
KERNELS = [dict(rows=60, E=3, N=5000, Kd=400), dict(rows=37, E=1, N=1000, Kd=7184), dict(rows=64, E=1, N=4104, Kd=2064),
           dict(rows=50, E=1, N=7168, Kd=2048), dict(rows=1000, E=40, N=520, Kd=528), dict(rows=2400, E=40, N=520, Kd=272),
           dict(rows=127, E=1, N=1024, Kd=8192), dict(rows=250, E=1, N=3080, Kd=4112), dict(rows=129, E=1, N=264, Kd=2048),
           dict(rows=512, E=16, N=128, Kd=4096, counts=[0, 301, 1, 2] + [17] * 12),
           dict(rows=320, E=10, N=1920, Kd=336, counts=[211, 65, 1] + [6] * 7),
           dict(rows=1536, E=16, N=256, Kd=4096, counts=[129, 1, 900] + [33] * 13)]


@pytest.mark.parametrize("kw", KERNELS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "counts"))
def test_tile_kernels(B, kw):
    for a in ("int8", "bf16"):
        for bias, dtype in ((False, torch.bfloat16), (True, torch.float32)):
            check(B, make(a=a, bias=bias, **kw), "small", dtype)


def test_split_tiles_in_graphs_and_on_two_streams(B):
    """Calls whose CTAs share tiles, one after another in a graph and at once on two streams."""
    sets = []
    for i in range(2):
        d = make(64, 1, 1024, 8192, seed=i)
        sets.append((d, B.pack_int8(d["w"])[1], reference(d, torch.bfloat16)[0], torch.cuda.Stream(),
                     [torch.empty(64, 1024, dtype=torch.bfloat16, device=DEV) for _ in range(12)]))
    torch.cuda.synchronize()
    graphs = []
    for d, packed, want, stream, outs in sets:
        with torch.cuda.stream(stream):
            _, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], out=outs[0])
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            for o in outs:
                B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], out=o, ws=ws)
        graphs.append((g, ws))
    for _ in range(5):
        for _, _, _, _, outs in sets:
            for o in outs:
                o.fill_(7.0)
        torch.cuda.synchronize()
        for (g, _), (_, _, _, stream, _) in zip(graphs, sets):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for d, packed, want, _, outs in sets:
            assert all(torch.equal(o, want) for o in outs)
    assert all(B.read_device_status(ws) == 0 for _, ws in graphs)


def test_tiles_sums_are_exact(B):
    for rows in (64, 128):
        check(B, make(rows, 1, 1024, 8192, extreme=True), "small", torch.float32)


def test_split_tiles_clear_their_counters(B):
    """CTAs that share a tile's inner dimension: the same bits whatever the workspace held."""
    d = make(64, 1, 1024, 8192)
    _, packed = B.pack_int8(d["w"], path="small")
    ref, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], path="small")
    want, _ = reference(d, torch.bfloat16)
    assert torch.equal(ref, want)
    for fill in (0, 1, 0xff):
        ws.fill_(fill)
        for _ in range(20):
            got, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], a_scales=d["as_"], ws=ws,
                                         path="small")
        assert torch.equal(got, want)


def test_tiles_store_in_bounds_and_keep_nan(B):
    for rows, N, Kd in ((130, 1000, 5008), (64, 1032, 8208)):
        d = make(rows, 1, N, Kd, a="bf16")
        _, packed = B.pack_int8(d["w"], path="small")
        ref, ws = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path="small")
        whole = torch.full(((rows + 32) * N,), 0x5A5A, dtype=torch.int16, device=DEV)
        out = whole[16 * N:(16 + rows) * N].view(torch.bfloat16).view(rows, N)
        need = ws.numel()
        owner = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        at = (-owner.data_ptr()) % 1024 + 1024
        B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path="small", out=out, ws=owner[at:at + need])
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert bool((whole[:16 * N] == 0x5A5A).all()) and bool((whole[(16 + rows) * N:] == 0x5A5A).all())
        assert bool((owner[:at] == 0xA5).all()) and bool((owner[at + need:] == 0xA5).all())
        d["a"][7, 3] = float("nan")
        got, _ = B.grouped_gemm_int8(d["off"], d["a"], packed, d["ws"], path="small")
        rest = [r for r in range(rows) if r != 7]
        assert bool(torch.isnan(got[7]).all()) and torch.equal(got[rest], ref[rest])
