"""The fp8 path's calls where element offsets pass 32 bits, and inside a CUDA
graph: a row's results do not depend on where it lies, nor on how the call was
launched, so both are compared with small eager calls, bit for bit where the
sums' order is the same."""
import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
T, H = 310000, 7168          # T * H passes 2^31


@pytest.fixture(scope="module")
def B():
    return load_binding()


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def codes(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * 110.0).clamp(-448, 448).to(F8)


def scales(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * 0.01 + 1e-3


def same(a, b):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def tall(rows):
    """T rows that repeat `rows` [n, ...]."""
    n = rows.shape[0]
    u = rows.view(torch.uint8)
    return u.repeat(-(-T // n), 1)[:T].contiguous().view(rows.dtype)


def test_gate_rows_far_apart(B):
    """Rows 2^30 elements apart."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(4, 256, generator=g, device="cuda").bfloat16()
    stride = 2 ** 30 + 8
    far = torch.empty(3 * stride + 256, dtype=torch.bfloat16, device="cuda").as_strided((4, 256), (stride, 1))
    far.copy_(rows)
    for kw in (dict(), dict(score="sigmoid", groups=8, topk_groups=4, group_score="top2")):
        a, b = B.gate(far, 8, **kw), B.gate(rows, 8, **kw)
        for k in a:
            same(a[k], b[k])


def test_norm_of_many_tokens(B):
    g = torch.Generator(device="cuda").manual_seed(1)
    few = torch.randn(1024, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    x = tall(few)
    out = B.add_rms_norm(x, w, residual=x)
    for at in (0, T - 7):
        part = x[at:at + 7].contiguous()
        ref = B.add_rms_norm(part, w, residual=part)
        for k in ref:
            same(out[k][at:at + 7], ref[k])


@pytest.mark.parametrize("path", ["large_pair", "small"])
def test_product_of_many_rows(B, path):
    """Both A and C past 2^31 elements.  Few rows share their tiles' K between
    CTAs in the small form, so there the sums' order differs: two roundings to
    bf16, each within 2^-8, and fp32 sums that are nothing beside them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N = H
    a, s = tall(codes(g, 500, H)), tall(scales(g, 500, H // 128))
    w, ws = codes(g, 2, N, H), scales(g, 2, N // 128, H // 128)
    cut = T - 9
    out, _ = B.grouped_gemm_fp8(torch.tensor([0, cut, T], dtype=torch.int32, device="cuda"), a, s, w, ws,
                                path=path)
    for e, at in ((0, 0), (0, cut - 9), (1, cut)):
        off = torch.tensor([0, 9, 9] if e == 0 else [0, 0, 9], dtype=torch.int32, device="cuda")
        ref, _ = B.grouped_gemm_fp8(off, a[at:at + 9].contiguous(), s[at:at + 9].contiguous(), w, ws,
                                    path=path)
        if path == "large_pair":
            same(out[at:at + 9], ref)
        else:
            d = (out[at:at + 9].double() - ref.double()).norm()
            assert d <= (2.0 ** -7 + 2.0 ** -10) * ref.double().norm()


def test_ffn_of_many_tokens(B):
    g = torch.Generator(device="cuda").manual_seed(3)
    E, N = 2, 256
    x, xs = tall(codes(g, 500, H)), tall(scales(g, 500, H // 128))
    w = (codes(g, E, N, H), scales(g, E, 2, H // 128), codes(g, E, H, N // 2), scales(g, E, H // 128, 1))

    def run(x, xs, expert):
        t = x.shape[0]
        # every token to one expert: its rows are the tokens in order
        off = torch.tensor([0] * (expert + 1) + [t] * (E - expert), dtype=torch.int32, device="cuda")
        assist = torch.zeros(t, 3, dtype=torch.int32, device="cuda")
        assist[:, 1] = torch.arange(t, dtype=torch.int32, device="cuda")
        y, ws = B.grouped_ffn_fp8(B.make_shape(t, 1, H, E, 1, N, ffn_path="large_pair"), x, xs, off, *w,
                                  assist=assist)
        assert B.read_device_status(ws) == 0
        return y

    y = run(x, xs, 1)
    for at in (0, T - 9):
        same(y[at:at + 9], run(x[at:at + 9].contiguous(), xs[at:at + 9].contiguous(), 1))


def test_in_a_cuda_graph(B):
    """Every call captured once, replayed on other inputs."""
    g = torch.Generator(device="cuda").manual_seed(4)
    t, h, E, K, N = 40, 1024, 16, 4, 512
    x = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    r = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    nw = torch.randn(h, generator=g, device="cuda").bfloat16()
    logits = torch.randn(t, E, generator=g, device="cuda")
    w = (codes(g, E, N, h), scales(g, E, N // 128, h // 128), codes(g, E, h, N // 2),
         scales(g, E, h // 128, N // 256))
    off = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    shape = B.make_shape(t, 1, h, E, K, N)

    def block():
        n = B.add_rms_norm(x, nw, residual=r)
        route = B.gate(logits, K, score="sigmoid")
        d = B.dispatch(None, route["expert_ids"], E, 1, mask=route["route_mask"], with_rows=False)
        y, ws = B.grouped_ffn_fp8(shape, n["q"], n["scales"], d["expert_offsets"], *w, assist=d["assist"])
        c, _ = B.grouped_gemm_fp8(off, n["q"], n["scales"], w[0][:1], w[1][:1])
        out = B.combine(y, d["route_row"], route["expert_scales"], E, 1, mask=route["route_mask"],
                        shared=n["residual_out"])
        return out, c, route["expert_ids"], n["q"], (n, route, d, y, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    for _ in range(3):
        x.copy_(torch.randn(t, h, generator=g, device="cuda"))
        logits.copy_(torch.randn(t, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got[:4], block()[:4]):
            same(a, b)
