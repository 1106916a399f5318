"""Refusals of the fp8 expert path's entry points: every bad argument is
reported on the host before any launch (fake device addresses, no GPU), and
the binding's own checks of types and shapes."""
import ctypes

import pytest
import torch

NULLPTR, PARAM, SHAPE, WORKSPACE, ALIGN = 161001, 161002, 561002, 561003, 561004

# fake addresses: only where no kernel could ever be handed one
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only checks")
A = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def B():
    from combine_route_count_prefix_gb300 import build as b
    b.build()
    from combine_route_count_prefix_gb300 import binding
    binding.lib()
    return binding


def norm(B, T=4, H=128, x=A, residual=None, w=A, wd=0, eps=1e-6, ro=None, y=A, q=None, s=None):
    return B.lib().moe_add_rms_norm(T, H, x, residual, w, wd, eps, ro, y, q, s, None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(H=4), SHAPE), (dict(H=132), SHAPE), (dict(H=16392), SHAPE), (dict(T=-1), SHAPE),
    (dict(wd=2), PARAM), (dict(eps=0.0), PARAM), (dict(eps=float("nan")), PARAM),
    (dict(eps=float("inf")), PARAM), (dict(ro=A), PARAM),
    (dict(x=None), NULLPTR), (dict(w=None), NULLPTR), (dict(y=None), NULLPTR),
    (dict(q=A), NULLPTR), (dict(s=A), NULLPTR),
    (dict(x=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(residual=MIS), ALIGN),
    (dict(q=A, s=MIS), ALIGN), (dict(T=0, x=None, y=None), 0),
])
def test_norm(B, kw, code):
    assert norm(B, **kw) == code


def gate(B, logits=A, ids=A, scales=A, bias=None, mask=None, rm=None, desc=True, **kw):
    d = dict(num_tokens=4, num_experts=64, topk=8, num_groups=8, topk_groups=4, logits_stride=64,
             logits_dtype=0, score=1, group_score=1, renormalize=1, scale=1.0, reserved=0) | kw
    p = ctypes.byref(B.MoeGateDesc(**d)) if desc else None
    return B.lib().moe_gate(p, logits, bias, mask, ids, scales, rm, None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(desc=False), NULLPTR), (dict(num_experts=0), SHAPE), (dict(num_experts=1025, num_groups=1, topk_groups=1, logits_stride=2000), SHAPE),
    (dict(topk=17, topk_groups=8), SHAPE), (dict(topk=0), SHAPE), (dict(num_groups=7), SHAPE),
    (dict(num_groups=0), SHAPE), (dict(topk_groups=9), SHAPE), (dict(topk_groups=0), SHAPE),
    (dict(topk=9, topk_groups=1), SHAPE), (dict(logits_stride=63), SHAPE), (dict(num_tokens=-1), SHAPE),
    (dict(num_tokens=1 << 31), SHAPE), (dict(num_tokens=1 << 60), SHAPE),
    (dict(logits_dtype=2), PARAM), (dict(score=2), PARAM), (dict(group_score=-1), PARAM),
    (dict(renormalize=2), PARAM), (dict(reserved=1), PARAM), (dict(scale=float("nan")), PARAM),
    (dict(logits=None), NULLPTR), (dict(ids=None), NULLPTR), (dict(scales=None), NULLPTR),
    (dict(logits=MIS), ALIGN), (dict(bias=MIS), ALIGN), (dict(ids=MIS), ALIGN),
    (dict(scales=MIS), ALIGN), (dict(num_tokens=0, logits=None, ids=None, scales=None), 0),
])
def test_gate(B, kw, code):
    assert gate(B, **kw) == code


def gemm(B, rows=16, E=2, N=128, Kd=128, off=A, a=A, sa=A, w=A, sw=A, c=A, od=1, path=0, ws=A,
         ws_bytes=1 << 30):
    return B.lib().moe_grouped_gemm_fp8(rows, E, N, Kd, off, a, sa, w, sw, c, od, path, ws,
                                        ctypes.c_size_t(ws_bytes), None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(N=12), SHAPE), (dict(Kd=24), SHAPE), (dict(Kd=8), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(rows=-1), SHAPE), (dict(N=(1 << 20) + 8), SHAPE),
    (dict(Kd=131088), SHAPE), (dict(rows=1 << 31), SHAPE),
    (dict(od=2), PARAM), (dict(path=4), PARAM), (dict(path=-1), PARAM),
    (dict(off=None), NULLPTR), (dict(a=None), NULLPTR), (dict(sa=None), NULLPTR),
    (dict(w=None), NULLPTR), (dict(sw=None), NULLPTR), (dict(c=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(a=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(c=MIS), ALIGN), (dict(sa=MIS), ALIGN),
    (dict(ws=ctypes.c_void_p((1 << 20) + 512)), ALIGN), (dict(ws_bytes=16), WORKSPACE),
    (dict(rows=0, a=None, sa=None, c=None), 0),
])
def test_gemm(B, kw, code):
    assert gemm(B, **kw) == code


def ffn(B, shape=None, x=A, xs=A, assist=A, off=A, w1=A, s1=A, w2=A, s2=A, y=A, ws=A, ws_bytes=1 << 40):
    s = shape or B.make_shape(16, 2, 128, 8, 2, 256)
    return B.lib().moe_grouped_ffn_fp8(ctypes.byref(s), x, xs, assist, off, w1, s1, w2, s2, y, ws,
                                       ctypes.c_size_t(ws_bytes), None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULLPTR), (dict(xs=None), NULLPTR), (dict(off=None), NULLPTR),
    (dict(w1=None), NULLPTR), (dict(s2=None), NULLPTR), (dict(y=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(x=MIS), ALIGN), (dict(w2=MIS), ALIGN), (dict(y=MIS), ALIGN),
    (dict(assist=MIS), ALIGN), (dict(xs=MIS), ALIGN), (dict(ws=MIS), ALIGN),
])
def test_ffn(B, kw, code):
    assert ffn(B, **kw) == code


@host_only
def test_ffn_shapes_and_workspace(B):
    for bad in (B.make_shape(16, 2, 128, 8, 2, 0), B.make_shape(16, 2, 128, 8, 2, 128),
                B.make_shape(16, 2, 136, 8, 2, 256), B.make_shape(16, 3, 128, 8, 2, 256)):
        assert ffn(B, shape=bad) == SHAPE
        with pytest.raises(B.MoeError):
            B.grouped_ffn_fp8_workspace_size(bad)
    s = B.make_shape(16, 2, 128, 8, 2, 256)
    need = B.grouped_ffn_fp8_workspace_size(s)
    assert ffn(B, shape=s, ws_bytes=need - 1) == WORKSPACE
    empty = B.make_shape(0, 1, 128, 8, 2, 256)
    assert ffn(B, shape=empty, x=None, xs=None, assist=None, y=None) == 0


def test_binding_checks(B):
    """Types, shapes and places that the binding refuses before the library sees them."""
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    x, w = torch.zeros(4, 128, dtype=bf), torch.zeros(128)
    with pytest.raises(TypeError):
        B.add_rms_norm(x.float(), w)
    with pytest.raises(TypeError):
        B.add_rms_norm(x, w.double())
    with pytest.raises(ValueError):
        B.add_rms_norm(x, w)                              # not on the GPU
    with pytest.raises(ValueError):
        B.add_rms_norm(x, w, residual=torch.zeros(4, 64, dtype=bf))
    with pytest.raises(ValueError):
        B.add_rms_norm(torch.zeros(128, 4, dtype=bf).t(), w)
    with pytest.raises(TypeError):
        B.gate(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        B.gate(torch.zeros(4, 8), 2)                      # not on the GPU
    off = torch.zeros(3, dtype=torch.int32)
    a, sa = torch.zeros(4, 256).to(f8), torch.zeros(4, 2)
    wt, sw = torch.zeros(2, 128, 256).to(f8), torch.zeros(2, 1, 2)
    with pytest.raises(TypeError):
        B.grouped_gemm_fp8(off, a.float(), sa, wt, sw)
    with pytest.raises(ValueError):
        B.grouped_gemm_fp8(off, a, sa[:, :1], wt, sw)
    with pytest.raises(ValueError):
        B.grouped_gemm_fp8(off, a, sa, wt, sw)
    s = B.make_shape(4, 1, 256, 2, 1, 256)
    with pytest.raises(ValueError):
        B.grouped_ffn_fp8(s, a, sa, off, wt, sw, wt, sw)
