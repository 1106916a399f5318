"""Refusals of moe_layer_few_tokens, moe_pack_int8, moe_grouped_gemm_int8 and
moe_block_norm: every bad argument is reported on the host before any launch
(fake device addresses, no GPU), and the binding's own checks of types, shapes
and places."""
import ctypes

import pytest
import torch

from test_devices import BF, F32, F8, I32, Stream, t, tensors
from test_devices import B as fake  # noqa: F401  (a binding that launches nothing)

NULLPTR, PARAM, SHAPE, WORKSPACE, ALIGN = 161001, 161002, 561002, 561003, 561004

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only checks")
A = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 2)
OFF16 = ctypes.c_void_p((1 << 20) + 16)
I8, U8 = torch.int8, torch.uint8


@pytest.fixture(scope="module")
def B():
    from combine_route_count_prefix_gb300 import build as b
    b.build()
    from combine_route_count_prefix_gb300 import binding
    binding.lib()
    return binding


# ------------------------------------------------------------------ the layer

def layer(B, shape=None, x=A, ids=A, probs=A, mask=None, shared=None, w1=A, s1=A, w2=A, s2=A, out=A,
          ws=A, ws_bytes=1 << 40, **kw):
    s = shape or B.make_shape(**(dict(T=4, P=1, H=128, E=8, K=2, N=256, ffn_path="small") | kw))
    return B.lib().moe_layer_few_tokens(ctypes.byref(s), x, ids, probs, mask, shared, w1, s1, w2, s2, out,
                                        ws, ctypes.c_size_t(ws_bytes), None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(T=257), SHAPE), (dict(T=513, K=1), SHAPE), (dict(T=1 << 40), SHAPE), (dict(T=-1), SHAPE),
    (dict(N=0), SHAPE), (dict(N=128), SHAPE), (dict(N=8448), SHAPE), (dict(H=136), SHAPE),
    (dict(H=8208), SHAPE), (dict(E=1025), SHAPE), (dict(K=17), SHAPE),
    (dict(ffn_path="large"), PARAM), (dict(ffn_path="large_pair"), PARAM),
    (dict(x=None), NULLPTR), (dict(ids=None), NULLPTR), (dict(probs=None), NULLPTR),
    (dict(w1=None), NULLPTR), (dict(s1=None), NULLPTR), (dict(w2=None), NULLPTR), (dict(s2=None), NULLPTR),
    (dict(out=None), NULLPTR), (dict(ws=None), NULLPTR), (dict(mask_kind=1), NULLPTR),
    (dict(mask=A), PARAM), (dict(has_shared=True), NULLPTR), (dict(shared=A), PARAM),
    (dict(x=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(ids=MIS), ALIGN), (dict(probs=MIS), ALIGN),
    (dict(w1=OFF16), ALIGN), (dict(w2=OFF16), ALIGN), (dict(ws=OFF16), ALIGN), (dict(s1=MIS), ALIGN),
    (dict(s2=MIS), ALIGN), (dict(has_shared=True, shared=MIS), ALIGN), (dict(ws_bytes=1024), WORKSPACE),
    (dict(T=0, x=None, ids=None, probs=None, out=None), 0),
])
def test_layer(B, kw, code):
    assert layer(B, **kw) == code


@host_only
def test_layer_workspace(B):
    s = B.make_shape(64, 1, 7168, 128, 8, 4096, ffn_path="small")
    need = B.layer_few_tokens_workspace_size(s)
    assert 512 * 2048 * 4 <= need < 8 << 20
    assert layer(B, shape=s, ws_bytes=need - 1) == WORKSPACE
    with pytest.raises(B.MoeError):
        B.layer_few_tokens_workspace_size(B.make_shape(64, 1, 7168, 128, 9, 4096, ffn_path="small"))


# ------------------------------------------------------------------ the product

def gemm(B, rows=16, E=2, N=128, Kd=128, off=A, a=A, ad=2, sa=A, w=A, sw=A, bias=None, c=A, od=1, path=0,
         ws=A, ws_bytes=1 << 40):
    return B.lib().moe_grouped_gemm_int8(rows, E, N, Kd, off, a, ad, sa, w, sw, bias, c, od, path, ws,
                                         ctypes.c_size_t(ws_bytes), None)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(N=12), SHAPE), (dict(N=0), SHAPE), (dict(Kd=24), SHAPE), (dict(Kd=0), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(rows=-1), SHAPE), (dict(N=(1 << 20) + 8), SHAPE), (dict(Kd=131072), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 24, Kd=131056), SHAPE),
    (dict(ad=0), PARAM), (dict(ad=3), PARAM), (dict(od=2), PARAM), (dict(path=4), PARAM), (dict(path=-1), PARAM),
    (dict(ad=1), PARAM),                                  # bf16 rows with scales
    (dict(off=None), NULLPTR), (dict(a=None), NULLPTR), (dict(sa=None), NULLPTR), (dict(w=None), NULLPTR),
    (dict(sw=None), NULLPTR), (dict(c=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(a=MIS), ALIGN), (dict(c=MIS), ALIGN), (dict(od=0, c=OFF16), ALIGN), (dict(sa=MIS), ALIGN),
    (dict(sw=MIS), ALIGN), (dict(bias=MIS), ALIGN), (dict(off=MIS), ALIGN), (dict(w=OFF16), ALIGN),
    (dict(ws=OFF16), ALIGN), (dict(ws_bytes=16), WORKSPACE),
    (dict(rows=0, a=None, sa=None, c=None), 0), (dict(rows=0, a=None, ad=1, sa=None, c=None), 0),
])
def test_gemm(B, kw, code):
    assert gemm(B, **kw) == code


@host_only
@pytest.mark.parametrize("args,code", [
    ((1, 12, 128, 0, A, A), SHAPE), ((1, 128, 8, 0, A, A), SHAPE), ((0, 128, 128, 0, A, A), SHAPE),
    ((1, 128, 128, 4, A, A), PARAM), ((1, 128, 128, 0, None, A), NULLPTR), ((1, 128, 128, 0, A, None), NULLPTR),
    ((1, 128, 128, 0, MIS, A), ALIGN), ((1, 128, 128, 0, A, OFF16), ALIGN),
])
def test_pack(B, args, code):
    assert B.lib().moe_pack_int8(*args, None) == code


@host_only
def test_packed_bytes(B):
    assert B.int8_packed_bytes(2, 136, 144, "small") == 2 * 136 * 144
    assert B.int8_packed_bytes(2, 136, 144, "large") == -(-2 * 136 * 144 * 2 // 1024) * 1024
    assert B.int8_packed_bytes(2, 136, 144) == B.int8_packed_bytes(2, 136, 144, "large") + 2 * 136 * 144
    for bad in ((0, 128, 128), (1, 12, 128), (1, 128, 24)):
        with pytest.raises(B.MoeError):
            B.int8_packed_bytes(*bad)


# ------------------------------------------------------------------ the norm

def norm(B, x=A, residual=A, post=None, gate=None, w=A, ro=A, y=A, q=None, s=None, desc=True, **kw):
    d = dict(num_tokens=4, hidden=128, gate_rows=0, gate_stride=0, weight_dtype=0, gate_act=0,
             residual_scale=1.0, branch_scale=1.0, eps=1e-6, reserved=0) | kw
    p = ctypes.byref(B.MoeBlockNormDesc(**d)) if desc else None
    return B.lib().moe_block_norm(p, x, residual, post, gate, w, ro, y, q, s, None)


G = dict(gate=A, gate_rows=2, gate_stride=128)


@host_only
@pytest.mark.parametrize("kw,code", [
    (dict(desc=False), NULLPTR), (dict(hidden=4), SHAPE), (dict(hidden=132), SHAPE), (dict(hidden=16392), SHAPE),
    (dict(num_tokens=-1), SHAPE), (dict(num_tokens=1 << 31), SHAPE), (dict(weight_dtype=2), PARAM),
    (dict(gate_act=2), PARAM), (dict(reserved=1), PARAM), (dict(eps=0.0), PARAM),
    (dict(eps=float("inf")), PARAM), (dict(residual_scale=float("nan")), PARAM),
    (dict(branch_scale=float("inf")), PARAM), (dict(gate=A), PARAM),
    (dict(G, gate=None), NULLPTR), (dict(G, gate_rows=3), SHAPE), (dict(G, gate_rows=8), SHAPE),
    (dict(G, gate_rows=-1), SHAPE), (dict(G, gate_stride=64), SHAPE), (dict(G, gate_stride=132), SHAPE),
    (dict(G, gate_stride=0), SHAPE), (dict(gate_stride=128), SHAPE),
    (dict(w=None), NULLPTR), (dict(w=None, y=None, q=A, s=A), NULLPTR), (dict(x=None), NULLPTR),
    (dict(residual=None), NULLPTR), (dict(ro=None), NULLPTR), (dict(q=A), NULLPTR), (dict(s=A), NULLPTR),
    (dict(x=MIS), ALIGN), (dict(residual=MIS), ALIGN), (dict(post=MIS), ALIGN), (dict(G, gate=MIS), ALIGN),
    (dict(w=MIS), ALIGN), (dict(ro=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(q=MIS, s=A), ALIGN),
    (dict(q=A, s=MIS), ALIGN), (dict(num_tokens=0, x=None, residual=None, ro=None, y=None), 0),
])
def test_norm(B, kw, code):
    assert norm(B, **kw) == code


# ------------------------------------------------------------------ the binding

def layer_args():
    return dict(x=t(4, 256, dtype=BF), expert_ids=t(4, 2, dtype=I32), expert_scales=t(4, 2),
                w1p=t(2 * 256 * 256, dtype=U8), scale1=t(2, 256), w2p=t(2 * 256 * 128, dtype=U8),
                scale2=t(2, 256), mask=t(4, dtype=U8), shared=t(4, 256, dtype=BF),
                out=t(4, 256, dtype=BF), ws=t(4096, dtype=U8))


def gemm_args():
    return dict(expert_offsets=t(3, dtype=I32), a=t(4, 256, dtype=I8), a_scales=t(4),
                w_packed=t(2 * 128 * 256, dtype=U8), w_scales=t(2, 128), bias=t(2, 128), out=t(4, 128),
                ws=t(4096, dtype=U8))


def norm_args():
    return dict(x=t(4, 256, dtype=BF), residual=t(4, 256, dtype=BF), weight=t(256), post_weight=t(256),
                gate=gate(2, 256), out=dict(residual_out=t(4, 256, dtype=BF), y=t(4, 256, dtype=BF),
                                            q=t(4, 256, dtype=F8), scales=t(4, 2)))


def gate(*shape):
    g = t(*shape, dtype=BF)
    g.dim = lambda: len(shape)
    return g


OPS = dict(layer_few_tokens=layer_args, grouped_gemm_int8=gemm_args, block_norm=norm_args)


def call(B, name, kw):
    if name == "layer_few_tokens":
        kw = dict(kw, shape=B.make_shape(4, 1, 256, 2, 2, 256, mask_kind=1, has_shared=True, ffn_path="small"))
    if name == "grouped_gemm_int8":
        kw = dict(kw, path="small")
    return getattr(B, name)(**dict(dict(stream=Stream()), **kw))


@pytest.fixture
def F(fake, monkeypatch):  # noqa: F811
    monkeypatch.setattr(fake, "int8_packed_bytes", lambda E, N, Kd, path="auto": E * N * Kd)
    return fake


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_the_current_gpu_are_taken(F, op):
    call(F, op, OPS[op]())
    assert len(F.called) == 1


@pytest.mark.parametrize("op,path", [(op, p) for op, f in OPS.items() for p, _ in tensors(f())])
def test_one_tensor_on_another_gpu_is_refused(F, op, path):
    kw = OPS[op]()
    dict(tensors(kw))[path].at = 1
    with pytest.raises(ValueError, match="cuda:"):
        call(F, op, kw)
    assert not F.called


@pytest.mark.parametrize("op", OPS)
def test_another_gpu_or_stream_is_refused(F, op):
    kw = OPS[op]()
    for _, v in tensors(kw):
        v.at = 1
    with pytest.raises(ValueError, match="current device"):
        call(F, op, kw)
    with pytest.raises(ValueError, match="stream"):
        call(F, op, dict(OPS[op](), stream=Stream(1)))
    assert not F.called


@pytest.mark.parametrize("op,path", [(op, p) for op, f in OPS.items() for p, _ in tensors(f()) if p != "ws"])
def test_other_types_and_shapes_are_refused(F, op, path):
    kw = OPS[op]()
    v = dict(tensors(kw))[path]
    v.dtype = torch.float16
    with pytest.raises(TypeError):
        call(F, op, kw)
    kw = OPS[op]()
    v = dict(tensors(kw))[path]
    v.shape = torch.Size((*v.shape[:-1], v.shape[-1] + 1))
    with pytest.raises(ValueError):
        call(F, op, kw)
    assert not F.called


def test_scales_go_with_int8_rows(F):
    with pytest.raises(ValueError, match="a_scales"):
        call(F, "grouped_gemm_int8", dict(gemm_args(), a_scales=None))
    with pytest.raises(ValueError, match="a_scales"):
        call(F, "grouped_gemm_int8", dict(gemm_args(), a=t(4, 256, dtype=BF)))
    call(F, "grouped_gemm_int8", dict(gemm_args(), a=t(4, 256, dtype=BF), a_scales=None))
