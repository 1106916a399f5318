"""moe_layer_few_tokens_y: which types an expert's output may have before the weighted
sum (fake device addresses, no GPU)."""
import ctypes

import pytest
import torch

from test_devices import B as fake  # noqa: F401  (a binding that launches nothing)
from test_int8_refusals import A, B, MIS, NULLPTR, PARAM, SHAPE, WORKSPACE, call, host_only, layer_args  # noqa: F401


def layer(B, y_dtype, x=A, ids=A, ws_bytes=1 << 40, **kw):  # noqa: F811
    s = B.make_shape(**(dict(T=4, P=1, H=128, E=8, K=2, N=256, ffn_path="small") | kw))
    return B.lib().moe_layer_few_tokens_y(ctypes.byref(s), y_dtype, x, ids, A, None, None, A, A, A, A, A, A,
                                          ctypes.c_size_t(ws_bytes), None)


@host_only
@pytest.mark.parametrize("y_dtype,kw,code", [
    (2, {}, PARAM), (3, {}, PARAM), (-1, {}, PARAM), (0, dict(T=257), SHAPE), (0, dict(x=None), NULLPTR),
    (0, dict(ws_bytes=1024), WORKSPACE), (0, dict(ffn_path="large"), PARAM), (1, dict(ids=None), NULLPTR),
    (2, dict(T=0, x=None, ids=None), PARAM),
])
def test_refusals(B, y_dtype, kw, code):  # noqa: F811
    assert layer(B, y_dtype, **kw) == code


def test_each_type_has_its_entry_point(fake):  # noqa: F811
    call(fake, "layer_few_tokens", layer_args())
    call(fake, "layer_few_tokens", dict(layer_args(), y_dtype=torch.bfloat16))
    call(fake, "layer_few_tokens", dict(layer_args(), y_dtype=torch.float32))
    assert fake.called == ["moe_layer_few_tokens"] * 2 + ["moe_layer_few_tokens_y"]
    with pytest.raises(TypeError, match="y_dtype"):
        call(fake, "layer_few_tokens", dict(layer_args(), y_dtype=torch.float16))
    assert len(fake.called) == 3
