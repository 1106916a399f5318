"""block_norm's gates and factors (tensors that only report where they are, nothing is launched)."""
import math

import pytest

from test_devices import BF, t
from test_devices import B as fake  # noqa: F401  (a binding that launches nothing)
from test_int8_refusals import call, gate, norm_args


def args(T, G):
    kw = dict(norm_args(), gate=gate(G, 256), x=t(T, 256, dtype=BF), residual=t(T, 256, dtype=BF))
    kw["out"] = dict(residual_out=t(T, 256, dtype=BF))
    return kw


@pytest.mark.parametrize("T,G", [(0, 0), (0, 1), (0, 3), (4, 1), (4, 4)])
def test_gates_of_a_batch(fake, T, G):  # noqa: F811
    """A batch may be empty whatever the gate's rows."""
    call(fake, "block_norm", args(T, G))
    assert fake.called == ["moe_block_norm"]


def test_tokens_need_a_gate_row(fake):  # noqa: F811
    with pytest.raises(ValueError, match="gate"):
        call(fake, "block_norm", args(4, 0))
    assert not fake.called


@pytest.mark.parametrize("name", ["residual_scale", "branch_scale"])
def test_zeros_of_either_sign_reach_the_call(fake, name, monkeypatch):  # noqa: F811
    seen = []
    monkeypatch.setattr(fake, "_call", lambda entry, desc, *a: seen.append(math.copysign(1.0, getattr(desc, name))))
    for v in (0.0, -0.0, 0.0, -0.0):
        call(fake, "block_norm", dict(args(4, 1), **{name: v}))
    assert seen == [1.0, -1.0, 1.0, -1.0]
