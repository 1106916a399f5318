"""A call's tensors have to be on one GPU, the current one, and what the
library remembers of a kernel is kept per GPU.  No GPU needed: the tensors here
only report where they are, and nothing is launched."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F8, BF, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


class Somewhere:
    """What the binding asks of a tensor, on GPU `at`."""

    def __init__(self, shape, dtype, at=0):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at
        self.is_cuda, self.device = True, torch.device("cuda", at)

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def stride(self, d):
        return 1 if d == len(self.shape) - 1 else int(self.shape[-1])

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1 << 40


class Stream:
    def __init__(self, at=0):
        self.device_index, self.cuda_stream = at, 0


@pytest.fixture
def B(monkeypatch):
    from combine_route_count_prefix_gb300 import binding
    calls = []
    monkeypatch.setattr(binding, "_call", lambda *a: calls.append(a[0]))
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "called", calls, raising=False)
    return binding


def t(*shape, dtype=F32):
    return Somewhere(shape, dtype)


def norm_args():
    return dict(x=t(4, 256, dtype=BF), weight=t(256), residual=t(4, 256, dtype=BF),
                out=dict(residual_out=t(4, 256, dtype=BF), y=t(4, 256, dtype=BF),
                         q=t(4, 256, dtype=F8), scales=t(4, 2)))


def gate_args():
    return dict(logits=t(4, 64), topk=2, bias=t(64), mask=t(4, dtype=torch.uint8),
                out=dict(expert_ids=t(4, 2, dtype=I32), expert_scales=t(4, 2),
                         route_mask=t(4, 2, dtype=torch.uint8)))


def gemm_args():
    return dict(expert_offsets=t(3, dtype=I32), a=t(4, 256, dtype=F8), a_scales=t(4, 2),
                w=t(2, 128, 256, dtype=F8), w_scales=t(2, 1, 2), out=t(4, 128),
                ws=t(4096, dtype=torch.uint8))


def ffn_args():
    return dict(x=t(4, 256, dtype=F8), x_scales=t(4, 2), expert_offsets=t(3, dtype=I32),
                w1=t(2, 256, 256, dtype=F8), w1_scales=t(2, 2, 2), w2=t(2, 256, 128, dtype=F8),
                w2_scales=t(2, 2, 1), assist=t(4, 3, dtype=I32), y=t(4, 256, dtype=BF),
                ws=t(4096, dtype=torch.uint8))


def call(B, name, kw):
    if name == "grouped_ffn_fp8":
        kw = dict(kw, shape=B.make_shape(4, 1, 256, 2, 1, 256))
    return getattr(B, name)(**dict(dict(stream=Stream()), **kw))


OPS = dict(add_rms_norm=norm_args, gate=gate_args, grouped_gemm_fp8=gemm_args,
           grouped_ffn_fp8=ffn_args)


def tensors(kw):
    """(path to) every tensor of the arguments."""
    for k, v in kw.items():
        if isinstance(v, Somewhere):
            yield k, v
        elif isinstance(v, dict):
            yield from ((f"{k}.{n}", u) for n, u in v.items())


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_the_current_gpu_are_taken(B, op):
    call(B, op, OPS[op]())
    assert len(B.called) == 1


@pytest.mark.parametrize("op,path", [(op, p) for op, f in OPS.items() for p, _ in tensors(f())])
def test_one_tensor_on_another_gpu_is_refused(B, op, path):
    kw = OPS[op]()
    dict(tensors(kw))[path].at = 1
    with pytest.raises(ValueError, match="cuda:"):
        call(B, op, kw)
    assert not B.called


@pytest.mark.parametrize("op", OPS)
def test_all_on_another_gpu_than_the_current_one_are_refused(B, op):
    kw = OPS[op]()
    for _, v in tensors(kw):
        v.at = 1
    with pytest.raises(ValueError, match="current device"):
        call(B, op, kw)
    assert not B.called


@pytest.mark.parametrize("op", OPS)
def test_a_stream_of_another_gpu_is_refused(B, op):
    with pytest.raises(ValueError, match="stream"):
        call(B, op, dict(OPS[op](), stream=Stream(1)))
    assert not B.called


def test_dispatch_and_combine_refuse_another_gpu(B):
    """The calls without a device of their own compare with the current one."""
    out = dict(expand_x=t(8, 64, dtype=BF), assist=t(8, 3, dtype=I32), expert_token_nums=None,
               expert_offsets=None, ep_recv_counts=None, route_row=t(8, dtype=I32))
    kw = dict(x=t(4, 64, dtype=BF), expert_ids=t(4, 2, dtype=I32), num_experts=8, num_partitions=1,
              ws=t(4096, dtype=torch.uint8), out=out, stream=Stream())
    B.dispatch(**kw)
    assert len(B.called) == 1
    kw["x"].at = 1
    with pytest.raises(ValueError, match="cuda:1"):
        B.dispatch(**kw)
    kw = dict(expand_x=t(8, 64, dtype=BF), route_row=t(8, dtype=I32), expert_scales=t(4, 2),
              num_experts=8, num_partitions=1, out=t(4, 64, dtype=BF), stream=Stream())
    B.combine(**kw)
    kw["expert_scales"].at = 1
    with pytest.raises(ValueError, match="cuda:1"):
        B.combine(**kw)
    assert len(B.called) == 2


LIMITS = r"""
#include "limits.cuh"
#include <cstdio>
int main() {
    moe::RaisedLimits r;
    int calls = 0;
    bool grant = true;
    auto raise = [&] { ++calls; return grant; };
    int k1, k2;
    auto expect = [&](int device, const void *k, size_t bytes, bool ok, int n) {
        const bool got = r.ensure(device, k, bytes, raise);
        if (got != ok || calls != n)
            printf("device %d bytes %zu: %d after %d calls\n", device, bytes, got, calls);
    };
    expect(0, &k1, 100, true, 1);
    expect(0, &k1, 100, true, 1);      // known
    expect(1, &k1, 100, true, 2);      // another device: raised there too
    expect(1, &k1, 60, true, 2);
    expect(0, &k2, 60, true, 3);       // another kernel
    expect(0, &k1, 200, true, 4);      // more than before, on this device alone
    expect(1, &k1, 200, true, 5);
    grant = false;
    expect(2, &k1, 10, false, 6);      // a refusal is not remembered
    grant = true;
    expect(2, &k1, 10, true, 7);
    return 0;
}
"""


def test_limits_are_kept_per_device(tmp_path):
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(LIMITS)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "combine_route_count_prefix_gb300", "csrc"), str(src), "-o",
                    str(exe), "-pthread"], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == ""
