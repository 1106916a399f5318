"""Calls of the fp8 MoE block of examples/ next to each other: they share
nothing but the weights."""
import importlib.util
import os

import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "fp8_moe_block.py")


@pytest.fixture(scope="module")
def block():
    load_binding()
    spec = importlib.util.spec_from_file_location("fp8_moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.random_block(1024, 16, 4, 512, 4, 2, seed=1)


def inputs(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(T, 1024, generator=g, device="cuda").bfloat16() for _ in range(2))


def test_streams_of_equal_length(block):
    """Two streams, many calls of the same length in flight on both."""
    args = [inputs(300, s) for s in range(2)]
    want = [block(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    # work in front of both, so that all the calls are queued before any begins
    busy = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(4):
                torch.mm(busy, busy)
    got = [[], []]
    for _ in range(30):
        for s, a, g in zip(streams, args, got):
            with torch.cuda.stream(s):
                g.append(block(*a))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for out in g:
            assert torch.equal(out.view(torch.int16), w.view(torch.int16))


def test_many_lengths_keep_no_memory(block):
    block(*inputs(8, 0))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in range(1, 200, 11):
        block(*inputs(T, T))
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before
