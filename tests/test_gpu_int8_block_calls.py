"""Calls of the int8 block of examples/ that its documentation allows: a length first met in a
graph's capture, no tokens, and which layer a call takes."""
import pytest
import torch

from test_gpu_int8_block import ex, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 150])
def test_a_length_first_met_in_a_capture(ex, T):  # noqa: F811
    block = ex.random_block(512, 512, 16, 4, 512, seed=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(*inputs(5, 512, 512, 0)[:2])          # another length: libraries and kernels are loaded
    torch.cuda.current_stream().wait_stream(side)
    static = inputs(T, 512, 512, 1)[:2]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(*static)
    for seed in (2, 3):
        new = inputs(T, 512, 512, seed)[:2]
        for s, n in zip(static, new):
            s.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got_now = [v.clone() for v in got]
        # without the graph, after it has run and on memory of its own
        for a, b in zip(got_now, block(*new)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_no_tokens(ex):  # noqa: F811
    block = ex.random_block(512, 512, 16, 4, 512, seed=7)
    for v in block(*inputs(0, 512, 512, 0)[:2]):
        assert v.shape == (0, 512)


@pytest.mark.parametrize("T,E,K,few", [(1, 16, 4, True), (64, 16, 4, True), (65, 16, 4, False), (128, 64, 4, True),
                                       (129, 64, 4, False)])
def test_the_layer_that_is_faster(ex, T, E, K, few, monkeypatch):  # noqa: F811
    """The few-token layer up to its 512 routes, and up to 16 an expert."""
    block = ex.random_block(512, 512, E, K, 256, seed=7)
    used = []
    for name in ("layer", "layer_few_tokens"):
        def wrap(*a, name=name, real=getattr(ex.B, name), **kw):
            used.append(name)
            return real(*a, **kw)
        monkeypatch.setattr(ex.B, name, wrap)
    block(*inputs(T, 512, 512, 0)[:2])
    assert used == ["layer_few_tokens" if few else "layer"]
