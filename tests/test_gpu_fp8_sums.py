"""moe_grouped_gemm_fp8 adds exact products in fp32: sums that need many bits.

Large products (448 x 448) come with small odd ones and leave again, in the
same block of 128, another instruction's part of it, and another block.  Every
partial sum in any order is a multiple of `unit` below 2^24 units, so 24 bits
hold all of them and the result is exact; fewer bits lose the small products
while a large one is in the sum."""
import numpy as np
import pytest
import torch

from gpu_util import load_binding

KD = 384
# (value, place in K) of the large factors of W; A's are 448 there
LARGE = [(448.0, 0), (-448.0, 127), (448.0, 130), (-448.0, 380)]
UNITS = [1.0, 2.0 ** -5]          # 18 and 23 bits below the largest partial sum


def case(unit, rows, N, seed):
    """A [rows, KD] and W [N, KD], all of them e4m3 numbers."""
    g = np.random.default_rng(seed)
    a = (2 * g.integers(0, 8, (rows, KD)) + 1.0) * (1.0 if unit == 1.0 else 0.25)
    w = (2 * g.integers(0, 8, (N, KD)) + 1.0) * (1.0 if unit == 1.0 else 0.125)
    w *= g.choice([-1.0, 1.0], w.shape)
    for v, k in LARGE:
        a[:, k], w[:, k] = 448.0, v
    return a, w


def narrow_sum(terms, bits):
    """32 products at a time and the sum so far, each cut to `bits` bits below
    the largest of them: what a narrow accumulator keeps of them."""
    acc = 0.0
    for i in range(0, terms.size, 32):
        t = np.append(terms[i:i + 32], acc)
        q = 2.0 ** (np.floor(np.log2(np.abs(t).max())) + 1 - bits)
        acc = float((np.trunc(t / q) * q).sum())
    return acc


@pytest.mark.parametrize("unit", UNITS)
def test_the_case_needs_the_bits(unit):
    a, w = case(unit, 4, 8, 0)
    assert torch.equal(torch.tensor(a).to(torch.float8_e4m3fn).double(), torch.tensor(a))
    assert torch.equal(torch.tensor(w).to(torch.float8_e4m3fn).double(), torch.tensor(w))
    p = a[:, None, :] * w
    assert np.all(p % unit == 0)
    # any partial sum of a block, and of the blocks' sums, fits 24 bits
    blocks = p.reshape(4, 8, 3, 128)
    assert np.abs(blocks).sum(3).max() < 2.0 ** 24 * unit
    assert np.abs(blocks.sum(3)).sum(2).max() < 2.0 ** 24 * unit
    ref = p.sum(2)
    for bits, exact in ((24, True), (16 if unit == 1.0 else 21, False), (14, False)):
        got = np.array([[narrow_sum(t, bits) for t in row] for row in p])
        assert (got == ref).all() if exact else not (got == ref).any(), bits


@pytest.mark.gpu
@pytest.mark.parametrize("unit", UNITS)
@pytest.mark.parametrize("path", ["large", "large_pair", "small"])
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_sums_are_exact(rows, path, unit):
    B = load_binding()
    a, w = case(unit, rows, 256, rows)
    f8 = torch.float8_e4m3fn
    out, _ = B.grouped_gemm_fp8(torch.tensor([0, rows], dtype=torch.int32).cuda(),
                                torch.tensor(a).to(f8).cuda(), torch.ones(rows, 3).cuda(),
                                torch.tensor(w[None]).to(f8).cuda(), torch.ones(1, 2, 3).cuda(),
                                out_dtype=torch.float32, path=path)
    np.testing.assert_array_equal(out.double().cpu().numpy(), a @ w.T)
