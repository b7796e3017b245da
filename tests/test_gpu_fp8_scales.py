"""fp8_linear for few tokens at the ends of the scales' range.  A block's sum c
times two factors 2^ex and 2^ew stands for a number that fp32 may hold where
2^(ex + ew) does not: every expected value here is exact."""

import math

import pytest
import torch

from fp8_communication_compression_gb300 import api

pytestmark = pytest.mark.gpu

N = 130


def code(v):
    return torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).item()


def linear(M, xs, ws, ex, ew, dtype):
    """y of tokens whose first block is 2^ex times xs (E4M3 values, one of them
    448) and a weight whose first blocks are ws, scale 2^ew; the second block
    is 448 at a place where the weight is 3, scales 1: adds 1344."""
    x = torch.zeros((M, 256), dtype=torch.float64)
    x[:, :len(xs)] = torch.tensor(xs, dtype=torch.float64) * 2.0 ** ex
    x[:, 128] = 448.0
    codes = torch.zeros((N, 256), dtype=torch.uint8)
    codes[:, :len(ws)] = torch.tensor([code(w) for w in ws], dtype=torch.uint8)
    codes[:, 128] = code(3.0)
    scale = torch.full((2, 2), 127, dtype=torch.uint8)
    scale[0] = 127 + ew if ew is not None else 255
    xb = x.bfloat16()
    assert torch.equal(xb.double(), x)
    return api.fp8_linear(xb.cuda(), codes.cuda(), scale.cuda(), dtype).cpu().double()


def expected(v, M, dtype):
    return torch.full((M, N), v, dtype=torch.float64).to(torch.float32).to(dtype).double()


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_factors_beyond_the_range_of_their_product(M, dtype):
    one = lambda v: expected(v, M, dtype)
    # a sum of zero at 2^(ex + ew) beyond fp32
    assert torch.equal(linear(M, [448.0, -448.0], [2.0, 2.0], 118, 120, dtype), one(1344.0))
    assert torch.equal(linear(M, [448.0, 0.0], [0.0, 5.0], 60, 120, dtype), one(1344.0))
    # a small sum at 2^130: 2^-9 2^-9 2^130 = 2^112
    assert torch.equal(linear(M, [448.0, 2.0 ** -9], [0.0, 2.0 ** -9], 65, 65, dtype), one(2.0 ** 112))
    # a sum of 448 * 128 * 2 at 2^100 2^-100 and the other way round
    for e in (100, -100):
        assert torch.equal(linear(M, [448.0, 448.0], [128.0, 128.0], e, -e, dtype), one(448.0 * 256 + 1344.0))
    # beyond fp32 for good
    assert (linear(M, [448.0], [2.0], 118, 100, dtype) == math.inf).all()
    # a NaN scale
    assert torch.isnan(linear(M, [448.0], [2.0], 0, None, dtype)).all()


@pytest.mark.parametrize("M", [1, 8])
def test_factors_whose_product_is_below_every_number(M):
    # 448 * 416 * 16 * 2^-155 is about 2^-133.5, a subnormal of fp32; nothing is added to it
    x = torch.zeros((M, 128), dtype=torch.float64)
    x[:, :16] = 448.0 * 2.0 ** -75
    codes = torch.full((N, 128), code(416.0), dtype=torch.uint8)
    scale = torch.full((1, 2), 127 - 80, dtype=torch.uint8)
    y = api.fp8_linear(x.bfloat16().cuda(), codes.cuda(), scale.cuda(), torch.float32).cpu()
    want = torch.tensor(448.0 * 416 * 16 * 2.0 ** -155, dtype=torch.float64).to(torch.float32)
    assert want > 0 and (y == want).all()
