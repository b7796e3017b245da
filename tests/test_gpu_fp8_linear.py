"""The block-scaled FP8 quantiser, its products and the linear layer on the
GPU against the float64 forms of fp8_reference.

Codes and scales are exact (the scale is a power of two).  A product's bound:
fp32 accumulation in any order of K terms, each addition off by at most
2^-23 of its operands (a truncating adder; 2^-24 when it rounds), so K 2^-23
times the sum of the terms' magnitudes, and half a bf16 step (2^-8 of the
value) where the output is bf16.  Products of small integers are exact.
"""

import math

import pytest
import torch

import fp8_reference as R
from fp8_communication_compression_gb300 import _lib, api

pytestmark = pytest.mark.gpu


def activation(rows, cols, seed, zero_rows=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(3.0 * torch.randn((rows, 1), generator=g))
    u = torch.rand((rows, cols), generator=g)
    x = torch.where(u < 0.9, 0.02 * x, x)
    if zero_rows and rows > 2:
        x[rows // 2] = 0
    if rows > 4:
        x[1] *= 2.0 ** -125          # down to bf16's subnormals: the exponent's lower end
        x[3] = torch.sign(x[3]) * 3.0e38
    return x.bfloat16().cuda()


def check_codes(codes, scale, x, tiles):
    rows, cols = x.shape
    q, E = R.quantise(x.cpu().double(), tiles)
    assert codes.shape == (rows, api.fp8_pitch(cols))
    assert torch.equal(R.code_values(codes)[:, :cols], q)
    assert not codes[:, cols:].any()
    plain = scale if tiles else api.fp8_scales(scale, rows, cols)
    assert torch.equal(plain.cpu().long() - 127, E)


SHAPES = [(1, 1), (1, 4096), (2, 17), (8, 128), (127, 129), (128, 128), (130, 250), (257, 1000), (300, 392), (5, 8200)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_is_exact_in_both_directions(rows, cols):
    x = activation(rows, cols, 1)
    c, s = api.fp8_quantize(x)
    check_codes(c, s, x, False)
    ct, st = api.fp8_quantize(x, rowwise=False, colwise=True)
    check_codes(ct, st, x.t().contiguous(), False)
    both = api.fp8_quantize(x, colwise=True)
    assert torch.equal(both[0], c) and torch.equal(both[2], ct)
    check_codes(both[0], both[1], x, False)
    check_codes(both[2], both[3], x.t().contiguous(), False)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_weight_is_exact(rows, cols):
    w = activation(rows, cols, 2, zero_rows=False)
    if rows > 128:
        w[:128, :128] = 0                # a tile of zeros
    c, s, ct, st = api.fp8_quantize_weight(w)
    check_codes(c, s, w, True)
    assert torch.equal(ct[:, :rows], c[:, :cols].t()) and not ct[:, rows:].any()
    assert torch.equal(st, s.t())


def test_quantize_marks_blocks_with_inf_or_nan():
    x = activation(6, 300, 3)
    x[0, 5], x[2, 140], x[4, 299] = math.nan, math.inf, -math.inf
    c, s = api.fp8_quantize(x)
    plain = api.fp8_scales(s, 6, 300)
    bad = {(0, 0), (2, 1), (4, 2)}
    for r in range(6):
        for b in range(3):
            nan_codes = torch.isnan(R.code_values(c[r, 128 * b:min(128 * b + 128, 300)]))
            if (r, b) in bad:
                assert plain[b, r] == 255 and nan_codes.all()
            else:
                assert plain[b, r] != 255 and not nan_codes.any()
    w = api.fp8_quantize_weight(activation(64, 300, 4, zero_rows=False)[4:].contiguous() * 1e-3)
    y = api.fp8_linear(x[4:5], w[0], w[1])
    assert torch.isnan(y).all()
    y = api.fp8_gemm(c, s, w[0], w[1])
    for r in (0, 2, 4):
        assert torch.isnan(y[r]).all()
    assert not torch.isnan(y[5]).any()


def integer_operand(rows, K, seed):
    """Codes of whole numbers of magnitude 0 .. 4 and scale bytes 126 .. 128."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-4, 5, (rows, K), generator=g).float()
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    plain = torch.randint(126, 129, (-(-K // 128), rows), generator=g).to(torch.uint8)
    return codes.cuda(), laid_out(plain, rows, K).cuda()


def laid_out(plain, rows, K):
    """Scale bytes [blocks, rows] in the stored layout; 0xFF (NaN) in the
    places that belong to no row or block."""
    G = -(-K // 512)
    out = torch.full((-(-rows // 128) * G * 512,), 255, dtype=torch.uint8)
    r, b = torch.arange(rows)[None], torch.arange(plain.shape[0])[:, None]
    at = ((r // 128 * G + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4)
    out[at.reshape(-1)] = plain.reshape(-1)
    return out.view(-(-rows // 128), G, 512)


def row_values(codes, scale):
    rows, K = codes.shape
    return R.values(codes, api.fp8_scales(scale, rows, K))


# (M, N, K): single tokens, sizes that fill no tile, split contractions,
# several tiles of every kind, and many tiles (the persistent kernel), with
# output rows that are and are not a multiple of 16 bytes
PRODUCTS = [(1, 1, 16), (1, 128, 128), (1, 200, 4096), (3, 5, 48), (16, 200, 272), (17, 130, 128), (37, 640, 2560),
            (64, 300, 1024), (127, 129, 144), (128, 256, 128), (129, 257, 1040), (200, 1000, 640), (1, 4096, 16),
            (5, 3000, 400), (1300, 2304, 256), (1301, 2305, 272), (2000, 2100, 1040), (100, 20000, 144),
            (4100, 700, 16), (2600, 2900, 144), (20, 260, 1680), (300, 300, 6160), (129, 130, 6544)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_of_whole_numbers_is_exact(M, N, K, dtype):
    # every product and partial sum is a multiple of 2^-2 below 2^18
    a, sa = integer_operand(M, K, 5)
    b, sb = integer_operand(N, K, 6)
    ref = row_values(a, sa) @ row_values(b, sb).t()
    out = torch.full((M, N), math.nan, dtype=dtype, device="cuda")
    api.fp8_gemm(a, sa, b, sb, out=out)
    assert torch.equal(out.cpu().double(), ref.to(dtype).double())


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_gemm_with_a_tiled_weight(M, N, K):
    a, sa = integer_operand(M, K, 7)
    b, _ = integer_operand(N, K, 8)
    sb = torch.randint(126, 129, (-(-K // 128), -(-N // 128)), generator=torch.Generator().manual_seed(9))
    sb = sb.to(torch.uint8).cuda()
    ref = row_values(a, sa) @ R.values(b, sb, tiles=True).t()
    assert torch.equal(api.fp8_gemm(a, sa, b, sb, torch.float32).cpu().double(), ref)


def product_bound(A, B, dtype):
    """(reference, bound) of A @ B.T."""
    ref = A @ B.t()
    tol = A.shape[1] * 2.0 ** -23 * (A.abs() @ B.abs().t())
    return ref, tol + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (130, 250), (301, 1040), (6000, 144), (40, 16384), (24, 16400)])
def test_few_tokens_of_whole_numbers_are_exact(M, N, K):
    # x whole numbers up to 4 with a 448 in every block (scale 1), weights
    # whole numbers with any tile scale: sums are whole multiples below 2^24
    g = torch.Generator().manual_seed(17)
    x = torch.randint(-4, 5, (M, K), generator=g).double()
    x[:, ::128] = 448.0
    codes, _ = integer_operand(N, api.fp8_pitch(K), 18)
    codes[:, K:] = 0
    scale = torch.randint(126, 129, (-(-K // 128), -(-N // 128)), generator=g).to(torch.uint8).cuda()
    ref = x @ R.values(codes, scale, tiles=True)[:, :K].t()
    for dtype in (torch.float32, torch.bfloat16):
        y = api.fp8_linear(x.bfloat16().cuda(), codes, scale, dtype)
        assert torch.equal(y.cpu().double(), ref.to(dtype).double())


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (7, 256, 2560), (130, 513, 777), (1200, 2400, 320)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_and_its_gradients(M, N, K, dtype):
    g = torch.Generator().manual_seed(10)
    x = torch.randn((M, K), generator=g).bfloat16().cuda()
    w = (0.05 * torch.randn((N, K), generator=g)).bfloat16().cuda()
    dy = (0.01 * torch.randn((M, N), generator=g)).bfloat16().cuda()
    c, s, ct, st = api.fp8_quantize_weight(w)
    W = R.values(c, s, tiles=True)[:, :K]
    deq = lambda t: R.dequantised(t.cpu().double())
    y = api.fp8_linear(x, c, s, dtype)
    assert y.dtype == dtype and y.shape == (M, N)
    ref, tol = product_bound(deq(x), W, dtype)
    assert ((y.cpu().double() - ref).abs() <= tol).all()
    # the same result as the two calls it stands for
    xc, xs = api.fp8_quantize(x)
    two = api.fp8_gemm(xc, xs, c, s, dtype)
    assert ((two.cpu().double() - ref).abs() <= tol).all()

    dx, dw = api.fp8_linear_backward(dy, x, ct, st, dw_dtype=dtype)
    ref, tol = product_bound(deq(dy), W.t().contiguous(), torch.bfloat16)
    assert dx.dtype == torch.bfloat16 and ((dx.cpu().double() - ref).abs() <= tol).all()
    ref, tol = product_bound(deq(dy.t()), deq(x.t()), dtype)
    assert dw.dtype == dtype and ((dw.cpu().double() - ref).abs() <= tol).all()
    # one gradient alone: the same bits
    only_x, none = api.fp8_linear_backward(dy, x, ct, st, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = api.fp8_linear_backward(dy, x, ct, st, dw_dtype=dtype, need_dx=False)
    assert none is None and torch.equal(only_w, dw)


def test_linear_gradients_against_differences():
    # the layer is bilinear in the quantised operands: along any direction
    # that keeps the codes, central differences of sum(dy y) are exact.  Whole
    # numbers up to 8 with scale 1 in every block (a 448 beside them) do.
    M, N, K = 130, 140, 256
    g = torch.Generator().manual_seed(11)
    x, w, dy = (torch.randint(-4, 5, sh, generator=g).double() for sh in ((M, K), (N, K), (M, N)))
    for t in (x, w, dy):
        t[::128, :] = 448.0
        t[:, ::128] = 448.0
    v = torch.randint(-4, 5, (M, K), generator=g).double()
    u = torch.randint(-4, 5, (N, K), generator=g).double()
    for t in (v, u):
        t[::128, :] = 0
        t[:, ::128] = 0
    dev = lambda t: t.bfloat16().cuda()
    wq = api.fp8_quantize_weight(dev(w))
    dx, dw = api.fp8_linear_backward(dev(dy), dev(x), wq[2], wq[3])

    def loss(xx, ww):
        q = api.fp8_quantize_weight(dev(ww))
        return (dy * api.fp8_linear(dev(xx), q[0], q[1], torch.float32).cpu().double()).sum()

    # sums below 2^24 units are exact in fp32; dx is rounded to bf16
    along_w = (loss(x, w + u) - loss(x, w - u)) / 2
    assert along_w == (dw.cpu().double() * u).sum()
    along_x = (loss(x + v, w) - loss(x - v, w)) / 2
    assert abs(along_x - (dx.cpu().double() * v).sum()) <= 2.0 ** -8 * (dx.cpu().double() * v).abs().sum()


def test_empty_sizes():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    w = api.fp8_quantize_weight(activation(40, 96, 12))
    assert api.fp8_linear(e(0, 96), w[0], w[1]).shape == (0, 40)
    dx, dw = api.fp8_linear_backward(e(0, 40), e(0, 96), w[2], w[3])
    assert dx.shape == (0, 96) and dw.shape == (40, 96) and not dw.any()
    c, s = api.fp8_quantize(e(3, 0))
    assert c.shape == (3, 0) and s.shape == (1, 0, 512)
    w0 = torch.empty((40, 0), dtype=torch.uint8, device="cuda")
    s0 = torch.empty((0, 1), dtype=torch.uint8, device="cuda")
    y = api.fp8_linear(e(3, 0), w0, s0)
    assert y.shape == (3, 40) and not y.any()


def test_refusals():
    x = activation(8, 256, 13)
    w = api.fp8_quantize_weight(activation(64, 256, 14))
    with pytest.raises(ValueError, match="contiguous"):
        api.fp8_quantize(x.t())
    with pytest.raises(TypeError):
        api.fp8_quantize(x.float())
    with pytest.raises(ValueError):
        api.fp8_quantize(x, rowwise=False)
    with pytest.raises(ValueError):
        api.fp8_linear(x[:, :128].contiguous(), w[0], w[1])       # another K
    with pytest.raises(ValueError):
        api.fp8_linear(x, w[0], w[1].t().contiguous())             # scales the wrong way round
    with pytest.raises(TypeError):
        api.fp8_linear(x, w[0], w[1], torch.float16)
    with pytest.raises(ValueError):
        api.fp8_linear_backward(x, x, w[2], w[3])
    with pytest.raises(_lib.TacoError, match="MISALIGNED"):
        flat = torch.zeros(8 * 256 + 1, dtype=torch.bfloat16, device="cuda")
        api.fp8_quantize(flat[1:].view(8, 256))
    with pytest.raises(_lib.TacoError, match="INVALID"):
        a, sa = integer_operand(8, 100, 15)
        b, sb = integer_operand(8, 100, 16)
        api.fp8_gemm(a, sa, b, sb)                                 # rows of 100 codes


def test_on_another_stream_and_in_a_graph():
    M, N, K = 70, 520, 900
    xs = [activation(M, K, 20 + i) for i in range(3)]
    dys = [activation(M, N, 30 + i) for i in range(3)]
    w = api.fp8_quantize_weight(activation(N, K, 40))
    bits = lambda t: t.view(torch.uint8)
    eager = [(api.fp8_linear(x, w[0], w[1]), *api.fp8_linear_backward(dy, x, w[2], w[3])) for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for x, dy, ref in zip(xs, dys, eager):
        got = (api.fp8_linear(x, w[0], w[1], stream=side), *api.fp8_linear_backward(dy, x, w[2], w[3], stream=side))
        side.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, ref))
    x, dy = xs[0].clone(), dys[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.fp8_linear(x, w[0], w[1])
        dx, dw = api.fp8_linear_backward(dy, x, w[2], w[3])
    for i in (1, 2, 0):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip((y, dx, dw), eager[i]))


def test_outputs_stay_inside_their_buffers():
    lib = _lib.load()
    G = 4096
    stream = torch.cuda.current_stream().cuda_stream

    def guarded(n):
        t = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
        return t, t.data_ptr() + G

    def intact(t, n):
        return (t[:G] == 0xA5).all() and (t[G + n:] == 0xA5).all()

    for rows, cols in ((1, 17), (129, 257), (300, 200)):
        x = activation(rows, cols, 50)
        P, Pt, cb, rb = api.fp8_pitch(cols), api.fp8_pitch(rows), -(-cols // 128), -(-rows // 128)
        for fn, sizes in ((lib.fp8_quantize, (rows * P, lib.fp8_scale_bytes(rows, cols), cols * Pt,
                                              lib.fp8_scale_bytes(cols, rows))),
                          (lib.fp8_quantize_weight, (rows * P, cb * rb, cols * Pt, cb * rb))):
            bufs = [guarded(n) for n in sizes]
            assert fn(x.data_ptr(), rows, cols, *[p for _, p in bufs], stream) == 0
            torch.cuda.synchronize()
            for (t, _), n in zip(bufs, sizes):
                assert intact(t, n)
    for M, N, K in ((1, 130, 144), (37, 257, 1040), (130, 129, 272), (1301, 2305, 144), (1300, 2304, 144)):
        a, sa = integer_operand(M, K, 51)
        b, sb = integer_operand(N, K, 52)
        for bf in (0, 1):
            n = M * N * (2 if bf else 4)
            t, p = guarded(n)
            assert lib.fp8_gemm(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), 0, M, N, K, p, bf, stream) == 0
            torch.cuda.synchronize()
            assert intact(t, n)
    assert api.taco_device_error(clear=True) == 0


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 3), (9, 7), (7, 15), (130, 129), (257, 1001), (128, 255), (256, 130),
                                       (300, 1300)])
def test_rows_inside_granules_between_guards(rows, cols):
    # a matrix between guards of NaN: a value read from outside would show in
    # a block's scale
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g).bfloat16().cuda()
    b = torch.full((x.numel() + 2048,), float("nan"), dtype=torch.bfloat16, device="cuda")
    b[1024:1024 + x.numel()] = x.flatten()
    inner = b[1024:1024 + x.numel()].view(rows, cols)
    codes, scale, codes_t, scale_t = api.fp8_quantize(inner, colwise=True)
    check_codes(codes, scale, x, False)
    check_codes(codes_t, scale_t, x.t().contiguous(), False)
    w = api.fp8_quantize_weight(inner)
    check_codes(w[0], w[1], x, True)
