"""The norms around a block on the GPU against the float64 forms.

Bounds: fp32 arithmetic with sums of d (or, for the gains' gradients, T)
terms in any order, (d + 64) 2^-23 or (T + d + 64) 2^-23 of the sum of the
terms' magnitudes, and half a bf16 step (2^-8 of the value) where the output
is bf16.  A quantised n is judged by the codes' meaning: its scale is that of
an n within the bound, and its values are off by half an E4M3 step more
(2^-4 of the value, or half of the smallest step, 2^-10, times the scale).
"""

import math

import pytest
import torch

import fp8_reference as R
from fp8_communication_compression_gb300 import _lib, api

pytestmark = pytest.mark.gpu

EPS = 1e-6


def make(T, d, mode, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    y = (r(T, d) * torch.exp(2 * r(T, 1))).bfloat16().cuda()
    h = (2 * r(T, d)).bfloat16().cuda()
    gp, gq = (1 + 0.2 * r(d)).cuda(), (1 + 0.2 * r(d)).cuda()
    gate = {"none": None, "channel": r(d).cuda(), "token": r(T, 1).cuda(), "full": r(T, d).bfloat16().cuda()}[mode]
    return y, h, gp, gq, gate


def half_step(ref):
    return 2.0 ** -8 * ref.abs() + 2.0 ** -134  # (bf16's subnormals)


SIZES = [(1, 1), (1, 4096), (3, 7), (5, 128), (17, 136), (9, 1000), (700, 257), (33, 2561), (400, 2560), (40, 5120),
         (6, 8200), (3, 16384), (2, 16383)]
MODES = ["none", "channel", "token", "full"]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("mode", MODES)
def test_forward(T, d, mode):
    s = 0.7
    y, h, gp, gq, gate = make(T, d, mode, 1)
    if T > 2:
        y[1] = 0                       # a row of zeros: z = 0
    h2, n = api.rmsnorm_gate_residual(y, h, gp, gq, gate, s, EPS)
    ref_h, ref_n = R.norm_forward(y, h, gp, gq, gate, s, EPS)
    u = (d + 64) * 2.0 ** -23
    z = ref_h - s * h.cpu().double()
    mag = (s * h.cpu().double()).abs() + z.abs()
    assert ((h2.cpu().double() - ref_h).abs() <= half_step(ref_h) + u * mag).all()
    rn = (ref_n / torch.where(ref_h == 0, torch.ones_like(ref_h), ref_h)).abs()
    tol_n = u * (ref_n.abs() + rn * mag)
    assert ((n.cpu().double() - ref_n).abs() <= half_step(ref_n) + tol_n).all()

    h3, codes, scale = api.rmsnorm_gate_residual_fp8(y, h, gp, gq, gate, s, EPS)
    assert torch.equal(h3.view(torch.int16), h2.view(torch.int16))
    assert codes.shape == (T, api.fp8_pitch(d))
    scale = api.fp8_scales(scale, T, d)
    assert not codes[:, d:].any()
    full = R.scale_full(scale, T, d, False)
    got = R.code_values(codes)[:, :d] * full
    assert ((got - ref_n).abs() <= 2.0 ** -4 * (ref_n.abs() + tol_n) + 2.0 ** -10 * full + tol_n).all()
    top = lambda t: torch.nn.functional.pad(t, (0, R.ceil_to(d, 128) - d)).view(T, -1, 128).abs().amax(2)
    lo = R.block_exponent((top(ref_n) - top(tol_n)).clamp(min=0))
    hi = R.block_exponent(top(ref_n) + top(tol_n))
    E = scale.cpu().long().t() - 127
    assert ((E >= torch.minimum(lo, hi)) & (E <= hi)).all()


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("mode", MODES)
def test_backward(T, d, mode):
    s = 0.7
    y, h, gp, gq, gate = make(T, d, mode, 2)
    if T > 2:
        y[1] = 0
    h2, _ = api.rmsnorm_gate_residual(y, h, gp, gq, gate, s, EPS)
    g = torch.Generator().manual_seed(3)
    dn, dh2 = ((0.1 * torch.randn((T, d), generator=g)).bfloat16().cuda() for _ in range(2))
    got = api.rmsnorm_gate_residual_backward(dn, dh2, y, h2, gp, gq, gate, s, EPS)
    ref = R.norm_backward(dn, dh2, y, h2, gp, gq, gate, s, EPS)
    mag = R.norm_backward(dn, dh2, y, h2, gp, gq, gate, s, EPS, magnitude=True)
    # statistics (d terms), G, its dot product (d terms), a sum over tokens
    u_row, u_sum = 4 * (d + 64) * 2.0 ** -23, (4 * (d + 64) + T) * 2.0 ** -23
    names = ("dy", "dh", "dg_post", "dg_pre", "dgate")
    for name, a, b, m in zip(names, got, ref, mag):
        if b is None:
            assert a is None
            continue
        tol = (u_sum if name in ("dg_post", "dg_pre") or mode == "channel" else u_row) * m
        if a.dtype == torch.bfloat16:
            tol = tol + half_step(b)
        assert a.shape == b.shape
        assert ((a.cpu().double() - b).abs() <= tol).all(), name
    again = api.rmsnorm_gate_residual_backward(dn, dh2, y, h2, gp, gq, gate, s, EPS)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


def test_no_tokens():
    y, h, gp, gq, gate = make(0, 256, "channel", 4)
    h2, n = api.rmsnorm_gate_residual(y, h, gp, gq, gate)
    assert h2.shape == n.shape == (0, 256)
    dy, dh, dgp, dgq, dgate = api.rmsnorm_gate_residual_backward(y, y, y, h, gp, gq, gate)
    assert dy.shape == dh.shape == (0, 256)
    for t in (dgp, dgq, dgate):
        assert t.shape == (256,) and not t.any()


def test_a_nan_stays_in_its_row():
    y, h, gp, gq, gate = make(6, 512, "channel", 5)
    y[2, 7] = math.nan
    h[4, 100] = math.inf
    h2, n = api.rmsnorm_gate_residual(y, h, gp, gq, gate)
    _, codes, scale = api.rmsnorm_gate_residual_fp8(y, h, gp, gq, gate)
    scale = api.fp8_scales(scale, 6, 512)
    for r in range(6):
        assert torch.isfinite(n[r]).all() == (r not in (2, 4))
        assert (scale[:, r] != 255).all() == (r not in (2, 4))


def test_refusals():
    y, h, gp, gq, _ = make(4, 64, "none", 6)
    with pytest.raises(ValueError, match="contiguous"):
        api.rmsnorm_gate_residual(y.t(), h.t(), gp, gq)
    with pytest.raises(ValueError):
        api.rmsnorm_gate_residual(y, h[:2], gp, gq)
    with pytest.raises(ValueError):
        api.rmsnorm_gate_residual(y, h, gp[:32], gq)
    with pytest.raises(TypeError):
        api.rmsnorm_gate_residual(y, h, gp.bfloat16(), gq)
    with pytest.raises(ValueError, match="gate"):
        api.rmsnorm_gate_residual(y, h, gp, gq, torch.ones(4, 2, device="cuda"))
    with pytest.raises(_lib.TacoError, match="INVALID"):
        api.rmsnorm_gate_residual(y, h, gp, gq, eps=0.0)
    big = torch.zeros((1, 16400), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(16400, device="cuda")
    with pytest.raises(_lib.TacoError, match="UNSUPPORTED"):
        api.rmsnorm_gate_residual(big, big, one, one)
    with pytest.raises(ValueError):
        api.rmsnorm_gate_residual_backward(y, y[:2], y, h, gp, gq)


def test_on_another_stream_and_in_a_graph():
    T, d = 50, 640
    sets = [make(T, d, "full", 10 + i) for i in range(2)]
    ref = [api.rmsnorm_gate_residual_backward(a[0], a[1], a[0], a[1], *a[2:]) for a in sets]
    fwd = [api.rmsnorm_gate_residual(*a) for a in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for a, r in zip(sets, ref):
        got = api.rmsnorm_gate_residual_backward(a[0], a[1], a[0], a[1], *a[2:], stream=side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, r))
    live = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = api.rmsnorm_gate_residual(*live)
        b = api.rmsnorm_gate_residual_backward(live[0], live[1], live[0], live[1], *live[2:])
    for i in (1, 0):
        for t, v in zip(live, sets[i]):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*f, *b), (*fwd[i], *ref[i])))


def test_outputs_stay_inside_their_buffers():
    lib = _lib.load()
    G = 4096
    stream = torch.cuda.current_stream().cuda_stream

    def guarded(n):
        t = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
        return t, t.data_ptr() + G, n

    for T, d in ((3, 7), (5, 136), (7, 257), (300, 264)):
        y, h, gp, gq, gate = make(T, d, "full", 20)
        for fp8 in (False, True):
            outs = [guarded(2 * T * d), guarded(T * api.fp8_pitch(d) if fp8 else 2 * T * d),
                    guarded(lib.fp8_scale_bytes(T, d))]
            assert lib.rmsnorm_gate_residual(y.data_ptr(), h.data_ptr(), gp.data_ptr(), gq.data_ptr(),
                                             gate.data_ptr(), 3, 1.0, EPS, T, d, outs[0][1], outs[1][1],
                                             outs[2][1] if fp8 else None, stream) == 0
            torch.cuda.synchronize()
            for t, _, n in outs:
                assert (t[:G] == 0xA5).all() and (t[G + n:] == 0xA5).all()
        ws = api._norm_workspace_bytes(T, d, 3, 0)
        outs = [guarded(n) for n in (2 * T * d, 2 * T * d, 4 * d, 4 * d, 2 * T * d, ws)]
        dy, dh, dgp, dgq, dg, w = (p for _, p, _ in outs)
        assert lib.rmsnorm_gate_residual_backward(y.data_ptr(), h.data_ptr(), y.data_ptr(), h.data_ptr(),
                                                  gp.data_ptr(), gq.data_ptr(), gate.data_ptr(), 3, 1.0, EPS, T, d,
                                                  dy, dh, dgp, dgq, dg, w, ws, stream) == 0
        torch.cuda.synchronize()
        for t, _, n in outs:
            assert (t[:G] == 0xA5).all() and (t[G + n:] == 0xA5).all()
    assert api.taco_device_error(clear=True) == 0


@pytest.mark.parametrize("mode,d", [("channel", 7200), ("none", 14400), ("full", 4608), ("full", 5760), ("full", 7680),
                                    ("token", 3600), ("full", 11520)])
def test_rows_that_fill_shared_memory(mode, d):
    # widths whose ring slots divide the room without a rest
    test_forward(3, d, mode)
    test_backward(3, d, mode)


# rows that start at every place of a 16-byte granule: more rows than CTAs,
# every shift, both ends of a granule, widths that change the units a thread
SHIFTED = [(1300, 1), (1301, 3), (1303, 9), (1300, 15), (2000, 66), (650, 250), (500, 1283), (340, 4090), (340, 4095),
           (200, 5119), (170, 6137), (160, 8186), (160, 10001)]


@pytest.mark.parametrize("T,d", SHIFTED)
@pytest.mark.parametrize("mode", ["none", "full"])
def test_rows_inside_granules(T, d, mode):
    test_forward(T, d, mode)
    test_backward(T, d, mode)


@pytest.mark.parametrize("T,d", [(3, 1), (9, 3), (700, 5), (1300, 13), (341, 1001), (161, 8189), (170, 4099)])
def test_odd_rows_stay_inside_their_buffers(T, d):
    lib = _lib.load()
    G = 4096
    stream = torch.cuda.current_stream().cuda_stream
    y, h, gp, gq, gate = make(T, d, "full", 21)
    # inputs between guards of NaN: a value read from outside would show
    def fenced(t):
        b = torch.full((t.numel() + 4096,), float("nan"), dtype=t.dtype, device="cuda")
        b[2048:2048 + t.numel()] = t.flatten()
        return b, b.data_ptr() + 2048 * t.element_size()

    ins = [fenced(t) for t in (y, h, gate)]
    out = torch.full((2, T * d + 4096), float("nan"), dtype=torch.bfloat16, device="cuda")
    at = [out.data_ptr() + 2 * (k * out.shape[1] + 2048) for k in range(2)]
    at = [a + (-a) % 16 for a in at]
    assert lib.rmsnorm_gate_residual(ins[0][1], ins[1][1], gp.data_ptr(), gq.data_ptr(), ins[2][1], 3, 1.0, EPS, T, d,
                                     at[0], at[1], None, stream) == 0
    torch.cuda.synchronize()
    want = api.rmsnorm_gate_residual(y, h, gp, gq, gate, 1.0, EPS)
    for k in range(2):
        first = (at[k] - out.data_ptr()) // 2 - k * out.shape[1]
        assert torch.equal(out[k, first:first + T * d].view(T, d), want[k])
        assert out[k, :first].isnan().all() and out[k, first + T * d:].isnan().all()
        assert not want[k].isnan().any()


@pytest.mark.parametrize("T,d,mode", [(4000, 2304, "channel"), (4000, 2304, "token"), (3648, 2560, "full"),
                                      (3647, 2560, "none"), (40001, 64, "token"), (20000, 264, "token"),
                                      (19713, 520, "token")])
def test_many_rows(T, d, mode):
    # one row at a time (2056 to 2560 columns); more tokens a CTA than their
    # gates are held at once
    test_forward(T, d, mode)
    test_backward(T, d, mode)


@pytest.mark.parametrize("T,d", [(700, 1792), (650, 2048), (320, 2816), (300, 3200), (310, 4096)])
@pytest.mark.parametrize("mode", MODES)
def test_forward_with_several_ctas_an_sm(T, d, mode):
    test_forward(T, d, mode)


@pytest.mark.parametrize("T,d", [(900, 1288), (800, 1536), (700, 2304), (500, 3584), (400, 3592), (700, 1537),
                                 (400, 2945), (350, 3081)])
@pytest.mark.parametrize("mode", MODES)
def test_forward_with_one_or_two_units_a_thread(T, d, mode):
    test_forward(T, d, mode)
