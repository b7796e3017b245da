"""The losses over the vocabulary on the GPU against the float64 forms, whose
bounds training_reference.py derives, and against differences of the loss."""

import math

import pytest
import torch

import training_reference as R
from fp8_communication_compression_gb300 import _lib, api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, V, N, dt, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn((T, N), generator=g)
    a = torch.randint(0, V, (T,), generator=g)
    x[torch.arange(T), a] += 4.0 * torch.rand(T, generator=g)
    return x.to(dt).cuda(), a.cuda(), g


def close(got, want, name=""):
    value, tol = want
    diff = (got.cpu().double().reshape(value.shape) - value).abs()
    assert torch.isfinite(diff).all() and (diff <= tol).all(), (name, float((diff - tol).max()), float(diff.max()))


SIZES = [(1, 1, 1), (1, 7, 9), (3, 8, 8), (5, 129, 256), (2, 1000, 1000), (9, 1001, 1001), (4, 4097, 4224),
         (64, 513, 513), (700, 260, 264), (1, 50257, 50304), (3, 50257, 50257), (40, 32003, 32003), (2, 131072, 131072),
         (2, 300001, 300001)]
TYPES = [BF, F32]


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,N", SIZES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_logprob_and_its_gradient(T, V, N, dt, tau):
    x, a, g = make(T, V, N, dt, 1)
    if T > 2:
        a[1] = -1
    logp, lse = api.token_logprob(x, a, V, tau)
    want, wlse, tol, tol_lse = R.logprob(x, a, V, tau)
    close(logp, (want, tol), "logp")
    close(lse, (wlse, tol_lse), "lse")
    dlogp = torch.randn(T, generator=g)
    if T > 4:
        dlogp[3] = 0.0
    # the gradient's definition takes the lse that it is given: no error of it
    given = lse.cpu().double()
    ref = R.softmax_grad(x, a, dlogp.double(), 4 * R.U * dlogp.double().abs(), V, tau, given, 4 * R.U * torch.ones(T))
    close(api.token_logprob_backward(dlogp.cuda(), x, a, lse, V, tau), ref, "dlogits")
    y = x.clone()
    out = api.token_logprob_backward(dlogp.cuda(), y, a, lse, V, tau, dlogits=y)
    assert out.data_ptr() == y.data_ptr()
    assert torch.equal(out, api.token_logprob_backward(dlogp.cuda(), x, a, lse, V, tau))


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,N", SIZES)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy_loss(T, V, N, dt, kl):
    tau, lo, hi = 0.9, 0.2, 0.3
    x, a, g = make(T, V, N, dt, 2)
    logp = R.logprob(x, a, V, tau)[0]
    moved = 0.3 * torch.randn(T, generator=g, dtype=torch.float64)
    for border in (math.log(1 - lo), math.log(1 + hi)):  # no ratio at a border of the clipping
        moved = torch.where((moved - border).abs() < 0.02, moved + 0.05, moved)
    old, ref = (logp - moved).float().cuda(), (logp + 0.3 * torch.randn(T, generator=g)).float().cuda()
    adv = torch.randn(T, generator=g).cuda()
    w = (torch.rand(T, generator=g) / T).cuda()
    if T > 4:
        adv[0], w[2], a[3] = 0.0, 0.0, -1
    got = api.policy_loss(x, a, old, adv, w, ref if kl else None, lo, hi, kl, V, tau, grad_scale=1.5)
    want = R.policy(x, a, old, adv, w, ref, lo, hi, kl, V, tau, 1.5)
    for name, v in want.items():
        close(getattr(got, name), v, name)
    assert not got.dlogits[:, V:].any()
    again = api.policy_loss(x, a, old, adv, w, ref if kl else None, lo, hi, kl, V, tau, need_grad=False)
    assert again.dlogits is None
    assert torch.equal(again.token_loss, got.token_loss) and torch.equal(again.loss, got.loss)
    y = x.clone()
    same = api.policy_loss(y, a, old, adv, w, ref if kl else None, lo, hi, kl, V, tau, 1.5, dlogits=y)
    assert torch.equal(y, got.dlogits) and torch.equal(same.loss, got.loss)


def test_policy_loss_against_differences():
    """Central differences of the float64 loss over fp32 logits: second-order
    error h^2 / 6 of a third derivative of at most a few w r A; the kernel's
    fp32 gradient within its bound."""
    T, V, h = 6, 33, 1e-4
    x, a, g = make(T, V, V, F32, 3)
    logp = R.logprob(x, a, V, 1.0)[0]
    old = (logp - torch.tensor([0.05, -0.1, 0.4, -0.5, 0.1, 0.0])).float().cuda()
    ref = (logp + 0.2 * torch.randn(T, generator=g)).float().cuda()
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 0.5, -2.0]).cuda()
    w = torch.full((T,), 1.0 / T).cuda()
    got = api.policy_loss(x, a, old, adv, w, ref, 0.2, 0.2, 0.1).dlogits.cpu().double()
    f = lambda z: R.policy(z, a, old, adv, w, ref, 0.2, 0.2, 0.1, V, 1.0)["loss"][0]
    base = x.cpu().double()
    for t in range(T):
        for j in (0, int(a[t]), V - 1):
            up, down = base.clone(), base.clone()
            up[t, j] += h
            down[t, j] -= h
            diff = (f(up) - f(down)) / (2 * h)
            assert abs(float(diff - got[t, j])) <= 1e-6


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,tail,V,N", [((1, 1), 0, 5, 5), ((3, 0, 2, 7), 4, 1000, 1024), ((40, 33), 3, 32001, 32001),
                                           ((300, 17, 5, 260, 1, 1), 0, 515, 515), ((0, 0), 2, 64, 64)])
@pytest.mark.parametrize("ls,mean", [(0.0, False), (0.2, True)])
def test_preference_loss(lens, tail, V, N, dt, ls, mean):
    T = sum(lens) + tail
    x, a, g = make(T, V, N, dt, 4)
    if lens[0] > 2:
        a[0] = -1                                   # a prompt
        a[sum(lens[:1]):sum(lens[:2])] = -1         # a sequence without tokens
    logp = R.logprob(x, a, V, 1.0)[0]
    ref = (logp + 0.5 * torch.randn(T, generator=g)).float().cuda()
    if tail:                                        # in no sequence: must not be read
        x[-1] = math.nan
        ref[-1] = math.nan
    offsets = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)]).cuda()
    for r in (ref, None):
        clean = x.clone()
        if tail:
            clean[-1] = 0.0
        want = R.preference(clean, a, offsets, None if r is None else r.nan_to_num(), 0.3, ls, mean, V, 1.0, 2.0)
        got = api.preference_loss(x, a, offsets, r, 0.3, ls, mean, V, grad_scale=2.0)
        for name, v in want.items():
            close(getattr(got, name), v, name)
    again = api.preference_loss(x, a, offsets, None, 0.3, ls, mean, V, need_grad=False)
    assert torch.equal(again.loss, got.loss) and again.dlogits is None
    y = x.clone()
    api.preference_loss(y, a, offsets, None, 0.3, ls, mean, V, grad_scale=2.0, dlogits=y)
    assert torch.equal(y, got.dlogits)


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
def test_masked_and_infinite_values(dt):
    T, V, N = 8, 777, 800
    x, a, g = make(T, V, N, dt, 5)
    low = torch.finfo(dt).min
    x[:, V:] = math.nan                       # padding is not read as values
    keep = a.clone()
    x[0, :600], x[1, :600] = -math.inf, low   # a masked vocabulary
    a[0], a[1] = 700, 650
    x[2] = -math.inf                          # masked altogether
    x[3, 5] = math.nan
    x[4, 5] = math.inf
    x[5] = low                                # all equal: log 1 / V
    x[6] = math.nan                           # not counted
    a[6] = -1
    a[7] = 3
    x[7, 3] = -math.inf                       # the token itself is masked
    logp, lse = api.token_logprob(x, a, V)
    for t, first in ((0, 600), (1, 600)):
        want, _, tol, _ = R.logprob(x[t:t + 1, first:], a[t:t + 1] - first, V - first, 1.0)
        assert abs(float(logp[t].cpu().double() - want)) <= float(tol)
    assert logp[2].isnan() and logp[3].isnan() and logp[4].isnan()
    assert abs(float(logp[5]) + math.log(V)) <= 1e-5
    assert float(logp[6]) == 0.0 and float(lse[6]) == 0.0 and float(logp[7]) == -math.inf
    one = torch.ones(T, device="cuda")
    d = api.token_logprob_backward(one, x, a, lse, V).float()
    assert not d[0, :600].any() and not d[1, :600].any() and d[3, :V].isnan().all() and not d[6].any()
    assert not d[:, V:].any()
    one[3] = 0.0
    assert not api.token_logprob_backward(one, x, a, lse, V)[3].any()
    # a policy loss counts neither rows of weight 0 nor what else they hold
    w = torch.tensor([1.0, 1.0, 0, 0, 0, 1.0, 1.0, 0], device="cuda")
    nan = torch.where(w == 0, torch.full_like(w, math.nan), torch.zeros_like(w))
    old = torch.where(w == 0, nan, logp - 0.1)
    got = api.policy_loss(x, a, old, 1.0 + nan, w, old.clone(), kl=0.1, vocab=V)
    assert got.loss.isfinite() and got.token_loss.isfinite().all() and got.dlogits.isfinite().all()
    assert not got.dlogits[w == 0].any() and got.dlogits[0].any()
    # targets outside the vocabulary show
    bad = keep.clone()
    bad[0] = V
    x, _, _ = make(T, V, N, dt, 5)
    logp, lse = api.token_logprob(x, bad, V)
    assert logp[0].isnan() and logp[1:].isfinite().all()
    d = api.token_logprob_backward(torch.ones(T, device="cuda"), x, bad, lse, V)
    assert d[0, :V].isnan().all() and d[1:].isfinite().all()
    got = api.policy_loss(x, bad, logp.nan_to_num(), torch.ones(T).cuda(), torch.ones(T).cuda(), vocab=V)
    assert got.loss.isnan() and got.dlogits[0, :V].isnan().all() and got.dlogits[1:].isfinite().all()


def test_nothing_counts():
    x, a, g = make(5, 100, 128, BF, 6)
    z = torch.zeros(5, device="cuda")
    got = api.policy_loss(x, a, z, z, z, vocab=100)
    assert float(got.loss) == 0.0 and not got.dlogits.any() and not got.logp.any()
    got = api.preference_loss(x, torch.full_like(a, -1), torch.tensor([0, 2, 5]).cuda(), vocab=100)
    assert abs(float(got.loss) - math.log(2)) <= 1e-6 and not got.dlogits.any()
    e = x[:0]
    got = api.policy_loss(e, a[:0], z[:0], z[:0], z[:0])
    assert float(got.loss) == 0.0 and got.dlogits.shape == (0, 128)
    logp, lse = api.token_logprob(e, a[:0])
    assert logp.shape == lse.shape == (0,)


def test_offsets_outside_the_rows_are_bounded():
    x, a, g = make(6, 50, 50, F32, 7)
    got = api.preference_loss(x, a, torch.tensor([-4, 3, 99]).cuda())
    want = api.preference_loss(x, a, torch.tensor([0, 3, 6]).cuda())
    assert torch.equal(got.loss, want.loss) and torch.equal(got.dlogits, want.dlogits)


def test_rows_do_not_touch_their_neighbours():
    """Gradients of a slice of a larger buffer leave what lies around it."""
    T, N = 3, 1003
    for dt in TYPES:
        x, a, g = make(T, N, N, dt, 8)
        whole = torch.full((T * N + 64,), 7.0, dtype=dt, device="cuda")
        out = whole[32:32 + T * N].view(T, N)
        z = torch.zeros(T, device="cuda")
        api.policy_loss(x, a, z - 7.0, z + 1.0, z + 1.0, dlogits=out)
        assert (whole[:32] == 7.0).all() and (whole[32 + T * N:] == 7.0).all()
        assert torch.equal(out, api.policy_loss(x, a, z - 7.0, z + 1.0, z + 1.0).dlogits)


def test_captured_and_on_another_stream():
    T, V = 33, 5001
    x, a, g = make(T, V, V, BF, 9)
    old, adv, w = (torch.randn(T, generator=g).cuda() for _ in range(3))
    old = old - 8.0
    offsets = torch.tensor([0, 10, 20, 30, 32]).cuda()
    call = lambda s=None: (*api.policy_loss(x, a, old, adv, w, stream=s), *api.preference_loss(x, a, offsets, old, stream=s))
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # two graphs, each with its own workspace, replayed in turn and at once
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    x2 = x.clone()
    x.copy_(x2 * 0.5)
    half = [t.clone() for t in call()]
    for source, expect in ((x2, want), (x2 * 0.5, half)):
        x.copy_(source)
        torch.cuda.synchronize()
        for gr, s in zip(graphs, (side, torch.cuda.Stream())):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(p, q) for p, q in zip(got, expect))
    assert _lib.load() and api.taco_device_error() == 0


def test_offsets_beyond_32_bits():
    """Rows behind 2^32 elements: 2^31 rows are too many, a long tensor is not."""
    N, T = 131072, 32769 + 3
    x = torch.zeros((T, N), dtype=BF, device="cuda")
    last = torch.randn((4, N), generator=torch.Generator().manual_seed(10)).to(BF).cuda()
    x[-4:] = last
    a = torch.full((T,), -1, device="cuda")
    a[-4:] = torch.tensor([0, 1, 70000, N - 1])
    logp, lse = api.token_logprob(x, a)
    want, wl, tol, tol_lse = R.logprob(last, a[-4:], N, 1.0)
    close(logp[-4:], (want, tol))
    close(lse[-4:], (wl, tol_lse))
    assert not logp[:-4].any()
    d = torch.zeros(T, device="cuda")
    d[-4:] = 1.0
    # the gradient takes the lse that it is given: the same bits wherever a row is
    small = api.token_logprob_backward(d[-4:], last, a[-4:], lse[-4:].contiguous())
    api.token_logprob_backward(d, x, a, lse, dlogits=x)
    assert torch.equal(x[-4:], small) and not x[:-4].any()


@pytest.mark.parametrize("dt,V", [(BF, 1000003), (F32, 500001)], ids=["bf16", "f32"])
def test_rows_longer_than_shared_memory(dt, V):
    """A vocabulary that a cluster's shared memory does not hold."""
    T = 3
    x, a, g = make(T, V, V, dt, 11)
    logp = R.logprob(x, a, V, 1.0)[0]
    old = (logp - 0.05).float().cuda()
    adv, w = torch.tensor([1.0, -1.0, 0.5]).cuda(), torch.tensor([0.5, 0.25, 0.0]).cuda()
    want = R.policy(x, a, old, adv, w, old, 0.2, 0.2, 0.1, V, 1.0)
    got = api.policy_loss(x, a, old, adv, w, old, kl=0.1)
    for name, v in want.items():
        close(getattr(got, name), v, name)
    y = x.clone()
    api.policy_loss(y, a, old, adv, w, old, kl=0.1, dlogits=y)
    assert torch.equal(y, got.dlogits)
    one = api.policy_loss(x[:1], a[:1], old[:1], adv[:1], w[:1])       # one row: its loss is the sum
    assert torch.equal(one.loss, one.token_loss[0]) and one.dlogits.any()


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [-1e4, -1e6, -3e6, -1e7, -1e9, -1e10, -1e30, 3e6, 1e10, 1e30])
def test_rows_of_one_large_value(dt, value):
    """Masked altogether by any value: every token has 1 / V.  Two rows of them
    hold a value above or below too, whose share is all or nothing."""
    V = 3001
    x = torch.full((4, V), value, dtype=dt, device="cuda")
    x[2, 7], x[3, 7] = x[2, 7] + abs(value) / 2, x[3, 7] - abs(value) / 2
    a = torch.tensor([0, V - 1, 7, 8]).cuda()
    logp, lse = api.token_logprob(x, a)
    want = torch.tensor([-math.log(V), -math.log(V), 0.0, -math.log(V - 1)])
    # training_reference.logprob's bound: the sum's roundings, and those of ln V
    tol = (V / 256 + 64) * 2.0 ** -22 + 4 * R.U * (math.log(V) + 1)
    assert ((logp.cpu() - want).abs() <= tol).all()
    z = torch.zeros(4, device="cuda")
    got = api.policy_loss(x, a, logp, z + 1.0, z + 1.0, clip_high=1e3)
    p = torch.full((4, V), 1.0 / V, dtype=torch.float64)
    p[2], p[3] = 0.0, 1.0 / (V - 1)
    p[2, 7], p[3, 7] = 1.0, 0.0
    hot = torch.zeros(4, V, dtype=torch.float64).scatter_(1, a.cpu()[:, None], 1.0)
    ref = p - hot                                          # r = 1, A = 1
    assert ((got.dlogits.cpu().double() - ref).abs() <= R.half_step(ref, dt) + 1e-5 * (p + hot)).all()
    assert ((got.logp.cpu() - want).abs() <= tol).all()
    # the preference loss too: slopes of -beta / 2 and beta / 2 (equal margins), halved by the two pairs
    pairs = api.preference_loss(x, a, torch.arange(5).cuda(), logp, beta=0.4)
    sign = torch.tensor([-1.0, 1.0, -1.0, 1.0], dtype=torch.float64)[:, None]
    ref = sign * 0.1 * (hot - p)
    assert ((pairs.dlogits.cpu().double() - ref).abs() <= R.half_step(ref, dt) + 1e-5 * (p + hot)).all()
