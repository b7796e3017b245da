"""What a call with ``stream=`` allocates: memory of that stream's pool (so that
it never shares a block with work still queued on the current stream), its
outputs kept from reuse while the current stream reads them.

The rule is checked on the CPU for every call, with a fake library and fake
streams that note where each allocation is made.  On the GPU a block that the
current stream has freed but still has to read must survive."""

import contextlib

import pytest
import torch

from fp8_communication_compression_gb300 import _lib, api

SIDE, CURRENT = object(), object()


class Noted(torch.Tensor):
    """A CPU tensor that passes for a CUDA tensor and notes its stream."""

    is_cuda = True
    made_on = CURRENT

    def record_stream(self, stream):
        self.recorded = stream


class FakeLibrary:
    def __getattr__(self, name):
        return lambda *args: 0


class Side:
    cuda_stream = 1


@pytest.fixture()
def notes(monkeypatch):
    state = {"on": CURRENT, "made": []}
    real_empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        before, state["on"] = state["on"], stream
        yield
        state["on"] = before

    def empty(*args, **kw):
        t = real_empty(*args, **kw).as_subclass(Noted)
        t.made_on = state["on"]
        state["made"].append(t)
        return t

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: CURRENT)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda x: empty(x.shape, dtype=x.dtype))
    monkeypatch.setattr(_lib, "load", FakeLibrary)
    monkeypatch.setattr(api, "_linear_workspace_bytes", lambda *a: 512)
    monkeypatch.setattr(api, "_norm_workspace_bytes", lambda *a: 512)
    return state


def t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Noted)


U8, F32 = torch.uint8, torch.float32
x, g, c, a = lambda: t((4, 256)), lambda: t(256, F32), lambda: t((4, 256), U8), lambda: t(8, F32)
w = lambda: (t((128, 256), U8), t((2, 1), U8), t((256, 128), U8), t((1, 2), U8))
CALLS = {
    "taco_compress": lambda s: api.taco_compress(x(), stream=s),
    "taco_decompress": lambda s: api.taco_decompress(c(), a(), a(), stream=s),
    "taco_compress_int8": lambda s: api.taco_compress_int8(x(), stream=s),
    "taco_decompress_int8": lambda s: api.taco_decompress_int8(t((4, 256), torch.int8), a(), a(), stream=s),
    "taco_reduce_shards": lambda s: api.taco_reduce_shards([c()] * 2, [a()] * 2, [a()] * 2, stream=s),
    "taco_reduce_decompress": lambda s: api.taco_reduce_decompress([c()] * 2, [a()] * 2, [a()] * 2, stream=s),
    "agoq_reduce_shards": lambda s: api.agoq_reduce_shards([c()] * 2, [a()] * 2, stream=s),
    "agoq_laaq_quantize": lambda s: api.agoq_laaq_quantize(x(), stream=s),
    "agoq_laaq_dequantize": lambda s: api.agoq_laaq_dequantize(t(512, U8), a(), 1024, stream=s),
    "agoq_laaq_dequantize_silu": lambda s: api.agoq_laaq_dequantize_silu(t(512, U8), a(), 1024, stream=s),
    "agoq_laaq_dequantize_rmsnorm": lambda s: api.agoq_laaq_dequantize_rmsnorm(t(512, U8), a(), 4, 256, g(), stream=s),
    "taco_e4m3_encode": lambda s: api.taco_e4m3_encode(g(), stream=s),
    "taco_gemm_compress": lambda s: api.taco_gemm_compress(x(), t((128, 256)), stream=s, split_tail=False),
    "agoq_gemm_laaq_quantize": lambda s: api.agoq_gemm_laaq_quantize(x(), t((128, 256)), stream=s, split_tail=False),
    "fp8_quantize": lambda s: api.fp8_quantize(x(), colwise=True, stream=s),
    "fp8_quantize_weight": lambda s: api.fp8_quantize_weight(x(), stream=s),
    "fp8_gemm": lambda s: api.fp8_gemm(c(), t((1, 1, 512), U8), w()[0], w()[1], stream=s),
    "fp8_linear": lambda s: api.fp8_linear(x(), *w()[:2], stream=s),
    "fp8_linear_backward": lambda s: api.fp8_linear_backward(t((4, 128)), x(), *w()[2:], stream=s),
    "rmsnorm_gate_residual": lambda s: api.rmsnorm_gate_residual(x(), x(), g(), g(), stream=s),
    "rmsnorm_gate_residual_fp8": lambda s: api.rmsnorm_gate_residual_fp8(x(), x(), g(), g(), stream=s),
    "rmsnorm_gate_residual_backward":
        lambda s: api.rmsnorm_gate_residual_backward(x(), x(), x(), x(), g(), g(), g(), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_stream_allocates_there(notes, name):
    side = Side()
    out = CALLS[name](side)
    outs = [o for o in (out if isinstance(out, tuple) else (out,)) if o is not None]
    assert notes["made"]
    for m in notes["made"]:
        assert m.made_on is side
    for o in outs:
        assert o.made_on is side and o.recorded is CURRENT


@pytest.mark.gpu
def test_memory_the_current_stream_still_reads_survives():
    M, N, K = 2048, 4096, 512
    side = torch.cuda.Stream()
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(N, device="cuda")
    wq = api.fp8_quantize_weight(torch.ones((N, K), dtype=torch.bfloat16, device="cuda"))
    wide = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for call in (lambda: (api.fp8_linear(x, wq[0], wq[1], stream=side),),
                 lambda: api.rmsnorm_gate_residual(wide, wide, gain, gain, stream=side)):
        for _ in range(3):
            old = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
            torch.cuda._sleep(20_000_000)  # the current stream is busy for some milliseconds
            kept = old.clone()
            del old                        # freed, but the clone has not read it yet
            got = call()
            side.synchronize()
            first = [o.clone() for o in got]
            torch.cuda.synchronize()
            assert bool((kept == 7.0).all())
            assert all(torch.equal(p, q) and bool(torch.isfinite(p).all()) for p, q in zip(got, first))


@pytest.mark.gpu
def test_calls_on_a_branch_of_a_captured_graph():
    M, N, K = 70, 512, 384
    g = torch.Generator().manual_seed(91)
    xs = [torch.randn((M, K), generator=g).bfloat16().cuda() for _ in range(2)]
    w = api.fp8_quantize_weight(torch.randn((N, K), generator=g).bfloat16().cuda())
    gain = torch.ones(K, device="cuda")
    eager = [(api.fp8_linear(x, w[0], w[1]), *api.rmsnorm_gate_residual_backward(x, x, x, x, gain, gain)[:4]) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = (api.fp8_linear(x, w[0], w[1], stream=side),
               *api.rmsnorm_gate_residual_backward(x, x, x, x, gain, gain, stream=side)[:4])
        torch.cuda.current_stream().wait_stream(side)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager[i]))
