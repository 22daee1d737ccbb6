"""The norm and cache helpers on another stream than the caller's, and in a graph."""
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402
from ternary_weight_linear_forward_amd import synth  # noqa: E402

from gpu_helpers import to_dev  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(M, K, seed):
    f = lambda s: to_dev(synth.activations_f32(M, K, seed + s))  # noqa: E731
    return f(0), f(1), (1.0 + 0.3 * f(2)[0]).contiguous(), f(3), f(4)


def test_outputs_on_another_stream():
    """A call on a side stream while the caller's stream still writes memory that it has freed, of the sizes of the
    call's outputs: what the call returns is not that memory."""
    M, K = 256, 3200
    x, r, w, dy, dh = inputs(M, K, 1)
    slots = torch.arange(M, device="cuda")
    cache = bl.KVCache.empty(M // 64, 25, 128)
    bl.cache_write(cache, x.view(M, 25, 128), r.view(M, 25, 128), slots)
    calls = {
        "norm": lambda s: bl.norm_quantize(x, w, residual=r, stream=s),
        "gradient": lambda s: bl.norm_backward(dy, x, w, dH=dh, stream=s),
        "read": lambda s: bl.cache_read(cache, slots, dtype=torch.float32, stream=s),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # the caller's stream is busy for some milliseconds, then writes
        for t in want:
            for _ in range(4):
                torch.empty_like(t).fill_(7)
        got = call(side)
        torch.cuda.synchronize()
        for g, t in zip(got, want):
            assert torch.equal(g, t), name


def test_graph_replay():
    """Norm, its gradient, cache write and read in one graph, replayed on other inputs in the same buffers."""
    M, K, H, D = 70, 640, 5, 128
    x, r, w, dy, dh = inputs(M, K, 11)
    slots = torch.arange(3, 3 + M, device="cuda")
    cache = bl.KVCache.empty(2, H, D)
    state = {}

    def run():
        h, q, beta = bl.norm_quantize(x, w, residual=r)
        v = bl.dequantize_act(q, beta, K)
        dx, dw = bl.norm_backward(dy, h, w, dH=dh)
        bl.cache_write(cache, v.view(M, H, D), h.view(M, H, D), slots)
        k2, v2 = bl.cache_read(cache, slots, dtype=torch.float32)
        state["out"] = [h, q, beta, v, dx, dw, k2, v2]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    held = state["out"]
    for turn in range(4):
        for t, n in zip((x, r, w, dy, dh), inputs(M, K, 100 * turn)):
            t.copy_(n)
        slots.copy_(torch.randperm(128, generator=torch.Generator().manual_seed(turn))[:M])
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, state["out"]):
            assert torch.equal(a, b), turn
