"""Refusals of the torch helpers around the BitLinears: shapes, dtypes and strides
are checked before anything is asked of a device."""
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

M, K = 4, 100


def rows(dtype=torch.float32, m=M, k=K):
    return torch.zeros((m, k), dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(Xq=rows(torch.uint8, k=112)), dict(Xq=rows(torch.float32, k=112)), dict(Xq=torch.zeros(M * 112, dtype=torch.int8)),
    dict(Xq=rows(torch.int8, k=99)), dict(Xq=rows(torch.int8, k=224)[:, ::2]), dict(beta=torch.zeros(M - 1)),
    dict(beta=torch.zeros(M + 1)), dict(beta=torch.zeros(M, dtype=torch.float64)), dict(beta=torch.zeros(2 * M)[::2]),
    dict(beta=torch.zeros((M, 1))), dict(out=rows(m=M - 1)), dict(out=rows(k=K - 1)), dict(out=rows(k=K + 1)),
    dict(out=rows(torch.float16)), dict(out=rows(k=2 * K)[:, ::2]),
    dict(dtype=torch.float16), dict(dtype=torch.int8), dict(K=113),
])
def test_dequantize_act_rejects(kw):
    a = dict(Xq=rows(torch.int8, k=112), beta=torch.zeros(M), K=K)
    a.update(kw)
    with pytest.raises(bl.BitlinearError):
        bl.dequantize_act(**a)


class Side:
    cuda_stream = 5


@pytest.fixture
def streams(monkeypatch):
    """Streams without a device: the current one is a name, and calls of the library note it."""
    state = {"now": "caller", "calls": [], "records": []}

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.old, state["now"] = state["now"], self.s

        def __exit__(self, *_):
            state["now"] = self.old

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 64
                state["calls"].append((name, state["now"], args[-1]))
                return bl.OK
            return call

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: state["now"])
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(bl, "_lib", Lib())
    monkeypatch.setattr(bl, "_stream", lambda s=None: (s or state["now"]))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["records"].append((t, s)))
    return state


def helper_calls():
    c = bl.KVCache.empty(2, 2, 16, device="cpu")
    kv, slots, i32 = torch.zeros((3, 2, 16)), torch.arange(3), lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {
        "norm_quantize": lambda s: bl.norm_quantize(rows(), torch.ones(K), residual=rows(), stream=s),
        "dequantize_act": lambda s: bl.dequantize_act(rows(torch.int8, k=112), torch.zeros(M), K, stream=s),
        "norm_backward": lambda s: bl.norm_backward(rows(), rows(), torch.ones(K), stream=s),
        "cache_write": lambda s: bl.cache_write(c, kv, kv, slots, stream=s),
        "cache_read": lambda s: bl.cache_read(c, slots, stream=s),
        "attention": lambda s: bl.attention(c, kv, i32(0, 1, 1)[:, None], i32(1, 2, 3), 3, return_lse=True, stream=s),
    }


@pytest.mark.parametrize("name", ["norm_quantize", "dequantize_act", "norm_backward", "cache_write", "cache_read", "attention"])
def test_another_stream(streams, name):
    """On another stream the whole call, its allocations included, runs with that stream as the current one, and
    what it returns is known to both streams."""
    side = Side()
    out = helper_calls()[name](side)
    assert [(n, now) for n, now, _ in streams["calls"]] == [("bitlinear_" + name, side)] and streams["now"] == "caller"
    for t in out if isinstance(out, tuple) else [out]:
        if t is not None:
            assert [s for x, s in streams["records"] if x is t] == ["caller"]
    assert [s for _, s in streams["records"]].count(side) >= 1  # (its inputs)
    streams["calls"].clear()
    streams["records"].clear()
    helper_calls()[name](None)
    assert [(n, now) for n, now, _ in streams["calls"]] == [("bitlinear_" + name, "caller")] and not streams["records"]
