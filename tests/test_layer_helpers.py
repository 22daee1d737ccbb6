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
