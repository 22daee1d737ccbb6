"""The norm's int8 rows through the C entry: every byte of a row's stride."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_host  # noqa: E402
from test_gpu_norm import rows  # noqa: E402

pytestmark = pytest.mark.gpu


# one, two and four pieces of eight a thread, and rows too long for the registers
@pytest.mark.parametrize("M,K", [(3, 200), (3, 1), (2, 9000), (2, 20011), (2, 40000), (1030, 100), (1030, 3000), (1030, 6000)])
@pytest.mark.parametrize("extra", [0, 16, 304, 9008])
def test_padding_up_to_the_stride(M, K, extra):
    print("norm rows", M, K, extra, flush=True)
    xt, _ = rows(M, K, 1 + K, "bf16")
    ldq = (K + 15) // 16 * 16 + extra
    q = torch.full((M + 1, ldq), 77, dtype=torch.int8, device="cuda")
    beta = torch.full((M + 1,), -7.0, device="cuda")
    st = bl.bitlinear_norm_quantize(xt.data_ptr(), bl.BF16, M, K, K, None, 0, None, 1e-5, None, bl.F32, 0, q.data_ptr(),
                                    bl.I8, ldq, bl.LAYOUT_I2, beta.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bl.OK
    _, want, wb = bl.norm_quantize(xt, keep_h=False)
    torch.cuda.synchronize()
    got = to_host(q)
    assert np.array_equal(got[:M, :K], to_host(want)[:, :K]) and np.array_equal(to_host(beta)[:M], to_host(wb))
    assert not got[:M, K:].any()
    assert (got[M] == 77).all() and float(beta[M]) == -7.0
