"""RMS norm with the residual's addition and int8 output, its gradient, and the
values of int8 rows, against plain binary64 formulas.

With u = 2^-24: h = fl(x + r) is off by u|h|, rho by 2u, the two products of y by
2u, so y and beta are within 5u; q's argument y (127 / beta) is within 12u of
its size, at most 127: |q - y 127 / beta| <= 0.5 + 127 * 12 u < 0.5 + 1e-4."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402
from ternary_weight_linear_forward_amd import synth  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def rows(M, K, seed, dtype, ld=None, scale=1.0):
    """[M x K] rows of a buffer with row stride ld, as (device view, fp32 values)."""
    x = (synth.activations_f32(M, K, seed) * np.float32(scale)).astype(np.float32)
    buf = np.full((M, ld or K), np.nan, np.float32)
    buf[:, :K] = x
    t = to_dev(synth.to_bf16_bits(np.nan_to_num(buf)) if dtype == "bf16" else buf)[:, :K]
    return t, (synth.bf16_bits_to_f32(synth.to_bf16_bits(x)) if dtype == "bf16" else x)


def values(t):
    a = to_host(t.contiguous())
    return synth.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a


def norm64(h, w, eps):
    h = h.astype(np.float64)
    v = np.mean(h * h, axis=1, keepdims=True) + eps
    rho = np.where(v > 0, 1.0 / np.sqrt(np.where(v > 0, v, 1.0)), 0.0)
    return h * rho * (1.0 if w is None else w.astype(np.float64)), rho


def check_q(q, beta, y):
    top = np.abs(y).max(axis=1)
    assert np.all(np.abs(beta - top) <= 5 * U * top + 1e-45)
    arg = np.where(top[:, None] > 0, y * 127.0 / np.where(top > 0, top, 1.0)[:, None], 0.0)
    assert np.abs(q - arg).max() <= 0.5 + 1e-4


CASES = [  # M, K, x, h, residual, weight, extra row elements of x
    (1, 1, "f32", "f32", True, True, 0), (1, 3200, "bf16", "bf16", True, True, 0), (3, 7, "bf16", "f32", True, True, 2),
    (5, 255, "f32", "bf16", True, False, 1), (16, 3200, "f32", "bf16", True, True, 0),
    (17, 8640, "bf16", "bf16", True, True, 8), (70, 1001, "f32", "f32", False, True, 3),
    (2, 8191, "bf16", "bf16", True, True, 5), (300, 640, "bf16", "f32", True, True, 0),
    (4, 16384, "f32", "f32", True, True, 0), (2, 20011, "bf16", "bf16", True, True, 0),
    (2, 70000, "bf16", "f32", True, True, 0), (1, 131072, "f32", "f32", True, True, 0), (9, 64, "bf16", "bf16", False, False, 0),
]


@pytest.mark.parametrize("M,K,xd,hd,res,wt,pad", CASES)
def test_norm_quantize(M, K, xd, hd, res, wt, pad):
    print("norm", M, K, xd, hd, res, wt, pad, flush=True)
    xt, x = rows(M, K, 1 + K, xd, K + pad)
    rt, r = rows(M, K, 2 + K, hd, K + (pad + 1) // 2, 3.0) if res else (None, None)
    w = (1.0 + 0.3 * synth.activations_f32(1, K, 3 + K)[0]).astype(np.float32) if wt else None
    h = x + r if res else x  # one binary32 addition
    H, Xq, beta = bl.norm_quantize(xt, None if w is None else to_dev(w), eps=EPS, residual=rt)
    torch.cuda.synchronize()
    want = synth.bf16_bits_to_f32(synth.to_bf16_bits(h)) if H.dtype == torch.bfloat16 else h
    assert np.array_equal(values(H), want)
    q = to_host(Xq)
    assert not q[:, K:].any()
    exact = x.astype(np.float64) + (r.astype(np.float64) if res else 0.0)
    check_q(q[:, :K], to_host(beta), norm64(exact, w, EPS)[0])
    # the same values in the tiled activation layouts, padding zero, and the residual updated in place
    for layout in (bl.LAYOUT_I2, bl.LAYOUT_B3, bl.LAYOUT_B1):
        if K > 65536:
            continue
        alias = rt.clone() if res else None
        H2, Xt, beta2 = bl.norm_quantize(xt, None if w is None else to_dev(w), eps=EPS, residual=alias, H=alias,
                                         keep_h=res, layout=layout)
        torch.cuda.synchronize()
        assert np.array_equal(to_host(beta2), to_host(beta))
        assert H2 is alias and (alias is None or np.array_equal(values(alias), want))
        S, F = {bl.LAYOUT_I2: (256, 4), bl.LAYOUT_B3: (320, 5), bl.LAYOUT_B1: (512, 8)}[layout]
        G, n = (M + 15) // 16, (K + S - 1) // S
        full = np.zeros((16 * G, n * S), np.int8)
        full[:M, :K] = q[:, :K]
        # [tg, i, s, g, d, e] -> [tg, s, d, g, i, e]
        tiled = full.reshape(G, 16, n, 4, F, 16).transpose(0, 2, 4, 3, 1, 5).reshape(-1)
        assert np.array_equal(to_host(Xt), tiled), layout


@pytest.mark.parametrize("K", [100, 3200])
def test_norm_degenerate_rows(K):
    """Zero rows, rows of one value, subnormal rows, the largest values, and a row cancelled by its residual."""
    x = np.zeros((7, K), np.float32)
    x[1] = 2.5
    x[2] = np.float32(1e-41)
    x[3] = np.float32(3e38) * np.sign(synth.activations_f32(1, K, 5)[0])
    x[4, -1] = 1.0
    x[5] = synth.activations_f32(1, K, 6)[0]
    x[6] = synth.activations_f32(1, K, 7)[0]
    r = np.zeros_like(x)
    r[5] = -x[5]
    for eps in (0.0, EPS):
        H, Xq, beta = bl.norm_quantize(to_dev(x), None, eps=eps, residual=to_dev(r))
        torch.cuda.synchronize()
        b, q = to_host(beta), to_host(Xq)[:, :K]
        assert b[0] == 0 and not q[0].any() and b[5] == 0 and not q[5].any()
        assert np.isfinite(b).all()
        for m in (1, 2, 3, 4, 6):
            if m == 2 and eps == 0.0:
                continue  # below: rho leaves the range of binary32 and is held at its largest value
            y = norm64(x[m:m + 1], None, float(np.float32(eps)))[0]
            check_q(q[m:m + 1], b[m:m + 1], y)
        assert np.all(np.abs(q[2]) == 127)


def test_norm_feeds_the_forward():
    """Both int8 forms give the forward's exact accumulators."""
    M, N, K = 5, 96, 640
    t = synth.ternary_weights(N, K, seed=4)
    P, g = to_dev(oracle.pack(t, bl.LAYOUT_I2)), to_dev(np.array([0.02], np.float32))
    xt, _ = rows(M, K, 11, "bf16")
    _, Xq, beta = bl.norm_quantize(xt, keep_h=False)
    _, Xt, beta_t = bl.norm_quantize(xt, keep_h=False, layout=bl.LAYOUT_I2)
    a = to_host(bl.forward(P, bl.LAYOUT_I2, g, Xq, N, K, beta=beta, y_dtype=torch.int32))
    b = to_host(bl.forward(P, bl.LAYOUT_I2, g, Xt, N, K, beta=beta_t, y_dtype=torch.int32))
    want = to_host(Xq)[:, :K].astype(np.int64) @ t.T.astype(np.int64)
    assert np.array_equal(a, want) and np.array_equal(b, want)


@pytest.mark.parametrize("M,K,ldq,vd,ldv", [(1, 1, 16, "f32", 1), (3, 100, 112, "bf16", 103), (70, 3200, 3200, "bf16", 3200),
                                           (2, 8641, 8656, "f32", 8641), (300, 48, 64, "f32", 50)])
def test_dequantize(M, K, ldq, vd, ldv):
    q = synth.int8_activations(M, ldq, seed=K)
    beta = np.abs(synth.activations_f32(1, M, seed=M)[0])
    out = torch.full((M, ldv), -7.0, dtype=torch.bfloat16 if vd == "bf16" else torch.float32, device="cuda")
    bl.dequantize_act(to_dev(q), to_dev(beta), K, out=out[:, :K])
    torch.cuda.synchronize()
    want = q[:, :K].astype(np.float32) * (beta / np.float32(127))[:, None]
    if vd == "bf16":
        want = synth.bf16_bits_to_f32(synth.to_bf16_bits(want))
    got = values(out)
    assert np.array_equal(got[:, :K], want)
    assert np.all(got[:, K:] == -7.0)


def bwd64(dy, h, w, dh, eps):
    dy, h = dy.astype(np.float64), h.astype(np.float64)
    w = np.ones(h.shape[1]) if w is None else w.astype(np.float64)
    _, rho = norm64(h, None, eps)
    g = dy * w
    c = rho ** 3 * np.mean(g * h, axis=1, keepdims=True)
    dx = rho * g - c * h + (0.0 if dh is None else dh.astype(np.float64))
    # terms of the error bound of dX (see test_norm_backward) and of dW's sum
    size = np.abs(rho * g) + np.abs(c * h) + rho ** 3 * np.mean(np.abs(g * h), axis=1, keepdims=True) * np.abs(h) + \
        (0.0 if dh is None else np.abs(dh.astype(np.float64)))
    t = dy * h * rho
    return dx, size, t.sum(0), np.abs(t).sum(0)


BWD = [(1, 1, "f32", True, True), (1, 3200, "bf16", True, True), (3, 7, "bf16", False, True), (100, 3200, "f32", True, True),
       (257, 1001, "bf16", True, False), (33, 8640, "bf16", True, True), (700, 96, "f32", True, True),
       (2, 20011, "f32", True, True), (3, 70000, "bf16", True, True), (1, 131072, "f32", False, True),
       (1030, 520, "bf16", True, True)]


@pytest.mark.parametrize("M,K,hd,with_dh,wt", BWD)
def test_norm_backward(M, K, hd, with_dh, wt):
    """dX: rho g is within 3.5u, c h within 6.5u of its size and u of the absolute sum in it, and the two additions
    add 2u of their terms: 8u of the sum of the terms' sizes, and one rounding to H's type.  dW: M terms, each within
    3.5u, summed in any order: (M + 4) u of the sum of the sizes."""
    print("norm backward", M, K, hd, with_dh, wt, flush=True)
    dyt, dy = rows(M, K, 21, "f32", K + 3)
    ht, h = rows(M, K, 22, hd, K + 1, 2.0)
    dht, dh = rows(M, K, 23, hd) if with_dh else (None, None)
    w = (1.0 + 0.3 * synth.activations_f32(1, K, 24)[0]).astype(np.float32) if wt else None
    wd = None if w is None else to_dev(w)
    dX, dW = bl.norm_backward(dyt, ht, wd, eps=EPS, dH=dht)
    again = bl.norm_backward(dyt, ht, wd, eps=EPS, dH=dht)
    only_dx, none = bl.norm_backward(dyt, ht, wd, eps=EPS, dH=dht, want_dw=False)
    torch.cuda.synchronize()
    dx64, size, dw64, dw_size = bwd64(dy, h, w, dh, float(np.float32(EPS)))
    out = 2.0 ** -8 if hd == "bf16" else 0.0
    assert np.all(np.abs(values(dX) - dx64) <= 8 * U * size + out * np.abs(dx64) + 1e-40)
    assert np.all(np.abs(to_host(dW) - dw64) <= (M + 4) * U * dw_size + 1e-40)
    assert np.array_equal(to_host(again[0]), to_host(dX)) and np.array_equal(to_host(again[1]), to_host(dW))
    assert none is None and np.array_equal(to_host(only_dx), to_host(dX))
    if with_dh:  # the gradient of the residual stream updated in place
        alias = dht.clone()
        bl.norm_backward(dyt, ht, wd, eps=EPS, dH=alias, dX=alias)
        torch.cuda.synchronize()
        assert np.array_equal(to_host(alias), to_host(dX))


def test_norm_backward_differences():
    """Central differences of f = sum dY y(h, w) in binary64 (step 1e-5: truncation near 1e-10, rounding near 1e-11 of
    f's terms; the kernel's binary32 gradient is within 1e-5 of the largest)."""
    M, K = 2, 12
    dyt, dy = rows(M, K, 31, "f32")
    ht, h = rows(M, K, 32, "f32")
    w = (1.0 + 0.3 * synth.activations_f32(1, K, 33)[0]).astype(np.float32)
    dX, dW = bl.norm_backward(dyt, ht, to_dev(w), eps=EPS)
    f = lambda hh, ww: float((dy * norm64(hh, ww, EPS)[0]).sum())  # noqa: E731
    h64, w64, e = h.astype(np.float64), w.astype(np.float64), 1e-5
    for m in range(M):
        for k in range(K):
            d = np.zeros((M, K))
            d[m, k] = e
            assert abs((f(h64 + d, w64) - f(h64 - d, w64)) / (2 * e) - float(dX[m, k])) < 1e-5 * np.abs(dy).max()
    for k in range(K):
        d = np.zeros(K)
        d[k] = e
        assert abs((f(h64, w64 + d) - f(h64, w64 - d)) / (2 * e) - float(dW[k])) < 1e-5 * M * np.abs(dy).max()


def test_norm_backward_zero_row():
    dyt, _ = rows(3, 40, 41, "f32")
    h = torch.zeros((3, 40), device="cuda")
    dX, dW = bl.norm_backward(dyt, h, None, eps=0.0)
    torch.cuda.synchronize()
    assert not to_host(dX).any() and not to_host(dW).any()
