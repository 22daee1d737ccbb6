"""The int8 key / value cache: every byte and scale that a write leaves, and what
reads give back, against numpy (bit for bit: one reciprocal and one product per
row, one product and one rounding per value, each in binary32)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402
from ternary_weight_linear_forward_amd import synth  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu


def place(t):
    return 16 * ((t % 16) // 4) + 8 * ((t % 64) // 32) + 4 * ((t % 32) // 16) + t % 4


def make(pages, heads, D, page, fill=77):
    c = bl.KVCache.empty(pages, heads, D, page)
    c.k.fill_(fill), c.v.fill_(fill), c.k_scale.fill_(-3.0), c.v_scale.fill_(-3.0)
    return c


def quant(x):
    """[T, H, D] fp32 -> int8 bytes, scales."""
    f = np.float32
    top = np.abs(x).max(-1)
    pre = np.where(top < f(2.0 ** -96), f(2.0 ** 64), f(1))
    safe = np.where(top > 0, top * pre, f(1))
    s = np.where(top > 0, f(127) * (f(1) / safe), f(0)).astype(np.float32)
    q = np.rint((x * pre[..., None]) * s[..., None])
    assert np.abs(q).max() <= 127
    return q.astype(np.int8), top / f(127)


def kv_input(T, H, D, seed, dtype, order):
    """[T, H, D] tensor of the given memory order, and its fp32 values."""
    x = synth.activations_f32(T * H, D, seed).reshape(T, H, D)
    if T * H > 3:
        x[T // 2, H // 2] = 0.0
        x[0, 0] *= np.float32(1e-39)
    bits = synth.to_bf16_bits(x) if dtype == "bf16" else x
    v = synth.bf16_bits_to_f32(bits) if dtype == "bf16" else x
    if order == "thd":
        t = to_dev(bits)
    elif order == "htd":  # head-major memory
        t = to_dev(np.ascontiguousarray(bits.transpose(1, 0, 2))).transpose(0, 1)
    else:                 # rows inside a wider, oddly aligned buffer
        buf = np.zeros((T, H * D + 5), bits.dtype)
        buf[:, 3:3 + H * D] = bits.reshape(T, H * D)
        t = to_dev(buf)[:, 3:3 + H * D].view(T, H, D)
    return t, v


CASES = [  # T, heads, D, page, dtype, order, slots
    (1, 1, 1, 64, "f32", "thd", "spread"), (1, 8, 128, 64, "bf16", "thd", "spread"), (16, 8, 128, 128, "bf16", "thd", "spread"),
    (64, 3, 100, 64, "f32", "htd", "run"), (200, 2, 128, 64, "bf16", "htd", "run"), (130, 5, 80, 192, "f32", "odd", "run"),
    (333, 2, 64, 256, "bf16", "odd", "run+7"), (500, 3, 100, 64, "bf16", "thd", "run+1"), (77, 2, 256, 64, "f32", "thd", "reverse"),
    (90, 1, 17, 128, "bf16", "odd", "spread"), (257, 4, 128, 64, "f32", "thd", "run+4"), (40, 33, 48, 64, "bf16", "thd", "holes"),
]


def slots_of(kind, T, page, rng):
    pages = (T + 80) // page + 3
    if kind == "spread":
        pages = T + 2
        return pages, rng.permutation(pages)[:T] * page + rng.integers(0, page, T)
    start = int(kind.split("+")[1]) if "+" in kind else 0
    t = np.arange(T) + start
    s = rng.permutation(pages)[t // page] * page + t % page
    if kind == "reverse":
        s = s[::-1].copy()
    if kind == "holes":
        s[::3] = np.array([-1, pages * page, -(1 << 40), 1 << 50])[np.arange(len(s[::3])) % 4]
    return pages, s


@pytest.mark.parametrize("T,H,D,page,dtype,order,kind", CASES)
def test_write_and_read(T, H, D, page, dtype, order, kind):
    print("cache", T, H, D, page, dtype, order, kind, flush=True)
    pages, s = slots_of(kind, T, page, np.random.default_rng(T + D))
    c = make(pages, H, D, page)
    kt, k = kv_input(T, H, D, 1, dtype, order)
    vt, v = kv_input(T, H, D, 2, dtype, order)
    st = to_dev(s.astype(np.int64))
    bl.cache_write(c, kt, vt, st)
    torch.cuda.synchronize()
    Dp = (D + 15) // 16 * 16
    wk, wv = np.full((pages, H, page, Dp), 77, np.int8), np.full((pages, H, page // 64, Dp, 64), 77, np.int8)
    wks, wvs = np.full((pages, H, page), -3, np.float32), np.full((pages, H, page), -3, np.float32)
    kq, kr = quant(k)
    vq, vr = quant(v)
    inside = (s >= 0) & (s < pages * page)
    for i in np.flatnonzero(inside):
        p, t = divmod(int(s[i]), page)
        wk[p, :, t] = 0
        wk[p, :, t, :D] = kq[i]
        wv[p, :, t // 64, :, place(t)] = 0
        wv[p, :, t // 64, :D, place(t)] = vq[i]
        wks[p, :, t], wvs[p, :, t] = kr[i], vr[i]
    assert np.array_equal(to_host(c.k), wk) and np.array_equal(to_host(c.k_scale), wks)
    assert np.array_equal(to_host(c.v), wv) and np.array_equal(to_host(c.v_scale), wvs)
    for out in (torch.float32, torch.bfloat16):
        gk, gv = bl.cache_read(c, st, dtype=out)
        torch.cuda.synchronize()
        for g, q, r in ((gk, kq, kr), (gv, vq, vr)):
            want = np.where(inside[:, None, None], q.astype(np.float32) * r[..., None], np.float32(0))
            if out == torch.bfloat16:
                assert np.array_equal(synth.bf16_bits_to_f32(to_host(g)), synth.bf16_bits_to_f32(synth.to_bf16_bits(want)))
            else:
                assert np.array_equal(to_host(g), want)


def test_empty_write_and_read():
    c = make(1, 2, 16, 64)
    e = torch.empty((0, 2, 16), device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    bl.cache_write(c, e, e, s)
    k, v = bl.cache_read(c, s, dtype=torch.float32)
    torch.cuda.synchronize()
    assert k.shape == (0, 2, 16) and v.shape == (0, 2, 16) and int((c.k != 77).sum()) == 0


def test_read_into_strided_rows():
    """cache_read writes only the rows' own elements."""
    c = make(2, 2, 20, 64)
    k, _ = kv_input(70, 2, 20, 5, "f32", "thd")
    s = torch.arange(70, device="cuda")
    bl.cache_write(c, k, k, s)
    K = torch.full((70, 2, 27), -5.0, device="cuda")
    V = torch.full((2, 70, 23), -5.0, device="cuda")
    st = bl.bitlinear_cache_read(c.desc, s.data_ptr(), 70, K.data_ptr(), 54, 27, V.data_ptr(), 23, 70 * 23, bl.F32,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == bl.OK
    ck, cv = bl.cache_read(c, s, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(K[:, :, :20], ck) and torch.equal(V.transpose(0, 1)[:, :, :20], cv)
    assert bool((K[:, :, 20:] == -5).all()) and bool((V[:, :, 20:] == -5).all())


def test_offsets_beyond_32_bits():
    """Slots whose bytes lie past 2^32: 5 GB of keys, written and read at both ends."""
    D, H, page = 256, 16, 1024
    pages = 1100  # 1100 * 16 * 1024 * 256 = 4.6e9 bytes of K
    c = bl.KVCache.empty(pages, H, D, page)
    s = np.array([0, pages * page - 1, pages * page - 64, 1050 * page + 5], np.int64)
    kt, k = kv_input(4, H, D, 8, "f32", "thd")
    vt, v = kv_input(4, H, D, 9, "f32", "thd")
    bl.cache_write(c, kt, vt, to_dev(s))
    gk, gv = bl.cache_read(c, to_dev(s), dtype=torch.float32)
    torch.cuda.synchronize()
    for g, x in ((gk, k), (gv, v)):
        q, r = quant(x)
        assert np.array_equal(to_host(g), q.astype(np.float32) * r[..., None])
    p, t = divmod(int(s[3]), page)
    assert np.array_equal(to_host(c.k[p, :, t, :D]), quant(k)[0][3])
