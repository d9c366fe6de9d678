"""int8 cache rows written and read back (q4g_kv_write_*_i8, q4g_kv_read_*_i8).

The format is exact: fp32 scale = amax / 127, codes clamp(rint(x / scale)), value
fp16(code * scale), with IEEE fp32 operations, so everything is compared bitwise with
numpy's and with the oracle's row quantiser; codes are also held to half a step of the
64-bit quotient. Rows that no call names keep a byte pattern."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q
from oracle import oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def sp():
    return torch.cuda.current_stream().cuda_stream


def rows_of(rng, n, n_kv, hd):
    """fp16 rows of many sizes; some zero, subnormal or at the type's largest value; ties."""
    x = rng.standard_normal((n, n_kv, hd)) * np.exp(2 * rng.standard_normal((n, n_kv, 1)))
    x = x.astype(np.float16)
    flat = x.reshape(-1, hd)
    for i in range(0, len(flat), 7):
        kind = (i // 7) % 5
        if kind == 0:
            flat[i] = 0
        elif kind == 1:
            flat[i] = rng.integers(-3, 4, hd) * np.float16(6e-8)
        elif kind == 2:
            flat[i, rng.integers(hd)] = 65504
        elif kind == 3:  # amax 127: scale 1, halves are ties
            flat[i] = rng.integers(-253, 254, hd) / 2
            flat[i, 0] = 127
        else:
            flat[i] = -flat[i]
    return x


def quantized(x):
    s = (np.abs(x.astype(np.float32)).max(-1) / np.float32(127)).astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))
    c = np.rint(x.astype(np.float32) / safe[..., None])
    return np.where(s[..., None] > 0, np.clip(c, -127, 127), 0).astype(np.int8), s


def values(c, s):
    return (c.astype(np.float32) * s[..., None]).astype(np.float16)


def empty_cache(shape, hd):
    return [torch.full(shape + (hd,), 77, dtype=torch.int8, device="cuda"),
            torch.full(shape, 5.5, dtype=torch.float32, device="cuda"),
            torch.full(shape + (hd,), 77, dtype=torch.int8, device="cuda"),
            torch.full(shape, 5.5, dtype=torch.float32, device="cuda")]


def ptrs(cache):
    return [t.data_ptr() for t in cache]


def on_gpu(x, stride):
    """x [n][n_kv][hd] with `stride` elements between rows; the gaps hold NaN."""
    n, n_kv, hd = x.shape
    buf = torch.full((max(n, 1), stride), float("nan"), dtype=torch.float16, device="cuda")
    buf[:n, :n_kv * hd] = torch.from_numpy(x.reshape(n, n_kv * hd)).cuda()
    return buf


@pytest.mark.parametrize("n,n_kv,hd,capacity,slot0,pad", [
    (1, 1, 512, 1, 0, 0), (1, 8, 256, 40, 39, 0), (37, 1, 512, 64, 13, 8), (300, 3, 256, 300, 0, 24),
    (1000, 2, 512, 5000, 1234, 0), (4099, 1, 256, 4100, 1, 128)])
def test_linear_write_then_read(n, n_kv, hd, capacity, slot0, pad):
    rng = np.random.default_rng(n + hd)
    k, v = rows_of(rng, n, n_kv, hd), rows_of(rng, n, n_kv, hd)
    stride = n_kv * hd + pad
    kd, vd = on_gpu(k, stride), on_gpu(v, stride)
    cache = empty_cache((capacity, n_kv), hd)
    Q.q4g_kv_write_linear_i8(kd.data_ptr(), vd.data_ptr(), n, stride, n_kv, hd, 0, slot0, capacity, *ptrs(cache), sp())
    for x, c, s in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        rc, rs = quantized(x)
        want_c = np.full((capacity, n_kv, hd), 77, np.int8)
        want_s = np.full((capacity, n_kv), 5.5, np.float32)
        want_c[slot0:slot0 + n], want_s[slot0:slot0 + n] = rc, rs
        np.testing.assert_array_equal(c.cpu().numpy(), want_c)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        # 64-bit: at most half a step off, but for the quotient's own fp32 rounding (127 * 2^-24)
        exact = x.astype(np.float64) / np.where(rs > 0, rs, 1).astype(np.float64)[..., None]
        assert np.max(np.abs(exact - rc)[rs > 0], initial=0) <= 0.5 + 127 * 2.0 ** -23
    ko, vo = torch.full_like(kd, 3.0), torch.full_like(vd, 3.0)
    Q.q4g_kv_read_linear_i8(*ptrs(cache), n_kv, hd, 0, slot0, capacity, n, ko.data_ptr(), vo.data_ptr(), stride, sp())
    for x, o in ((k, ko), (v, vo)):
        o = o.cpu().numpy()
        np.testing.assert_array_equal(o[:, :n_kv * hd].reshape(n, n_kv, hd), values(*quantized(x)))
        assert np.all(o[:, n_kv * hd:] == 3.0), "the gap between rows was written"


def test_the_oracles_quantiser_gives_the_same_rows():
    rng = np.random.default_rng(3)
    x = rows_of(rng, 60, 1, 256)
    cache = empty_cache((60, 1), 256)
    xd = on_gpu(x, 256)
    Q.q4g_kv_write_linear_i8(xd.data_ptr(), xd.data_ptr(), 60, 256, 1, 256, 0, 0, 60, *ptrs(cache), sp())
    for i in range(60):
        codes, scale = O.kv_quantize_row(x[i, 0].view(np.uint16))
        np.testing.assert_array_equal(cache[0][i, 0].cpu().numpy(), codes)
        assert float(cache[1][i, 0]) == float(np.float32(scale))


@pytest.mark.parametrize("n_kv,hd", [(1, 512), (4, 256)])
def test_slots_scatter_and_gather(n_kv, hd):
    rng = np.random.default_rng(n_kv)
    n, cap = 333, 1000
    k, v = rows_of(rng, n, n_kv, hd), rows_of(rng, n, n_kv, hd)
    slots = rng.permutation(cap)[:n].astype(np.int64)
    slots[5], slots[100], slots[332] = -1, cap, 2 ** 62  # skipped rows
    live = (slots >= 0) & (slots < cap)
    kd, vd = on_gpu(k, n_kv * hd), on_gpu(v, n_kv * hd)
    sd = torch.from_numpy(slots).cuda()
    cache = empty_cache((cap, n_kv), hd)
    Q.q4g_kv_write_linear_i8(kd.data_ptr(), vd.data_ptr(), n, n_kv * hd, n_kv, hd, sd.data_ptr(), 0, cap, *ptrs(cache),
                             sp())
    for x, c, s in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        rc, rs = quantized(x)
        want_c = np.full((cap, n_kv, hd), 77, np.int8)
        want_s = np.full((cap, n_kv), 5.5, np.float32)
        want_c[slots[live]], want_s[slots[live]] = rc[live], rs[live]
        np.testing.assert_array_equal(c.cpu().numpy(), want_c)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    ko, vo = torch.full_like(kd, 3.0), torch.full_like(vd, 3.0)
    Q.q4g_kv_read_linear_i8(*ptrs(cache), n_kv, hd, sd.data_ptr(), 0, cap, n, ko.data_ptr(), vo.data_ptr(), n_kv * hd,
                            sp())
    for x, o in ((k, ko), (v, vo)):
        want = np.where(live[:, None, None], values(*quantized(x)), np.float16(0))
        np.testing.assert_array_equal(o.cpu().numpy().reshape(n, n_kv, hd), want)
    same = torch.full((9,), int(slots[0]), dtype=torch.int64, device="cuda")  # a read may repeat a slot
    Q.q4g_kv_read_linear_i8(*ptrs(cache), n_kv, hd, same.data_ptr(), 0, cap, 9, ko.data_ptr(), vo.data_ptr(),
                            n_kv * hd, sp())
    assert torch.equal(ko[:9], ko[:1].expand(9, -1))


@pytest.mark.parametrize("n,ring,pos0", [(1, 1, 0), (5, 16, 14), (16, 16, 7), (40, 16, 1000003), (1531, 2048, 5000),
                                         (3, 512, 2 ** 62 + 511)])
@pytest.mark.parametrize("n_kv,hd", [(8, 256), (1, 512)])
def test_ring_write_then_read(n, ring, pos0, n_kv, hd):
    rng = np.random.default_rng(n + ring)
    k, v = rows_of(rng, n, n_kv, hd), rows_of(rng, n, n_kv, hd)
    kd, vd = on_gpu(k, n_kv * hd), on_gpu(v, n_kv * hd)
    cache = empty_cache((n_kv, ring), hd)
    Q.q4g_kv_write_ring_i8(kd.data_ptr(), vd.data_ptr(), n, n_kv * hd, n_kv, hd, pos0, ring, *ptrs(cache), sp())
    for x, c, s in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        rc, rs = quantized(x)
        want_c = np.full((n_kv, ring, hd), 77, np.int8)
        want_s = np.full((n_kv, ring), 5.5, np.float32)
        for t in range(n):  # in order: a later row replaces an older one
            want_c[:, (pos0 + t) % ring], want_s[:, (pos0 + t) % ring] = rc[t], rs[t]
        np.testing.assert_array_equal(c.cpu().numpy(), want_c)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    m = min(n, ring)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    Q.q4g_kv_read_ring_i8(*ptrs(cache), n_kv, hd, pos0 + n - m, ring, m, ko.data_ptr(), vo.data_ptr(), n_kv * hd, sp())
    for x, o in ((k, ko), (v, vo)):
        np.testing.assert_array_equal(o[:m].cpu().numpy().reshape(m, n_kv, hd), values(*quantized(x))[n - m:])


def test_rows_that_are_not_finite():
    """A NaN takes code 0 and leaves its row alone; an infinite value makes the row read as NaN."""
    x = np.ones((3, 1, 256), np.float16)
    x[0, 0, 7], x[1, 0, 9], x[2] = np.nan, np.inf, np.nan
    xd = on_gpu(x, 256)
    cache = empty_cache((3, 1), 256)
    Q.q4g_kv_write_linear_i8(xd.data_ptr(), xd.data_ptr(), 3, 256, 1, 256, 0, 0, 3, *ptrs(cache), sp())
    c, s = cache[0].cpu().numpy()[:, 0], cache[1].cpu().numpy()[:, 0]
    assert c[0, 7] == 0 and np.all(np.delete(c[0], 7) == 127) and s[0] == np.float32(1) / np.float32(127)
    assert np.isinf(s[1]) and np.all(c[1] == 0) and s[2] == 0 and np.all(c[2] == 0)
    o = torch.empty((3, 256), dtype=torch.float16, device="cuda")
    Q.q4g_kv_read_linear_i8(*ptrs(cache), 1, 256, 0, 0, 3, 3, o.data_ptr(), o.data_ptr(), 256, sp())
    o = o.cpu().numpy()
    assert np.all(np.isnan(o[1])) and np.all(o[2] == 0) and o[0, 7] == 0


def test_row_offsets_beyond_32_bits():
    """Cache rows whose byte offset passes 2^32 (a 5 GB cache)."""
    cap, hd = (1 << 32) // 512 + 4096, 512
    cache = [torch.empty((cap, 1, hd), dtype=torch.int8, device="cuda"),
             torch.empty((cap, 1), dtype=torch.float32, device="cuda")]
    rng = np.random.default_rng(8)
    x = rows_of(rng, 20, 1, hd)
    xd = on_gpu(x, hd)
    both = [cache[0].data_ptr(), cache[1].data_ptr()]
    # K and V may share a cache when they share rows: both writes store the same bytes
    Q.q4g_kv_write_linear_i8(xd.data_ptr(), xd.data_ptr(), 20, hd, 1, hd, 0, cap - 20, cap, *both, *both, sp())
    rc, rs = quantized(x)
    np.testing.assert_array_equal(cache[0][cap - 20:].cpu().numpy(), rc)
    np.testing.assert_array_equal(cache[1][cap - 20:].cpu().numpy(), rs)
    o = torch.empty((20, hd), dtype=torch.float16, device="cuda")
    Q.q4g_kv_read_linear_i8(*both, *both, 1, hd, 0, cap - 20, cap, 20, o.data_ptr(), o.data_ptr(), hd, sp())
    np.testing.assert_array_equal(o.cpu().numpy(), values(rc, rs)[:, 0])


def test_captured_and_replayed_on_another_stream():
    rng = np.random.default_rng(1)
    k = rows_of(rng, 6, 1, 512)
    kd = on_gpu(k, 512)
    cache = empty_cache((32, 1), 512)
    o = torch.zeros((6, 512), dtype=torch.float16, device="cuda")
    slots = torch.arange(6, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        Q.q4g_kv_write_linear_i8(kd.data_ptr(), kd.data_ptr(), 6, 512, 1, 512, slots.data_ptr(), 0, 32, *ptrs(cache),
                                 sp())
        Q.q4g_kv_read_linear_i8(*ptrs(cache), 1, 512, slots.data_ptr(), 0, 32, 6, o.data_ptr(), o.data_ptr(), 512, sp())
    for shift in (0, 20):
        slots.copy_(torch.arange(6, device="cuda") + shift)
        kd.copy_(torch.from_numpy(np.roll(k, shift + 1, 0).reshape(6, 512)))
        g.replay()
        torch.cuda.synchronize()
        rc, rs = quantized(np.roll(k, shift + 1, 0))
        np.testing.assert_array_equal(cache[0][shift:shift + 6].cpu().numpy(), rc)
        np.testing.assert_array_equal(o.cpu().numpy(), values(rc, rs)[:, 0])
