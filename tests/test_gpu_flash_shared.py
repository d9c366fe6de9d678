"""q4g_flash_decode_shared and _i8 against softmax(q K^T) V in 64 bits.

Tolerance, per output element. Scores: products of fp16 values (or of fp16 and int8
codes) are exact in fp32 and a sum over head_dim runs in at most head_dim / 16 + 16
steps of relative error 2^-23, one more for a row's scale, so a score is off by at
most D = (hd / 16 + 18) 2^-23 max sum|q k| and a probability by the factor e^(2 D). The
probabilities (times an int8 row's scale) enter the second product as fp16: 2^-11
relative, or 2^-32 of the row's largest when they fall below fp16's normal range. The
result is rounded to fp16 (2^-11, or 2^-25 absolute). With a = sum p |v|:
  |o - o64| <= 2^-11 |o64| + (2^-11 + 2 D + 2^-20) a + keys 2^-32 max|v| + 2^-25."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def sp():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, sigma):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).half()


class Batch:
    def __init__(self, batch, n_q, n_kv, hd, prefix, cap, lens, i8=False, seed=0, peak=2.0):
        g = gen(seed)
        self.dims = (batch, n_q, n_kv, hd)
        self.prefix, self.cap, self.i8 = prefix, cap, i8
        self.q = normal(g, (batch, n_q, hd), peak * hd ** -0.25)
        shapes = [(prefix, n_kv, hd), (prefix, n_kv, hd), (batch, cap, n_kv, hd), (batch, cap, n_kv, hd)]
        sig = [hd ** -0.25, 1.0, hd ** -0.25, 1.0]
        if i8:
            self.kv = [(torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8),
                        (0.5 + torch.rand(s[:-1], generator=g, device="cuda")) * w / 73) for s, w in zip(shapes, sig)]
        else:
            self.kv = [normal(g, s, w) for s, w in zip(shapes, sig)]
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda") if cap else None
        self.out = torch.full((batch, n_q, hd), 7.0, dtype=torch.float16, device="cuda")
        nb = Q.q4g_flash_decode_shared_workspace_bytes(batch, n_q, n_kv, hd)
        self.ws = torch.full((nb,), 0xff, dtype=torch.uint8, device="cuda")  # NaN patterns

    def run(self):
        ptr = lambda t: t.data_ptr() if t is not None and t.numel() else 0  # noqa: E731
        tail = (self.cap, ptr(self.len), self.out.data_ptr(), self.ws.data_ptr(), self.ws.numel(), sp())
        if self.i8:
            kp, vp, ko, vo = [[ptr(c), ptr(s)] for c, s in self.kv]
            Q.q4g_flash_decode_shared_i8(self.q.data_ptr(), *self.dims, *kp, *vp, self.prefix, *ko, *vo, *tail)
        else:
            kp, vp, ko, vo = [ptr(t) for t in self.kv]
            Q.q4g_flash_decode_shared(self.q.data_ptr(), *self.dims, kp, vp, self.prefix, ko, vo, *tail)
        return self.out

    def rows(self, i, h, b=None):
        t = self.kv[i]
        if self.i8:
            c, s = (t[0][..., h, :], t[1][..., h]) if b is None else (t[0][b, :, h], t[1][b, :, h])
            return c.double() * s.double()[..., None]
        return (t[:, h] if b is None else t[b, :, h]).double()

    def check(self):
        batch, n_q, n_kv, hd = self.dims
        got = self.out.double()
        G = n_q // n_kv
        lens = [0] * batch if self.len is None else [min(max(int(n), 0), self.cap) for n in self.len.tolist()]
        for h in range(n_kv):
            kp, vp = self.rows(0, h), self.rows(1, h)
            for b in range(batch):
                n = lens[b]
                k = torch.cat([kp, self.rows(2, h, b)[:n]]) if self.cap else kp
                v = torch.cat([vp, self.rows(3, h, b)[:n]]) if self.cap else vp
                o = got[b, h * G:(h + 1) * G]
                if k.shape[0] == 0:
                    assert torch.all(o == 0), f"sequence {b} has no row and is not zero"
                    continue
                q = self.q[b, h * G:(h + 1) * G].double()
                p = torch.softmax(q @ k.t(), dim=-1)
                ref, a = p @ v, p @ v.abs()
                D = (hd / 16 + 18) * 2.0 ** -23 * (q.abs() @ k.abs().t()).amax(dim=-1, keepdim=True)
                tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2 * D + 2.0 ** -20) * a + \
                    k.shape[0] * 2.0 ** -32 * v.abs().max() + 2.0 ** -25
                bad = (o - ref).abs() > tol
                assert not bool(bad.any()) and not bool(torch.isnan(o).any()), \
                    f"sequence {b} kv head {h}: {int(bad.sum())} off, worst {float(((o - ref).abs() / tol).max())}"


SHAPES = [(16, 1, 512), (16, 8, 256), (8, 2, 256)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("batch,prefix,cap,lens", [
    (1, 1, 0, []), (1, 0, 1, [1]), (2, 100, 32, [0, 32]), (3, 127, 5, [5, 0, 1]), (3, 128, 130, [129, 128, 127]),
    (5, 129, 300, [300, 1, 0, 255, 257]), (4, 2000, 64, [64, 63, 33, 1]), (9, 0, 200, [0, 1, 200, 3, 0, 77, 128, 9, 64])])
def test_against_64_bits(batch, prefix, cap, lens, n_q, n_kv, hd, i8):
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens, i8, seed=prefix + batch)
    t.run()
    t.check()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("batch,n_q,n_kv,hd,prefix,cap", [
    (33, 16, 1, 512, 5003, 40), (64, 16, 8, 256, 1000, 17), (17, 24, 8, 256, 777, 100), (2, 96, 1, 512, 3001, 70),
    (1, 256, 2, 256, 513, 130), (256, 8, 1, 512, 300, 3), (7, 5, 5, 512, 1025, 20), (3, 16, 1, 512, 40000, 1000)])
def test_many_rows_heads_and_sequences(batch, n_q, n_kv, hd, prefix, cap, i8):
    lens = np.random.default_rng(batch).integers(0, cap + 1, batch).tolist()
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens, i8, seed=batch)
    t.run()
    t.check()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("batch,n_q,n_kv,hd,prefix,cap", [(130, 128, 2, 512, 1000, 5), (130, 130, 2, 512, 1000, 0),
                                                          (100, 64, 1, 256, 1500, 300), (256, 96, 3, 256, 700, 40)])
def test_many_segments_of_many_tiles_per_cta(batch, n_q, n_kv, hd, prefix, cap, i8):
    """More units than CTAs, each of several tiles: every ring is full of the next segment's
    rows while one ends. Right, and the same bits each time."""
    lens = np.random.default_rng(n_q).integers(0, cap + 1, batch).tolist()
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens if cap else [], i8, seed=prefix)
    first = t.run().clone()
    t.check()
    for _ in range(40):
        t.out.zero_()
        assert torch.equal(t.run(), first)


@pytest.mark.parametrize("i8", [False, True])
def test_rows_behind_the_length_are_never_used(i8):
    """Own rows from own_len on hold NaN and infinities, and so does what surrounds them."""
    t = Batch(4, 16, 1, 512, 300, 150, [0, 1, 129, 100], i8, seed=3)
    for b, n in enumerate([0, 1, 129, 100]):
        for x in t.kv[2:]:
            if i8:
                x[1][b, n:] = float("nan") if b % 2 else float("inf")
            else:
                x[b, n:] = float("nan") if b % 2 else float("inf")
    t.run()
    for x in t.kv[2:]:
        for b, n in enumerate([0, 1, 129, 100]):
            (x[1] if i8 else x)[b, n:] = 0
    t.check()


def test_lengths_outside_the_capacity_are_clamped():
    t = Batch(3, 16, 1, 512, 50, 20, [-5, 21, 2 ** 31 - 1], seed=4)
    t.run()
    t.check()


@pytest.mark.parametrize("i8", [False, True])
def test_sharp_and_rising_scores(i8):
    """Scores that rise along the keys by far more than fp16's exponent range, and a
    softmax that one key takes."""
    t = Batch(4, 16, 1, 512, 1500, 40, [40, 3, 0, 17], i8, seed=5, peak=30.0)
    ramp = torch.linspace(0, 3, 1500, device="cuda")[:, None, None]
    d = torch.randn(512, device="cuda") * 512 ** -0.25
    if not i8:
        t.kv[0] = (t.kv[0].float() + ramp * d).half()
        t.q = (t.q.float() * 0.2 + 3 * d).half()
    t.run()
    t.check()


def test_row_scales_of_many_sizes():
    """int8 rows whose scales differ by many powers of two, zero among them."""
    t = Batch(3, 16, 1, 512, 700, 30, [30, 0, 11], True, seed=6)
    for i, x in enumerate(t.kv):
        if i % 2 == 1:
            e = torch.randint(-24, 9, x[1].shape, generator=gen(i), device="cuda")
            x[1].copy_(torch.exp2(e.float()))
            x[1][..., 0][torch.rand(x[1].shape[:-1], generator=gen(9 + i), device="cuda") < 0.2] = 0.0
    t.run()
    t.check()


@pytest.mark.parametrize("i8", [False, True])
def test_all_values_zero(i8):
    t = Batch(2, 16, 1, 512, 200, 10, [10, 0], i8, seed=7)
    for x in (t.kv[1], t.kv[3]):
        (x[1] if i8 else x).zero_()
    t.run()
    assert torch.all(t.out == 0)


@pytest.mark.parametrize("n_q,n_kv,hd", SHAPES)
def test_no_rows_at_all(n_q, n_kv, hd):
    for cap, lens in ((0, []), (40, [0, -1, 0])):
        t = Batch(3, n_q, n_kv, hd, 0, cap, lens)
        assert torch.all(t.run() == 0)


def test_row_offsets_beyond_32_bits():
    """A prefix whose K and V pass 4 GB each; the reference runs in pieces of keys."""
    P, hd, batch = 4_300_077, 512, 2
    t = Batch(batch, 16, 1, hd, 0, 8, [8, 3], seed=12)
    t.prefix = P
    t.kv[0] = torch.empty((P, 1, hd), dtype=torch.float16, device="cuda")
    t.kv[1] = torch.empty((P, 1, hd), dtype=torch.float16, device="cuda")
    g = gen(13)
    step = 1 << 18
    for x, w in zip(t.kv[:2], (hd ** -0.25, 1.0)):
        for i in range(0, P, step):
            x[i:i + step] = normal(g, x[i:i + step].shape, w)
    t.kv[0][-5:] *= 3  # the last rows count
    t.run()
    q = t.q.double()
    for b in range(batch):
        n = int(t.len[b])
        own = (t.rows(2, 0, b)[:n], t.rows(3, 0, b)[:n])
        m = torch.full((16, 1), -1e300, dtype=torch.float64, device="cuda")
        l, o, a, D, vmax = 0.0, 0.0, 0.0, 0.0, 0.0
        for i in list(range(0, P, step)) + [None]:
            k, v = own if i is None else (t.kv[0][i:i + step, 0].double(), t.kv[1][i:i + step, 0].double())
            s = q[b] @ k.t()
            new = torch.maximum(m, s.amax(-1, keepdim=True))
            f, p = torch.exp(m - new), torch.exp(s - new)
            l, o, a, m = l * f + p.sum(-1, keepdim=True), o * f + p @ v, a * f + p @ v.abs(), new
            D = max(D, (hd / 16 + 18) * 2.0 ** -23 * float((q[b].abs() @ k.abs().t()).amax()))
            vmax = max(vmax, float(v.abs().max()))
        ref, a = o / l, a / l
        tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2 * D + 2.0 ** -20) * a + (P + n) * 2.0 ** -32 * vmax + 2.0 ** -25
        assert bool(((t.out[b].double() - ref).abs() <= tol).all()), b


def test_same_as_one_sequence_after_the_other():
    """Against the one-sequence entry point over prefix and own rows laid end to end."""
    t = Batch(3, 16, 1, 512, 1000, 50, [50, 1, 30], seed=8)
    t.run()
    nb = Q.q4g_flash_decode_workspace_bytes(16, 512)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    for b, n in enumerate([50, 1, 30]):
        k = torch.cat([t.kv[0], t.kv[2][b, :n]]).contiguous()
        v = torch.cat([t.kv[1], t.kv[3][b, :n]]).contiguous()
        o = torch.empty((16, 512), dtype=torch.float16, device="cuda")
        Q.q4g_flash_decode_linear(t.q[b].data_ptr(), 16, 1, 512, k.data_ptr(), v.data_ptr(), 1000 + n, o.data_ptr(),
                                  ws.data_ptr(), nb, sp())
        assert float((o.float() - t.out[b].float()).abs().max()) <= 4e-3


@pytest.mark.parametrize("i8", [False, True])
def test_a_nan_stays_with_its_sequence(i8):
    """A NaN among one sequence's queries or own rows reaches that sequence alone."""
    t = Batch(6, 16, 1, 512, 500, 40, [40, 7, 30, 0, 5, 40], i8, seed=14)
    clean = t.run().clone()
    t.q[1, 3, 100] = float("nan")
    if i8:
        t.kv[2][1][2, 4] = float("nan")
        t.kv[3][1][5, 39] = float("nan")
    else:
        t.kv[2][2, 4, 0, 9] = float("nan")
        t.kv[3][5, 39, 0, 11] = float("nan")
    out = t.run()
    assert torch.equal(out[[0, 3, 4]], clean[[0, 3, 4]])
    assert torch.all(torch.isnan(out[1, 3])) and torch.equal(out[1, :3], clean[1, :3])
    assert torch.equal(out[1, 4:], clean[1, 4:]) and torch.all(torch.isnan(out[2]))
    if i8:
        assert torch.all(torch.isnan(out[5]))
    else:
        assert torch.all(torch.isnan(out[5, :, 11])) and torch.equal(out[5, :, :11], clean[5, :, :11])


def test_two_calls_at_once():
    """Two streams, a workspace each, many calls in flight: the same bits as alone."""
    a = Batch(9, 16, 1, 512, 4000, 200, [200, 1, 0, 33, 150, 128, 64, 90, 17], seed=15)
    b = Batch(12, 16, 8, 256, 700, 60, list(range(0, 60, 5)), True, seed=16)
    want = [t.run().clone() for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for t, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                t.out.zero_()
                t.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_repeats_bitwise_and_leaves_inputs_alone():
    t = Batch(6, 16, 1, 512, 3000, 64, [64, 0, 5, 32, 63, 1], seed=9)
    before = [x.clone() for x in t.kv] + [t.q.clone()]
    first = t.run().clone()
    for _ in range(3):
        t.out.fill_(0)
        assert torch.equal(t.run(), first)
    for a, b in zip(before, t.kv + [t.q]):
        assert torch.equal(a, b)


def test_two_graphs_share_a_workspace_and_lengths_change():
    """Two captured calls on one workspace, replayed in turn on a stream of their own, the
    lengths changed in between."""
    a = Batch(4, 16, 1, 512, 900, 80, [1, 2, 3, 4], seed=10)
    b = Batch(4, 16, 8, 256, 500, 80, [80, 0, 9, 40], True, seed=11)
    big = a.ws if a.ws.numel() > b.ws.numel() else b.ws
    a.ws = b.ws = big
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            t.run()
        graphs.append(g)
    for step in range(3):
        for t, g in zip((a, b), graphs):
            t.len.add_(7 * step)
            t.out.fill_(5)
            g.replay()
            torch.cuda.synchronize()
            t.check()
