"""q4g_token_logprobs against its formulas in 64 bits.

Tolerance. d = (x - m) / T costs two roundings of 2^-24 |d|; a term exp(d) costs 2^-22
(the instruction) and, at exp(d) |d| <= 1, 2^-22 more through d; a sum of n terms in
fp32 adds up to n * 2^-24, where one thread sums at most n = vocab / 256 + 32 terms and
lists of 16 join. So |ln S| is off by at most A = (n + 16) * 2^-24, a log probability by
A + 2^-22 |d|, and the entropy, whose second part is a ratio of two such sums of size at
most ln(vocab), by A * (2 + 2 ln vocab)."""
from __future__ import annotations

import math

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


def run(x, targets, T=1.0, n=0, stride=None, skew=0):
    rows, vocab = x.shape
    stride = stride or vocab
    buf = torch.full((rows * stride + skew + 8,), float("nan"), dtype=torch.float32, device="cuda")
    view = torch.as_strided(buf, (rows, vocab), (stride, 1), skew)
    view.copy_(torch.as_tensor(x))
    t = torch.as_tensor(targets, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 9.0, dtype=torch.float32, device="cuda")
    ent = torch.full((rows,), 9.0, dtype=torch.float32, device="cuda")
    ids = torch.full((rows, max(n, 1)), -9, dtype=torch.int32, device="cuda")
    tops = torch.full((rows, max(n, 1)), 9.0, dtype=torch.float32, device="cuda")
    Q.q4g_token_logprobs(view.data_ptr(), rows, vocab, stride, T, t.data_ptr(), lp.data_ptr(), ent.data_ptr(), n,
                         ids.data_ptr(), tops.data_ptr(), torch.cuda.current_stream().cuda_stream)
    return [a.cpu().numpy() for a in (lp, ent, ids[:, :n], tops[:, :n])]


def as_fp32(want):
    """A value beyond fp32's range, as (lowest - 1) / 0.5 = -6.8e38, is -inf in an fp32
    output: rounding to nearest takes |want| >= 2^128 - 2^103 to infinity."""
    return math.copysign(math.inf, want) if abs(want) >= 2.0 ** 128 - 2.0 ** 103 else want


def check(x, targets, T=1.0, n=0, **kw):
    lp, ent, ids, tops = run(x, targets, T, n, **kw)
    x = np.asarray(x, np.float32)
    rows, vocab = x.shape
    A = (vocab / 256 + 48) * 2.0 ** -24
    for r in range(rows):
        m = float(x[r].max())
        d = (x[r].astype(np.float64) - m) / float(np.float32(T))
        w = np.exp(d)
        S = w.sum()
        H = math.log(S) - (w[w > 0] * d[w > 0]).sum() / S
        t = int(targets[r])
        if 0 <= t < vocab:
            want = as_fp32(d[t] - math.log(S))
            assert (lp[r] == want) if math.isinf(want) else abs(lp[r] - want) <= A + 2.0 ** -22 * abs(d[t]), (r, lp[r], want)
        else:
            assert math.isnan(lp[r])
        assert abs(ent[r] - H) <= A * (2 + 2 * math.log(vocab)), (r, ent[r], H)
        order = np.argsort(-x[r], kind="stable")[:n]
        np.testing.assert_array_equal(ids[r], order)
        for got, want in zip(tops[r], map(as_fp32, d[order] - math.log(S))):
            assert (got == want) if math.isinf(want) else abs(got - want) <= A + 2.0 ** -22 * abs(want)


@pytest.mark.parametrize("rows,vocab,n,T", [
    (1, 1, 1, 1.0), (3, 2, 2, 1.0), (2, 33, 32, 0.7), (5, 1000, 0, 1.0), (4, 4096, 8, 1.0), (7, 4097, 20, 1.3),
    (2, 32003, 32, 0.25), (1, 262144, 8, 1.0), (6, 262144, 20, 1.0), (40, 65537, 1, 2.0), (300, 5003, 5, 1.0)])
def test_random_rows(rows, vocab, n, T):
    rng = np.random.default_rng(rows + vocab)
    x = (30 * np.tanh(rng.standard_normal((rows, vocab)) * 0.1)).astype(np.float32)
    check(x, rng.integers(0, vocab, rows), T, n)


@pytest.mark.parametrize("skew,pad", [(1, 0), (2, 1), (3, 3), (0, 5), (1, 7)])
def test_strides_and_alignments(skew, pad):
    rng = np.random.default_rng(skew + pad)
    x = rng.standard_normal((9, 8191)).astype(np.float32) * 4
    check(x, rng.integers(0, 8191, 9), 1.0, 6, stride=8191 + pad, skew=skew)


def test_orders_and_ties():
    """Rising and falling rows (every tile beats the last, or none does), constant rows,
    few distinct values, signed zeros: the lowest index first among equals."""
    V = 70001
    rng = np.random.default_rng(0)
    up = np.linspace(-20, 20, V, dtype=np.float32)
    rows = [up, up[::-1].copy(), np.zeros(V, np.float32), rng.integers(0, 3, V).astype(np.float32),
            np.where(rng.random(V) < 0.5, np.float32(0.0), np.float32(-0.0)), np.full(V, -7.25, np.float32)]
    check(np.stack(rows), [0, V - 1, 5, 17, 3, 2], 1.0, 32)


def test_masked_rows():
    """-inf and the type's lowest value in masked places, down to one live logit and to none."""
    V = 20000
    rng = np.random.default_rng(5)
    x = rng.standard_normal((5, V)).astype(np.float32)
    x[0, rng.random(V) < 0.9] = -np.inf
    x[1] = -np.inf
    x[1, 12345] = 3.0
    x[2, rng.random(V) < 0.9] = np.finfo(np.float32).min
    x[3] = np.finfo(np.float32).min
    x[4] = -np.inf
    x[4, :7] = np.finfo(np.float32).min
    check(x, [0, 12345, 1, 2, 3], 1.0, 12)
    check(x, [V - 1, 7, 1, 2, 9], 0.5, 12)
    lp, ent, ids, tops = run(np.full((2, V), -np.inf, np.float32), [3, -1], 1.0, 4)
    assert lp[0] == -np.inf and np.isnan(lp[1]) and np.all(ent == 0)
    np.testing.assert_array_equal(ids, np.tile(np.arange(4), (2, 1)))
    assert np.all(tops == -np.inf)


def test_targets_outside_the_vocabulary():
    x = np.random.default_rng(1).standard_normal((4, 500)).astype(np.float32)
    check(x, [-1, 500, 2 ** 31 - 1, -2 ** 31], 1.0, 3)


def test_rows_that_are_not_finite():
    x = np.random.default_rng(2).standard_normal((3, 9000)).astype(np.float32)
    x[0, 100], x[1, 8999], x[2] = np.nan, np.inf, np.nan
    lp, ent, ids, tops = run(x, [5, 6, 7], 1.0, 8)
    assert np.all(np.isnan(lp)) and np.all(np.isnan(ent)) and np.all(np.isnan(tops))
    assert np.all((ids >= 0) & (ids < 9000))
    lp, ent, ids, tops = run(x[:1, 200:700], [5], 1.0, 8)  # the rows beside it are unaffected
    assert np.all(np.isfinite(lp)) and np.all(np.isfinite(tops))


def test_extreme_spread_and_temperature():
    x = np.zeros((4, 1000), np.float32)
    x[0, 3], x[0, 4] = 3e38, -3e38
    x[1, 1], x[2, 2] = 100.0, 1e-30
    for T in (1e-3, 1.0, 1e3, 1e38):
        check(x, [3, 1, 2, 0], T, 4)


def test_same_bits_every_time_and_no_output_past_the_rows():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((3, 262144)).astype(np.float32)
    a = run(x, [1, 2, 3], 1.0, 20)
    for _ in range(4):
        b = run(x, [1, 2, 3], 1.0, 20)
        for u, v in zip(a, b):
            np.testing.assert_array_equal(u, v)


def test_outputs_that_are_not_wanted():
    x = torch.randn(2, 3000, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    ent = torch.full((4,), 9.0, device="cuda")
    ids = torch.full((3, 2), -9, dtype=torch.int32, device="cuda")
    Q.q4g_token_logprobs(x.data_ptr(), 2, 3000, 3000, 1.0, 0, 0, ent.data_ptr(), 0, 0, 0, st)
    Q.q4g_token_logprobs(x.data_ptr(), 2, 3000, 3000, 1.0, 0, 0, 0, 2, ids.data_ptr(), 0, st)
    p = torch.softmax(x.double(), -1)
    torch.testing.assert_close(ent[:2].double(), -(p * p.log()).sum(-1), rtol=0, atol=1e-5)
    assert torch.all(ent[2:] == 9) and torch.all(ids[2] == -9)
    assert torch.equal(ids[:2].long(), torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :2])


def test_many_rows():
    """More rows than one launch's grid holds."""
    rows = 65535 + 130
    x = torch.randn(rows, 17, device="cuda")
    t = torch.randint(0, 17, (rows,), device="cuda", dtype=torch.int32)
    lp = torch.empty(rows, device="cuda")
    ids = torch.empty((rows, 3), dtype=torch.int32, device="cuda")
    Q.q4g_token_logprobs(x.data_ptr(), rows, 17, 17, 1.0, t.data_ptr(), lp.data_ptr(), 0, 3, ids.data_ptr(), 0,
                         torch.cuda.current_stream().cuda_stream)
    want = torch.log_softmax(x.double(), -1).gather(1, t.long()[:, None])[:, 0]
    # one term per thread and a few joins: (17 / 256 + 48) 2^-24, and 2^-22 |d|, |d| < 16
    torch.testing.assert_close(lp.double(), want, rtol=0, atol=49 * 2 ** -24 + 16 * 2 ** -22)
    assert torch.equal(ids.long(), torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :3])
