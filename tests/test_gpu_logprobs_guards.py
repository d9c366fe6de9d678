"""q4g_token_logprobs: what lies behind its outputs and between its rows, calls in flight
on several streams, captured and replayed calls."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

pytestmark = pytest.mark.gpu

GUARD = 512


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Call:
    """Outputs with a pattern behind them; NaN behind the logits and between their rows."""

    def __init__(self, rows, vocab, n, T=1.0, pad=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.shape, self.n, self.T = g, (rows, vocab), n, T
        self.buf = torch.full((rows, vocab + pad), float("nan"), device="cuda")
        self.t = torch.empty(rows, dtype=torch.int32, device="cuda")
        # (buffer, values that belong to the call)
        f = lambda k: (torch.full((k + GUARD,), 9.0, device="cuda"), k)  # noqa: E731
        self.outs = [f(rows), f(rows),
                     (torch.full((rows * n + GUARD,), -9, dtype=torch.int32, device="cuda"), rows * n), f(rows * n)]
        self.new_inputs()

    def new_inputs(self):
        rows, vocab = self.shape
        self.buf[:, :vocab] = torch.randn((rows, vocab), generator=self.g, device="cuda") * 4
        self.t.copy_(torch.randint(0, vocab, (rows,), generator=self.g, device="cuda"))

    def run(self):
        lp, ent, ids, tops = [o[0].data_ptr() for o in self.outs]
        Q.q4g_token_logprobs(self.buf.data_ptr(), *self.shape, self.buf.shape[1], self.T, self.t.data_ptr(), lp, ent,
                             self.n, ids if self.n else 0, tops if self.n else 0,
                             torch.cuda.current_stream().cuda_stream)

    def clear(self):
        for o, k in self.outs:
            o[:k] = 77

    def values(self):
        return [o[:k].clone() for o, k in self.outs]

    def intact(self):
        return all(bool((o[k:] == (-9 if o.dtype == torch.int32 else 9)).all()) for o, k in self.outs)

    def check(self):
        """Ids equal; log probabilities: one thread adds up vocab / 256 + 32 terms at most,
        lists of 16 join, 2^-24 each, and 2^-22 |d|."""
        rows, vocab = self.shape
        x = self.buf[:, :vocab]
        d = (x.double() - x.double().amax(-1, keepdim=True)) / float(np.float32(self.T))
        want = d - torch.log(torch.exp(d).sum(-1, keepdim=True))
        lp, _, ids, tops = self.values()
        tol = (vocab / 256 + 48) * 2.0 ** -24 + 2.0 ** -22 * float(d.abs().max())
        assert float((lp.double() - want.gather(1, self.t.long()[:, None])[:, 0]).abs().max()) <= tol
        if self.n:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :self.n]
            assert torch.equal(ids.view(rows, self.n).long(), order)
            assert float((tops.view(rows, self.n).double() - want.gather(1, order)).abs().max()) <= tol


SHAPES = [(1, 1, 1, 0), (1, 262144, 8, 0), (3, 262144, 32, 5), (18, 30000, 3, 0), (19, 30000, 3, 1), (5, 4097, 0, 3),
          (297, 5003, 20, 0), (600, 1000, 1, 7), (1200, 33, 32, 0)]


@pytest.mark.parametrize("rows,vocab,n,pad", SHAPES)
def test_nothing_is_written_behind_the_outputs(rows, vocab, n, pad):
    c = Call(rows, vocab, n, 0.9, pad, seed=rows)
    for _ in range(3):
        c.clear()
        c.run()
        c.check()
        assert c.intact()
        c.new_inputs()


def test_more_rows_than_a_launch_holds_leave_the_rest_alone():
    c = Call(65535 + 7, 40, 2, seed=3)
    c.run()
    c.check()
    assert c.intact()


def test_captured_and_replayed_with_other_logits():
    calls = [Call(2, 262144, 8, seed=4), Call(300, 5003, 5, 0.7, 3, seed=5), Call(40, 70001, 0, seed=6)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for c in calls:
            c.run()
    for _ in range(3):
        for c in calls:
            c.new_inputs()
            c.clear()
        g.replay()
        torch.cuda.synchronize()
        for c in calls:
            c.check()
            assert c.intact()


def test_every_one_of_many_calls_at_once_is_right():
    calls = [Call(1, 262144, 32, seed=7), Call(16, 200003, 20, seed=8), Call(256, 65537, 4, 1.3, 1, seed=9)]
    want = []
    for c in calls:
        c.run()
        want.append(c.values())
        c.check()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in calls]
    for _ in range(50):
        for c, st, w, x in zip(calls, streams, wrong, want):
            with torch.cuda.stream(st):
                c.clear()
                c.run()
                for a, b in zip(c.values(), x):
                    w.add_((a != b).sum())
    torch.cuda.synchronize()
    assert [int(w) for w in wrong] == [0, 0, 0]
