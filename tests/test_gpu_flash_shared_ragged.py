"""q4g_flash_decode_shared and _i8 with hostile bytes wherever the call must not look or
write: behind each sequence's own rows, behind the output and behind the workspace."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q
from test_gpu_flash_shared import Batch, sp

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def guarded(t):
    """The batch with a pattern behind its output and its workspace; what checks them."""
    n, nb = t.out.numel(), t.ws.numel()
    out = torch.full((n + GUARD,), 321.0, dtype=torch.float16, device="cuda")
    ws = torch.full((nb + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")
    t.out, t.ws = out[:n].view(t.out.shape), ws[:nb]

    def intact():
        return bool((out[n:] == 321.0).all()) and bool((ws[nb:] == 0xa5).all())
    return intact


def spoil(t, lens):
    """NaN and infinities in every own row (int8: its scales) from the length on."""
    for x in t.kv[2:]:
        rows = x[1] if t.i8 else x
        for b, n in enumerate(lens):
            rows[b, n:] = float("nan") if b % 2 else float("-inf") if b % 4 else float("inf")


def clear(t, lens):
    for x in t.kv[2:]:
        for b, n in enumerate(lens):
            (x[1] if t.i8 else x)[b, n:] = 0


# (sequences, query heads, KV heads, head_dim, prefix, capacity): own units below the number
# of CTAs, and several for each; with a prefix in pieces, as one line, and with none
CASES = [(16, 16, 1, 512, 300, 150), (17, 16, 8, 256, 200, 270), (20, 8, 2, 256, 0, 140), (64, 16, 8, 256, 0, 300),
         (48, 16, 8, 256, 130, 40), (200, 16, 2, 512, 0, 290), (256, 8, 2, 256, 1000, 19), (40, 130, 2, 256, 500, 141)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("batch,n_q,n_kv,hd,prefix,cap", CASES)
def test_what_lies_behind_ragged_lengths_changes_nothing(batch, n_q, n_kv, hd, prefix, cap, i8):
    """Lengths of every remainder mod 16: bitwise what zeros behind them give, and right."""
    lens = [b % 16 + 16 * (b * 5 % ((cap - b % 16) // 16 + 1)) for b in range(batch)]
    assert {n % 16 for n in lens} == set(range(16)) and max(lens) <= cap
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens, i8, seed=batch)
    intact = guarded(t)
    clear(t, lens)
    want = t.run().clone()
    t.check()
    spoil(t, lens)
    for _ in range(5):
        t.out.fill_(7.0)
        assert torch.equal(t.run(), want)
    assert intact()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("batch,n_q,n_kv,hd,prefix,cap", [
    (1, 16, 1, 512, 1, 0), (3, 1, 1, 256, 700, 9), (5, 7, 7, 512, 5000, 0), (2, 1024, 1, 512, 300, 20),
    (256, 64, 1, 256, 129, 3), (9, 192, 3, 512, 0, 500), (1, 16, 1, 512, 100000, 128)])
def test_nothing_is_written_behind_output_and_workspace(batch, n_q, n_kv, hd, prefix, cap, i8):
    lens = np.random.default_rng(n_q).integers(0, cap + 1, batch).tolist()
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens if cap else [], i8, seed=batch)
    intact = guarded(t)
    t.run()
    t.check()
    assert intact()


def test_every_one_of_many_calls_at_once_is_right():
    """Three streams, a workspace each and calls of different kinds in flight: every call's
    output is compared on its stream."""
    ts = [Batch(9, 16, 1, 512, 4000, 200, [200, 1, 0, 33, 150, 128, 64, 90, 17], seed=21),
          Batch(12, 16, 8, 256, 700, 60, list(range(0, 60, 5)), True, seed=22),
          Batch(70, 64, 2, 512, 600, 90, [b % 91 for b in range(70)], True, seed=23)]
    want = [t.run().clone() for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in ts]
    for _ in range(100):
        for t, st, w, x in zip(ts, streams, wrong, want):
            with torch.cuda.stream(st):
                t.out.zero_()
                w.add_((t.run() != x).sum())
    torch.cuda.synchronize()
    assert [int(w) for w in wrong] == [0, 0, 0]
    Q.q4g_model_check(0, sp())
