"""The probabilities of q4g_flash_decode_shared and _i8 carry more bits than the output.

A call over a batch gives what one call per sequence gives: the probabilities enter the
second product as two fp16 numbers (2^-22 relative), so nothing of fp16 is left but the
output's own rounding. Values that nearly cancel show it: with o = sum p v close to zero
against a = sum p |v|, an error of 2^-12 in one probability is far above the output's
rounding, 2^-11 |o|.

Tolerance. A query has one entry that is not zero, 1 or 1/2, so a score is one exact
product. Two keys have scores of 0.4 to 3.5, all others -60 or less: those have
probabilities below 2^-80 and count for nothing. A probability is 2^e with |e| <= 16: the
factor log2 e, a row's scale, the product and two subtractions are each off by at most half
an ulp below 16, 2^-21, or less, four such errors together; 2^-21 ln 2 is a relative error
of 2^-21.5 of the probability; exp2 adds 2^-22, hi + lo 2^-22. A partial's weight in the
join is another 2^e, with one subtraction. That is below 2^-18 for a probability, as much
again for the sum under the fraction, whose n keys add n 2^-24. The fp32 sums of values
run in steps of 16 keys, hi and lo, and up to 32 partials: (n / 8 + 32) 2^-23 a. Together
  |o - o64| <= 2^-11 |o64| + 2^-25 + (2^-17 + n 2^-24 + (n / 8 + 32) 2^-23) a."""
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


def call(q, n_kv, rows, prefix, lens, i8):
    """rows: K and V of [batch][prefix + cap][n_kv][hd], fp16 or (codes, scales); the prefix is sequence 0's."""
    batch, n_q, hd = q.shape
    flat = [t for x in rows for t in (x if i8 else (x,))]
    pre, own = [t[0, :prefix].contiguous() for t in flat], [t[:, prefix:].contiguous() for t in flat]
    out = torch.empty((batch, n_q, hd), dtype=torch.float16, device="cuda")
    nb = Q.q4g_flash_decode_shared_workspace_bytes(batch, n_q, n_kv, hd)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    fn = Q.q4g_flash_decode_shared_i8 if i8 else Q.q4g_flash_decode_shared
    fn(q.data_ptr(), batch, n_q, n_kv, hd, *[t.data_ptr() for t in pre], prefix, *[t.data_ptr() for t in own],
       own[0].shape[1], lens.data_ptr(), out.data_ptr(), ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    return out


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n_q,n_kv,hd", [(16, 1, 512), (16, 8, 256), (96, 1, 512)])
@pytest.mark.parametrize("batch,prefix,first,second", [
    (1, 2, 0, 1), (4, 2, 0, 1), (3, 1, 0, 1), (5, 700, 3, 699), (2, 1000, 130, 1003), (9, 300, 299, 301)])
def test_values_that_nearly_cancel(batch, prefix, first, second, n_q, n_kv, hd, i8):
    """Two keys that count, `first` in the prefix and `second` there or among the own rows."""
    cap, G = 4, n_q // n_kv
    n = prefix + cap
    rng = np.random.default_rng(prefix + batch)
    # head g of a KV head sees the scores of one of two key columns, whole or halved
    dims = np.stack([rng.permutation(hd)[:2] for _ in range(n_kv)])
    gap = rng.integers(1, 88, (n_kv, 2)) / 32.0  # of the two scores
    q = np.zeros((batch, n_q, hd), np.float16)
    K, V = np.zeros((n, n_kv, hd)), np.zeros((n, n_kv, hd))
    for h in range(n_kv):
        for g in range(G):
            q[:, h * G + g, dims[h, g % 2]] = 1.0 if g % 4 < 2 else 0.5
        K[:, h, dims[h]] = -127.0  # -127 and -63.5: rows of scale 1
        K[first, h, dims[h]], K[second, h, dims[h]] = 112.0, 112.0 - 32 * gap[h]  # rows of scale 1/32
        # column d of the values cancels for the heads g with g % 4 == d % 4: v2 = -v1 p1 / p2
        kind = np.arange(hd) % 4
        ratio = np.exp(np.where(kind < 2, 1.0, 0.5) * gap[h, kind % 2])
        v1 = np.maximum(np.rint(rng.integers(60, 121, hd) / ratio), 1)
        V[first, h], V[second, h] = v1, -np.minimum(np.rint(v1 * ratio), 127)
    ks, vs = np.ones((n, n_kv), np.float32), np.full((n, n_kv), 3 / 64, np.float32)
    ks[[first, second]] = 1 / 32
    every = lambda x, t: torch.from_numpy(x).to(t).cuda().expand(batch, *x.shape).contiguous()  # noqa: E731
    if i8:
        rows = [(every(x, torch.int8), every(s, torch.float32)) for x, s in ((K, ks), (V, vs))]
    else:
        rows = [every(x * s[..., None], torch.float16) for x, s in ((K, ks), (V, vs))]
    qd = torch.from_numpy(q).cuda()
    lens = torch.full((batch,), cap, dtype=torch.int32, device="cuda")
    out = call(qd, n_kv, rows, prefix, lens, i8).double()
    near = 0
    for h in range(n_kv):
        k, v = (torch.from_numpy(x[:, h] * s[:, h, None].astype(np.float64)).cuda() for x, s in ((K, ks), (V, vs)))
        for b in range(batch):
            o = out[b, h * G:(h + 1) * G]
            p = torch.softmax(qd[b, h * G:(h + 1) * G].double() @ k.t(), -1)
            ref, a = p @ v, p @ v.abs()
            tol = 2.0 ** -11 * ref.abs() + 2.0 ** -25 + (2.0 ** -17 + n * 2.0 ** -24 + (n / 8 + 32) * 2.0 ** -23) * a
            near += int((ref.abs() < a / 64).sum())
            bad = (o - ref).abs() > tol
            assert not bool(bad.any()), (b, h, int(bad.sum()), float(((o - ref).abs() / tol).max()))
    assert near > batch * n_q * hd // 16  # the case does hold values that nearly cancel
