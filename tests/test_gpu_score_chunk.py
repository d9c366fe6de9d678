"""q4g_score_chunk against one decode step per token of the same decoder: through ring wraps
and the window's slide, with a ring that leaves room for one or three rows a pass, an fp16
head, int8 rows, and a row's outputs left out.

Tolerance. Both sides are within 2e-2 of the logits' RMS of the exact logits (the decode
tolerance; multi-row products round in another order), so they differ by e = 4e-2 RMS at
most, a log probability at temperature T by 2 e / T, and the entropy, whose gradient with
respect to the logits sums to at most 2 ln V in magnitude, by 2 e ln V / T. Ids are held
to be alternatives that lie within 2 e of the list's own logit."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import datagen as DG
from datagen import synth as S
from datagen import workloads as WL
from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

pytestmark = pytest.mark.gpu

SMALL = dict(n_layers=6, hidden=256, n_q_heads=2, ffn=512, vocab=512, sl_kv_heads=1)
CONFIGS = {
    "wraps": WL.decoder(**SMALL, window=32, ring=64),
    "one_row_a_pass": WL.decoder(**SMALL, window=32, ring=33),
    "three_rows_a_pass": WL.decoder(**SMALL, window=13, ring=16),
    "int8_rows": dict(WL.decoder(**SMALL, window=32, ring=64), kv_int8=1),
    "fp16_head": WL.TINY_F16,
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("T", [1.0, 0.6])
@pytest.mark.parametrize("name", CONFIGS)
def test_scores_of_a_text_in_chunks(name, T):
    cfg = CONFIGS[name]
    V, n, sp = cfg["vocab"], 150, S.stream_ptr()
    g = S.SynthDecoder(cfg, seed=3, variant=1)
    a, b = g.new_cache(n), g.new_cache(n)
    ids = torch.from_numpy(DG.uniform_int(3, DG.STREAM_PREFIX_IDS, n + 1, V).astype(np.int32)).cuda()
    lp, ent = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    tid = torch.full((n, 3), -9, dtype=torch.int32, device="cuda")
    am = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    pos = 0
    for s in (1, 64, 3, 5, 64, 13):  # pieces of a text, ends inside a pass
        Q.q4g_score_chunk(g.handle, a.handle, ids[pos:].data_ptr(), ids[pos + 1:].data_ptr(), s, pos, T,
                          lp[pos:].data_ptr(), ent[pos:].data_ptr() if s != 5 else 0, 3, tid[pos:].data_ptr(), 0,
                          am[pos:].data_ptr() if s != 3 else 0, sp)
        pos += s
    assert pos == n
    logits = torch.empty((n, V), device="cuda")
    for t in range(n):
        Q.q4g_decode_step(g.handle, b.handle, int(ids[t]), t, logits[t].data_ptr(), 0, sp)
    torch.cuda.synchronize()
    Q.q4g_model_check(g.handle, sp)
    x = logits.double()
    e = 4e-2 * x.square().mean(-1).sqrt()
    d = torch.log_softmax(x / float(np.float32(T)), -1)
    want = d.gather(1, ids[1:].long()[:, None])[:, 0]
    assert bool(((lp.double() - want).abs() <= 2 * e / T + 1e-4).all())
    H = -(d.exp() * d).sum(-1)
    live = ent != 9.0
    assert int(live.sum()) == n - 5 and bool((ent[68:73] == 9.0).all())
    assert bool(((ent.double() - H).abs() <= 2 * e * math.log(V) / T + 1e-4)[live].all())
    top = torch.sort(x, dim=-1, descending=True).values[:, :3]
    assert bool(((x.gather(1, tid.long()) - top).abs() <= 2 * e[:, None]).all())
    kept = am != -9
    assert int(kept.sum()) == n - 3 and torch.equal(am[kept], tid[kept, 0])


def test_the_12b_class_head_scores_its_own_logits():
    """Six layers and the 262,144-token head of the 12B-class decoder: the scores are the log
    probabilities of the logits that verify rows give, in 64 bits."""
    cfg = dict(WL.B12, n_layers=6)
    V, sp, s = cfg["vocab"], S.stream_ptr(), 6
    g = S.SynthDecoder(cfg, seed=0)
    a, b = g.new_cache(64), g.new_cache(64)
    ids = torch.from_numpy(DG.uniform_int(1, DG.STREAM_PREFIX_IDS, s + 1, V).astype(np.int32)).cuda()
    lp, ent = torch.empty(s, device="cuda"), torch.empty(s, device="cuda")
    tid, tlp = torch.empty((s, 20), dtype=torch.int32, device="cuda"), torch.empty((s, 20), device="cuda")
    Q.q4g_score_chunk(g.handle, a.handle, ids.data_ptr(), ids[1:].data_ptr(), s, 0, 1.0, lp.data_ptr(),
                      ent.data_ptr(), 20, tid.data_ptr(), tlp.data_ptr(), 0, sp)
    logits = torch.empty((s, V), device="cuda")
    for i in (0, 4):
        n = min(4, s - i)
        Q.q4g_verify_block(g.handle, b.handle, ids[i:].data_ptr(), n, i, n, logits[i:].data_ptr(), 0, sp)
    torch.cuda.synchronize()
    Q.q4g_model_check(g.handle, sp)
    d = torch.log_softmax(logits.double(), -1)
    # a thread sums V / 256 terms at most, lists of 16 join (2^-24 each), |d| <= 60 (softcap 30)
    tol = (V / 256 + 48) * 2.0 ** -24 + 60 * 2.0 ** -22
    assert float((lp.double() - d.gather(1, ids[1:].long()[:, None])[:, 0]).abs().max()) <= tol
    assert float((ent.double() + (d.exp() * d).sum(-1)).abs().max()) <= tol * (2 + 2 * math.log(V))
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(tid.long(), order)
    assert float((tlp.double() - d.gather(1, order)).abs().max()) <= tol
