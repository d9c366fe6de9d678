"""The operators for several continuations of one prompt used together, and the scoring
path of a decoder."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import datagen as DG
from datagen import synth as S
from datagen import workloads as WL
from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def sp():
    return torch.cuda.current_stream().cuda_stream


def test_continuations_of_one_prompt_step_by_step():
    """A prompt's K/V rows go into an int8 cache; four continuations then append a row
    per step, attend prompt and own rows, and get the log probabilities of their next
    tokens from a q4_0 head, all on one side stream. In 64 bits from the same inputs, the
    rows quantised by the format's own formula."""
    n_q, hd, P, cap, batch, V, steps = 16, 512, 777, 8, 4, 5000, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda s, w: (torch.randn(s, generator=g, device="cuda") * w).half()  # noqa: E731
    kp, vp = rnd((P, 1, hd), hd ** -0.25), rnd((P, 1, hd), 1.0)
    ks, vs = rnd((steps, batch, 1, hd), hd ** -0.25), rnd((steps, batch, 1, hd), 1.0)
    qs = rnd((steps, batch, n_q, hd), 2 * hd ** -0.25)
    w = torch.randn((V, n_q * hd), generator=g, device="cuda") * 0.02
    codes = torch.empty((V, n_q * hd // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((V, n_q * hd // 32), dtype=torch.float16, device="cuda")
    Q.q4g_q4_0_pack(w.data_ptr(), V, n_q * hd, codes.data_ptr(), scales.data_ptr(), 1, sp())
    Q.q4g_q4_0_unpack(codes.data_ptr(), scales.data_ptr(), V, n_q * hd, w.data_ptr(), 1, sp())
    new = lambda *s: [torch.zeros(s + (hd,), dtype=torch.int8, device="cuda"), torch.zeros(s, device="cuda")]  # noqa: E731
    pre, own = [*new(P, 1), *new(P, 1)], [*new(batch, cap, 1), *new(batch, cap, 1)]
    nb = Q.q4g_flash_decode_shared_workspace_bytes(batch, n_q, 1, hd)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.empty((steps, batch, n_q, hd), dtype=torch.float16, device="cuda")
    logits = torch.empty((steps, batch, V), device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    targets = torch.randint(0, V, (steps, batch), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = torch.empty((steps, batch), device="cuda"), torch.empty((steps, batch), device="cuda")
    ids = torch.empty((steps, batch, 5), dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    p = lambda ts: [t.data_ptr() for t in ts]  # noqa: E731
    with torch.cuda.stream(st):
        Q.q4g_kv_write_linear_i8(kp.data_ptr(), vp.data_ptr(), P, hd, 1, hd, 0, 0, P, *p(pre), sp())
        for t in range(steps):
            slots = torch.arange(batch, device="cuda") * cap + t
            Q.q4g_kv_write_linear_i8(ks[t].data_ptr(), vs[t].data_ptr(), batch, hd, 1, hd, slots.data_ptr(), 0,
                                     batch * cap, *p(own), sp())
            lens.fill_(t + 1)
            Q.q4g_flash_decode_shared_i8(qs[t].data_ptr(), batch, n_q, 1, hd, *p(pre), P, *p(own), cap,
                                         lens.data_ptr(), out[t].data_ptr(), ws.data_ptr(), nb, sp())
            Q.q4g_gemv(codes.data_ptr(), scales.data_ptr(), V, n_q * hd, out[t].data_ptr(), batch,
                       logits[t].data_ptr(), sp())
            Q.q4g_token_logprobs(logits[t].data_ptr(), batch, V, V, 1.0, targets[t].data_ptr(), lp[t].data_ptr(),
                                 ent[t].data_ptr(), 5, ids[t].data_ptr(), 0, sp())
    st.synchronize()

    def deq(x):  # the int8 row format
        x = x.cpu().numpy().astype(np.float32)
        s = (np.abs(x).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
        return torch.from_numpy(np.rint(x / s).astype(np.float64) * s.astype(np.float64)).cuda()

    K0, V0, K1, V1 = deq(kp)[:, 0], deq(vp)[:, 0], deq(ks)[:, :, 0], deq(vs)[:, :, 0]
    for t in range(steps):
        for b in range(batch):
            k, v = torch.cat([K0, K1[:t + 1, b]]), torch.cat([V0, V1[:t + 1, b]])
            pr = torch.softmax(qs[t, b].double() @ k.t(), -1)
            ref = pr @ v
            # fp16 probabilities and output: 2^-11 of sum p|v| and of |o|, as much again for fp32 scores
            tol = 2.0 ** -11 * (ref.abs() + 2 * (pr @ v.abs()))
            assert bool(((out[t, b].double() - ref).abs() <= tol).all()), (t, b)
            z = w.double() @ out[t, b].reshape(-1).double()
            err = float((logits[t, b].double() - z).abs().max())
            want = torch.log_softmax(z, -1)
            # log softmax moves by at most twice what a logit moves; its own fp32 error is below 1e-5 here
            assert abs(float(lp[t, b]) - float(want[targets[t, b].long()])) <= 2 * err + 1e-5
            assert abs(float(ent[t, b]) + float((want.exp() * want).sum())) <= 25 * err + 1e-4
            assert torch.equal(ids[t, b].long(), torch.sort(logits[t, b], descending=True, stable=True).indices[:5])


@pytest.mark.parametrize("kv_int8", [0, 1])
@pytest.mark.parametrize("S_", [1, 7, 64])
def test_score_chunk_is_the_logprobs_of_the_decoders_rows(S_, kv_int8):
    """Each row's outputs are q4g_token_logprobs of the verify rows' logits, bitwise, and
    the cache afterwards continues as after a prefill."""
    cfg = dict(WL.TINY, kv_int8=kv_int8)
    V = cfg["vocab"]
    gm = S.SynthDecoder(cfg, seed=2, variant=1)
    a, b = gm.new_cache(256), gm.new_cache(256)
    ids = torch.from_numpy(DG.uniform_int(2, DG.STREAM_PREFIX_IDS, 90, V).astype(np.int32)).cuda()
    for c in (a, b):
        Q.q4g_prefill_chunk(gm.handle, c.handle, ids.data_ptr(), 20, 0, 0, 0, sp())
    part, nxt = ids[20:20 + S_], ids[21:21 + S_].contiguous()
    lp, ent = torch.full((S_ + 1,), 9.0, device="cuda"), torch.full((S_ + 1,), 9.0, device="cuda")
    tid = torch.full((S_ + 1, 4), -9, dtype=torch.int32, device="cuda")
    tlp = torch.full((S_ + 1, 4), 9.0, device="cuda")
    am = torch.full((S_ + 1,), -9, dtype=torch.int32, device="cuda")
    Q.q4g_score_chunk(gm.handle, a.handle, part.data_ptr(), nxt.data_ptr(), S_, 20, 0.8, lp.data_ptr(), ent.data_ptr(),
                      4, tid.data_ptr(), tlp.data_ptr(), am.data_ptr(), sp())
    logits = torch.empty((S_, V), device="cuda")
    best = torch.empty(S_, dtype=torch.int32, device="cuda")
    for i in range(0, S_, 4):
        n = min(4, S_ - i)
        Q.q4g_verify_block(gm.handle, b.handle, part[i:].data_ptr(), n, 20 + i, n, logits[i:].data_ptr(),
                           best[i:].data_ptr(), sp())
    want = [torch.empty_like(x[:S_]) for x in (lp, ent, tid, tlp)]
    Q.q4g_token_logprobs(logits.data_ptr(), S_, V, V, 0.8, nxt.data_ptr(), want[0].data_ptr(), want[1].data_ptr(), 4,
                         want[2].data_ptr(), want[3].data_ptr(), sp())
    torch.cuda.synchronize()
    ref = torch.log_softmax(logits.double() / np.float64(np.float32(0.8)), -1)
    # V / 256 + 48 roundings of a sum, four of |d| <= 80
    assert float((lp[:S_].double() - ref.gather(1, nxt.long()[:, None])[:, 0]).abs().max()) <= 64 * 2 ** -24 + 80 * 2 ** -22
    assert torch.equal(am[:S_], best) and torch.equal(tid[:S_, 0], best)
    assert torch.equal(tid[:S_], want[2])
    for got, w in ((lp, want[0]), (ent, want[1]), (tlp, want[3])):
        # rows split over another number of CTAs add up in another order
        assert float((got[:S_] - w).abs().max()) <= 2 * (64 * 2 ** -24 + 80 * 2 ** -22)
        assert torch.all(got[S_] == 9)
    assert int(am[S_]) == -9
    outs = []
    for c in (a, b):
        lg = torch.empty(V, device="cuda")
        Q.q4g_decode_step(gm.handle, c.handle, 5, 20 + S_, lg.data_ptr(), 0, sp())
        outs.append(lg)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    Q.q4g_model_check(gm.handle, sp())


def test_score_chunk_refuses():
    gm = S.SynthDecoder(WL.TINY, seed=2, variant=1)
    c = gm.new_cache(64)
    x = torch.zeros(64, dtype=torch.int32, device="cuda")
    f = torch.zeros(64, device="cuda")

    def call(S_=4, pos0=0, T=1.0, targets=x.data_ptr(), lp=f.data_ptr(), n=0, ids=x.data_ptr()):
        Q.q4g_score_chunk(gm.handle, c.handle, ids, targets, S_, pos0, T, lp, 0, n, 0, 0, 0, sp())

    for status, kw in ((Q.Q4G_ERANGE, dict(S_=0)), (Q.Q4G_ERANGE, dict(S_=65)), (Q.Q4G_ERANGE, dict(pos0=61)),
                       (Q.Q4G_ERANGE, dict(pos0=-1)), (Q.Q4G_EINVAL, dict(T=0.0)), (Q.Q4G_EINVAL, dict(targets=0)),
                       (Q.Q4G_EINVAL, dict(targets=0, lp=0)), (Q.Q4G_EINVAL, dict(n=3)), (Q.Q4G_EINVAL, dict(ids=0)),
                       (Q.Q4G_ERANGE, dict(pos0=2 ** 63 - 1))):
        with pytest.raises(Q.Q4GError) as e:
            call(**kw)
        assert e.value.status == status, kw
    call()
    Q.q4g_model_check(gm.handle, sp())
