"""Calls that q4g_kv_write/read_*_i8, q4g_flash_decode_shared(_i8), q4g_token_logprobs
and q4g_score_chunk refuse before any launch: sizes, ranges, alignment, missing and
foreign pointers. Host checks only; the addresses below are never read."""
from __future__ import annotations

import math

import pytest

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

P = 1 << 20  # an aligned address that no device owns
EINVAL, ERANGE = Q.Q4G_EINVAL, Q.Q4G_ERANGE


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def refused(status, fn, defaults, **kw):
    with pytest.raises(Q.Q4GError) as e:
        fn(*dict(defaults, **kw).values())
    assert e.value.status == status, str(e.value)


CACHE = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P)
WL = dict(k=P, v=P, n_rows=4, row_stride=512, n_kv=1, head_dim=512, slots=0, slot0=0, capacity=8, **CACHE, stream=None)
WR = dict(k=P, v=P, n_rows=4, row_stride=2048, n_kv=8, head_dim=256, pos0=0, ring=8, **CACHE, stream=None)
RL = dict(**CACHE, n_kv=1, head_dim=512, slots=0, slot0=0, capacity=8, n_rows=4, k=P, v=P, row_stride=512, stream=None)
RR = dict(**CACHE, n_kv=8, head_dim=256, pos0=0, ring=8, n_rows=4, k=P, v=P, row_stride=2048, stream=None)
KV = {"write_linear": (Q.q4g_kv_write_linear_i8, WL), "write_ring": (Q.q4g_kv_write_ring_i8, WR),
      "read_linear": (Q.q4g_kv_read_linear_i8, RL), "read_ring": (Q.q4g_kv_read_ring_i8, RR)}


@pytest.mark.parametrize("which", KV)
@pytest.mark.parametrize("status,kw", [
    (EINVAL, dict(head_dim=128)), (EINVAL, dict(n_kv=0)), (ERANGE, dict(n_rows=-1)), (ERANGE, dict(n_rows=1 << 40)),
    (EINVAL, dict(row_stride=248)), (EINVAL, dict(row_stride=8196)), (EINVAL, dict(k=0)), (EINVAL, dict(v=P + 8)),
    (EINVAL, dict(k_codes=P + 4)), (EINVAL, dict(v_scales=P + 2)), (EINVAL, dict(k_scales=0)),
    (EINVAL, dict())])  # the last: valid sizes, memory that is not the current device's
def test_kv_calls_refuse(which, status, kw):
    refused(status, *KV[which], **kw)


@pytest.mark.parametrize("which", ["write_linear", "read_linear"])
@pytest.mark.parametrize("status,kw", [
    (ERANGE, dict(slot0=5)), (ERANGE, dict(slot0=-1)), (ERANGE, dict(slot0=1 << 62)), (ERANGE, dict(capacity=0)),
    (ERANGE, dict(capacity=(1 << 30) + 1)), (EINVAL, dict(slots=P, slot0=1)), (EINVAL, dict(slots=P + 4))])
def test_linear_slots_refused(which, status, kw):
    refused(status, *KV[which], **kw)


def test_ring_positions_refused():
    for which in ("write_ring", "read_ring"):
        refused(ERANGE, *KV[which], pos0=-1)
        refused(ERANGE, *KV[which], pos0=2 ** 63 - 2)
        refused(ERANGE, *KV[which], ring=0)
    refused(ERANGE, *KV["read_ring"], n_rows=9)


def test_kv_calls_of_no_rows_do_nothing():
    for fn, a in KV.values():
        fn(*dict(a, n_rows=0, k=0, v=0, k_codes=0, v_codes=0, k_scales=0, v_scales=0).values())


DIMS = dict(q=P, batch=4, n_q=16, n_kv=1, head_dim=512)
SH = dict(**DIMS, k_prefix=P, v_prefix=P, prefix_len=100, k_own=P, v_own=P, own_capacity=16, own_len=P, out=P, ws=P,
          ws_bytes=1 << 40, stream=None)
SH8 = dict(**DIMS, kp=P, kps=P, vp=P, vps=P, prefix_len=100, ko=P, kos=P, vo=P, vos=P, own_capacity=16, own_len=P,
           out=P, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("status,kw", [
    (EINVAL, dict(head_dim=64)), (EINVAL, dict(n_q=15, n_kv=2)), (EINVAL, dict(n_q=0)), (EINVAL, dict(n_kv=-1)),
    (EINVAL, dict(n_q=1040)), (ERANGE, dict(batch=0)), (ERANGE, dict(batch=257)), (ERANGE, dict(prefix_len=-1)),
    (ERANGE, dict(prefix_len=(1 << 30) + 1)), (ERANGE, dict(own_capacity=-1)), (ERANGE, dict(own_capacity=1 << 25)),
    (ERANGE, dict(batch=256, own_capacity=1 << 23)), (EINVAL, dict(q=0)), (EINVAL, dict(out=P + 8)),
    (EINVAL, dict(ws=P + 16)), (EINVAL, dict(ws=0)), (EINVAL, dict(own_len=0)), (EINVAL, dict(own_len=P + 2)),
    (EINVAL, dict(ws_bytes=255)), (EINVAL, dict())])
def test_shared_refuses(status, kw):
    refused(status, Q.q4g_flash_decode_shared, SH, **kw)
    refused(status, Q.q4g_flash_decode_shared_i8, SH8, **kw)


def test_shared_rows_refused():
    for kw in (dict(k_prefix=0), dict(v_prefix=P + 8), dict(k_own=0), dict(v_own=P + 4)):
        refused(EINVAL, Q.q4g_flash_decode_shared, SH, **kw)
    for kw in (dict(kp=0), dict(kps=0), dict(vps=P + 2), dict(kos=0), dict(vo=P + 4), dict(vos=P + 1)):
        refused(EINVAL, Q.q4g_flash_decode_shared_i8, SH8, **kw)


LP = dict(logits=P, rows=4, vocab=1000, row_stride=1000, temperature=1.0, targets=P, logprob=P, entropy=P, n_top=5,
          top_ids=P, top_logprobs=P, stream=None)


@pytest.mark.parametrize("status,kw", [
    (ERANGE, dict(rows=-1)), (ERANGE, dict(rows=(1 << 20) + 1)), (ERANGE, dict(vocab=0)),
    (ERANGE, dict(vocab=(1 << 30) + 1, row_stride=1 << 31)), (EINVAL, dict(row_stride=999)),
    (EINVAL, dict(temperature=0.0)), (EINVAL, dict(temperature=-1.0)), (EINVAL, dict(temperature=math.inf)),
    (EINVAL, dict(temperature=math.nan)), (EINVAL, dict(temperature=1e-40)), (ERANGE, dict(n_top=-1)),
    (ERANGE, dict(n_top=33)), (ERANGE, dict(vocab=4, row_stride=4)), (EINVAL, dict(targets=0)),
    (EINVAL, dict(logprob=0)), (EINVAL, dict(top_ids=0, top_logprobs=0)),
    (EINVAL, dict(targets=0, logprob=0, entropy=0, n_top=0)), (EINVAL, dict(logits=0)), (EINVAL, dict(logits=P + 2)),
    (EINVAL, dict(entropy=P + 1)), (EINVAL, dict())])
def test_logprobs_refuses(status, kw):
    refused(status, Q.q4g_token_logprobs, LP, **kw)


def test_logprobs_of_no_rows_does_nothing():
    Q.q4g_token_logprobs(*dict(LP, rows=0, logits=0).values())


def test_score_chunk_without_handles_refused():
    refused(EINVAL, Q.q4g_score_chunk, dict(m=0, c=0, ids=P, targets=P, S=4, pos0=0, temperature=1.0, logprob=P,
                                            entropy=0, n_top=0, top_ids=0, top_lp=0, argmax=0, stream=None))


def test_binding_limit_matches_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "q4g.h")).read()
    assert int(re.search(r"#define Q4G_LOGPROBS_MAX_TOP (\d+)", text).group(1)) == Q.Q4G_LOGPROBS_MAX_TOP


def test_stalls_without_a_model_refused():
    for opt, value in ((Q.Q4G_OPT_TEST_STALL, -1), (Q.Q4G_OPT_TEST_STALL, 6), (Q.Q4G_OPT_PDL, 1)):
        with pytest.raises(Q.Q4GError) as e:
            Q.q4g_model_set_option(0, opt, value)
        assert e.value.status == EINVAL
    Q.q4g_model_set_option(0, Q.Q4G_OPT_TEST_STALL, 0)  # none
