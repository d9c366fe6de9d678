"""The give-up path of q4g_flash_decode_shared and _i8, without a fault: one barrier of one
CTA waits for an arrival that never comes, its wait gives up after 20 ms, the other roles
end, what is in flight is waited for, the call's kernels finish, and q4g_model_check reports
Q4G_ETIMEOUT to a caller that has no model. The next calls are right again."""
from __future__ import annotations

import time

import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q
from test_gpu_flash_shared import Batch, sp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# three units of work and more for the first CTA; a piece of a line; one of a long prefix;
# ragged own rows alone, again several units
CASES = [(130, 128, 2, 512, 1000, 5), (100, 64, 1, 256, 1500, 300), (8, 16, 1, 512, 40000, 100),
         (64, 16, 8, 256, 0, 333)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("stall,batch,n_q,n_kv,hd,prefix,cap",
                         [(s, *c) for s in (1, 2, 3, 4) for c in CASES] + [(5, *CASES[0]), (5, *CASES[3])])
def test_a_wait_that_gives_up_is_reported(stall, batch, n_q, n_kv, hd, prefix, cap, i8):
    lens = [(37 * b + 5) % (cap + 1) for b in range(batch)]
    t = Batch(batch, n_q, n_kv, hd, prefix, cap, lens, i8, seed=stall)
    nb = t.ws.numel()
    guarded = torch.full((nb + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    t.ws = guarded[:nb]
    Q.q4g_model_check(0, sp())
    want = t.run().clone()
    Q.q4g_model_check(0, sp())
    Q.q4g_model_set_option(0, Q.Q4G_OPT_TEST_STALL, stall)
    t0 = time.monotonic()
    t.run()
    with pytest.raises(Q.Q4GError) as e:
        Q.q4g_model_check(0, sp())
    assert e.value.status == Q.Q4G_ETIMEOUT and "shared-prefix" in str(e.value)
    assert time.monotonic() - t0 < 5
    assert bool((guarded[nb:] == 0xa5).all())
    Q.q4g_model_check(0, sp())  # the word was cleared
    for _ in range(3):
        t.out.zero_()
        assert torch.equal(t.run(), want)
    Q.q4g_model_check(0, sp())
