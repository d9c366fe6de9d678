"""Head counts whose fp16 row passes 2^31 elements, written to int8 rows and read back."""
from __future__ import annotations

import pytest
import torch

from int4_q4_gemv_b200 import build as B
from int4_q4_gemv_b200 import q4g as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("n_kv,hd", [((1 << 22) + 3, 512), ((1 << 23) + 5, 256)])
def test_heads_beyond_32_bits(n_kv, hd, ring):
    """One row of n_kv heads, 2^31 + 3 hd elements or more, all zero but for a few heads on
    both sides of 2^31; K and V are the same rows. A live head holds 127 at one place and
    whole numbers elsewhere: scale 1, so codes and read-back values equal the input."""
    st = torch.cuda.current_stream().cuda_stream
    x = torch.zeros((n_kv, hd), dtype=torch.float16, device="cuda")
    live = torch.tensor([0, 1, 2 ** 31 // hd - 1, 2 ** 31 // hd, n_kv - 1], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(hd)
    rows = torch.randint(-126, 127, (len(live), hd), generator=g, device="cuda").half()
    rows[:, 7] = 127
    x[live] = rows
    codes = torch.full((n_kv, hd), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((n_kv,), 5.5, dtype=torch.float32, device="cuda")
    cache = [codes.data_ptr(), scales.data_ptr()] * 2
    if ring:
        Q.q4g_kv_write_ring_i8(x.data_ptr(), x.data_ptr(), 1, n_kv * hd, n_kv, hd, 5, 1, *cache, st)
    else:
        Q.q4g_kv_write_linear_i8(x.data_ptr(), x.data_ptr(), 1, n_kv * hd, n_kv, hd, 0, 0, 1, *cache, st)
    assert torch.equal(codes[live], rows.to(torch.int8))
    assert int(codes.count_nonzero()) == int(rows.count_nonzero())
    assert torch.equal(scales.nonzero()[:, 0], live) and bool((scales[live] == 1).all())
    x.fill_(3.0)
    if ring:
        Q.q4g_kv_read_ring_i8(*cache, n_kv, hd, 5, 1, 1, x.data_ptr(), x.data_ptr(), n_kv * hd, st)
    else:
        Q.q4g_kv_read_linear_i8(*cache, n_kv, hd, 0, 0, 1, 1, x.data_ptr(), x.data_ptr(), n_kv * hd, st)
    assert torch.equal(x[live], rows)
    assert int(x.count_nonzero()) == int(rows.count_nonzero())
