"""The timeout path of mla_cache_weights on the GPU, made to happen without a
fault (see test_gpu_timeout.py): the issuing warp of every CTA waits on a
barrier that nothing completes.  The wait gives up after a short limit; the
kernel records MLA_ERR_TIMEOUT, lets its copies and products land, frees its
tensor memory and returns, so that the same call on a fresh workspace gives
the right weights."""
import numpy as np
import pytest

import mla_latent_kv_10_gb300 as mla
from oracle import cache as oc
from test_gpu_cache import case_and_query, gather, lse_of

pytestmark = pytest.mark.gpu
MLA_ERR_TIMEOUT = -7


@pytest.fixture(scope="module", autouse=True)
def built():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    mla.load_library()
    yield
    mla.mla_set_timeout_test(0, -1)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("B,Lq,H,G,n,stall_page", [
    (2, 1, 16, 1, 700, 0),      # one tile, one pass
    (2, 2, 128, 1, 700, 0),     # two blocks of rows
    (2, 2, 128, 1, 700, 2),     # before the second
    (2, 4, 64, 4, 300, 6),      # four groups, before the last
    (12, 1, 16, 1, 8100, 0),    # several tiles a CTA: rings and accumulators in use
    (12, 1, 16, 1, 8100, 4),
])
def test_wait_that_gives_up_sets_timeout_and_context_stays_usable(kv, B, Lq, H, G, n, stall_page):
    c, q = case_and_query(kv, B, Lq, H, G, [n - 37 * b for b in range(B)])
    lse = lse_of(kv, c, q)
    want, st = gather(kv, c, q, lse)
    assert st == 0
    mla.mla_set_timeout_test(50_000, stall_page)  # 50 us
    try:
        _, st = gather(kv, c, q, lse)
    finally:
        mla.mla_set_timeout_test(0, -1)
    assert st == MLA_ERR_TIMEOUT
    got, st = gather(kv, c, q, lse)
    assert st == 0 and np.array_equal(got.numpy(), want.numpy())
    if B == 2:
        ref = oc.gathered_weights(c.dims, kv, q, c.cache, c.block_table, c.seq_lens, lse.double().numpy())
        assert np.all(np.abs(got.double().numpy() - ref) <= 2.0 ** -14 * ref)
