"""GPU tests of the arithmetic of mla_cache_weights at the ends of what it
accepts."""
import numpy as np
import pytest
import torch

import mla_latent_kv_10_gb300 as mla
from oracle import cache as oc
from test_gpu_cache import case_and_query, gather, lse_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    mla.load_library()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("scale", [1e-30, 1e-37, 1.2e-38, 1e-40, 1.5e-45])
def test_hidden_keys_weigh_nothing_at_tiny_scales(kv, scale):
    """Every score is next to zero: a key that a row sees weighs exp(-lse),
    one that it does not see nothing.  Tolerance: that of the other tests of
    the weights against 64 bits."""
    c, q = case_and_query(kv, 2, 3, 16, 1, [3, 190])
    c.dims["scale"] = float(torch.tensor(scale, dtype=torch.float32))
    lse = lse_of(kv, c, q)
    want = oc.gathered_weights(c.dims, kv, q, c.cache, c.block_table, c.seq_lens, lse.double().numpy())
    got, st = gather(kv, c, q, lse)
    assert st == 0
    assert np.all(np.abs(got.double().numpy() - want) <= 2.0 ** -14 * want)
