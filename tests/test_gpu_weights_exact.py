"""GPU tests of the arithmetic of mla_cache_weights: scales at the ends of what
it accepts, and the exponent's exactness."""
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


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("scale", [192.0 ** -0.5, 0.0625, 0.05])
@pytest.mark.parametrize("mag", [300.0, 3000.0])
def test_the_exponent_is_exact_at_large_scores(kv, scale, mag):
    """Queries with one column other than zero, in the RoPE part: a score is
    one product of bf16 numbers, exact in fp32, whatever the tensor core does
    with sums.  What is left, relative to a weight 2^z with |z| < 8 (z = score
    * log2 e - lse * log2 e, formed from parts that are exact to 2^-48):
      two roundings at the size of z, 2^-22 each, times ln 2;
      exp2 of z and of what the lse's rounding left off, 2^-22 each;
      seven additions (four of a thread's sums of 16 heads, two to join them,
      one to the weight), 2^-24 each:
    1.3e-6, below 2^-19.  A term with 8 <= |z| < 16 weighs at most 2^-8 and
    its roundings are twice as large (1.6e-6 in all, still below); 16 heads
    with |z| >= 16 weigh at most 2^-12 together, of which 2^-18 is less than
    2^-30.  Dropping a correction, or adding it where it is rounded away,
    costs half a unit of an exponent of some hundreds: 2^-17 and more."""
    c, q = case_and_query(kv, 2, 1, 16, 1, [300, 129])
    d = c.dims
    d["scale"] = float(torch.tensor(scale, dtype=torch.float32))
    g = torch.Generator().manual_seed(77)
    # keys just below two, a few bf16 steps apart
    col = (2.0 - 2.0 ** -7 * torch.randint(0, 6, c.cache.shape[:2], generator=g)).to(torch.bfloat16)
    raw = c.cache.view(torch.uint8).view(*c.cache.shape[:2], -1).clone()
    at = {"bf16": 1024, "fp8": 512, "fp4": 288}[kv] + 2 * 5
    raw[:, :, at:at + 2] = col.view(torch.uint8).view(*col.shape, 2)
    c.cache = raw.view(c.cache.dtype).view(c.cache.shape)
    q = torch.zeros_like(q)
    q[..., 512 + 5] = (mag * (1.0 + 0.03 * torch.arange(16))).to(torch.bfloat16)
    lse = lse_of(kv, c, q)
    want = oc.gathered_weights(d, kv, q, c.cache, c.block_table, c.seq_lens, lse.double().numpy())
    got, st = gather(kv, c, q, lse)
    assert st == 0
    err = np.abs(got.double().numpy() - want)
    print("largest error relative to the weight: 2^%.2f" % np.log2((err / np.maximum(want, 2.0 ** -8)).max() + 1e-30))
    assert np.all(err <= 2.0 ** -19 * want + 2.0 ** -30)
