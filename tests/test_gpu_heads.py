"""Whole steps at every number of heads the decode takes, with grouped latents
and several new tokens: half the heads of a token (a copy's rows in the grouped
decode) need not divide a block's 128 query rows."""
import pytest

import mla_latent_kv_10_gb300 as mla
from mla_latent_kv_10_gb300.inputs import make_case
from parity_util import check_case, run_gpu, sample_pairs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    mla.load_library()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("H", [48, 80, 96, 112])
@pytest.mark.parametrize("Lq", [1, 2, 3, 4])
def test_step_at_every_number_of_heads(Lq, H, G, kv):
    c = make_case(B=3, Lq=Lq, H=H, G=G, seq_lens=[Lq, 65, 700], table="perm", seed=10 * H + Lq, kv=kv)
    got = run_gpu(c)
    assert got["status"] == 0
    check_case(c, got, sample_pairs(c, 8))
