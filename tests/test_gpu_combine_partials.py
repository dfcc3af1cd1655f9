"""The merge of the split partials for every small number of them, on every
form of the kernel: partials of known values, put where a decode left its own,
against the definition in 64 bits.

Tolerances: a weight exp(lse_k - L) is off by 2^-24 of |lse_k - L| <= 40 and
by its exponential's 2^-22 (together below 2^-17 where it counts), the sum of
up to 20 products by 20 * 2^-24 of their sizes, the result by half a step of
bf16, 2^-8: |o - ref| <= 2^-8 |ref| + 2^-16 sum_k w_k |o_k|; |L - ref| <= 2^-20
max(1, |ref|) (a sum and a logarithm, an addition at the size of L)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_10_gb300 as mla
from mla_latent_kv_10_gb300.inputs import make_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    mla.load_library()


def merged(c, bufs, n):
    """(o_lat, lse) of the merge and of its definition; n: partials a sequence."""
    d = c.dims
    B, H, G = d["B"], d["H"], d["G"]
    d_g = 512 // G
    g = torch.Generator().manual_seed(n + 100 * G)
    o = torch.randn(bufs.slots, 128, H, 4, generator=g)          # [slot][column / 4][row][4]
    l = 3.0 * torch.randn(bufs.slots, H, generator=g)
    l[:, 1] = -float("inf")                                      # a row without keys
    l[::2, 2] -= 200.0                                           # partials that weigh nothing
    l[1::3, 3] = -float("inf")
    bufs.o_part.copy_(o.reshape(bufs.o_part.shape))
    bufs.lse_part.copy_(l)
    bufs.o_lat.fill_(float("nan"))
    bufs.lse.fill_(float("nan"))
    mla.mla_combine_splits(d, bufs.o_part, bufs.lse_part, bufs.workspace, bufs.o_lat, bufs.lse)
    ws = bufs.workspace.cpu().numpy()[32:].view(np.int32)        # off[B + 1], nlen[B], slot0[B], nslot[B]
    first, count = ws[2 * B + 1:3 * B + 1], ws[3 * B + 1:4 * B + 1]
    assert np.all(count == n), count
    o = o.double().numpy().transpose(0, 2, 1, 3).reshape(bufs.slots, H, 512)
    l = l.double().numpy()
    ref, size, lse = np.zeros((B, H, d_g)), np.zeros((B, H, d_g)), np.full((B, H), -np.inf)
    for b in range(B):
        for h in range(H):
            k = slice(first[b], first[b] + n)
            if np.all(l[k, h] == -np.inf):
                continue
            lse[b, h] = np.logaddexp.reduce(l[k, h])
            w = np.exp(l[k, h] - lse[b, h])[:, None]
            x = o[k, h, h * G // H * d_g:][:, :d_g]
            ref[b, h], size[b, h] = (w * x).sum(0), (w * np.abs(x)).sum(0)
    return bufs.o_lat[:, 0].double().cpu().numpy(), bufs.lse[:, 0].double().cpu().numpy(), ref, size, lse


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 10, 16, 20])
@pytest.mark.parametrize("B,H,G", [
    (1, 16, 1), (2, 48, 1), (1, 32, 2), (1, 32, 4), (2, 128, 4), (1, 16, 8), (3, 128, 8),  # 16 columns a block
    (3, 128, 1), (7, 128, 4),                                                              # 64
])
def test_every_number_of_partials(B, H, G, n):
    if B * n > 70:
        n = 70 // B
    c = make_case(B=B, Lq=1, H=H, G=G, seq_lens=[64 * n] * B, table="perm", seed=1)
    t = {k: v.cuda() for k, v in c.tensors().items()}
    bufs = mla.DecodeBuffers(c.dims)
    bufs.q_cat.zero_()
    mla.mla_decode_paged(c.dims, bufs.q_cat, t["cache"], t["block_table"], t["seq_lens"], B * n, bufs.o_part,
                         bufs.lse_part, bufs.workspace)
    o, l, ref, size, lse = merged(c, bufs, n)
    assert np.all(np.abs(o - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * size)
    live = np.isfinite(lse)
    assert np.array_equal(np.isneginf(l), ~live)
    assert np.all(np.abs(l[live] - lse[live]) <= 2.0 ** -20 * np.maximum(1.0, np.abs(lse[live])))
    assert mla.mla_get_device_status(bufs.workspace) == 0
