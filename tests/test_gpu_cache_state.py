"""GPU tests of what mla_cache_weights and mla_cache_evict leave behind: the
weights and positions outlive the call, so a sequence or a page that the call
refuses must not change them."""
import numpy as np
import pytest
import torch

import mla_latent_kv_10_gb300 as mla
from oracle import cache as oc
from test_gpu_cache import FMT, MLA_ERR_BAD_SEQLEN, MLA_ERR_BAD_TABLE, case_and_query, evict, lse_of, same, status_of, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    mla.load_library()


def start_weights(dims):
    g = torch.Generator().manual_seed(31)
    return torch.rand(dims["B"], dims["max_pages"] * 64, generator=g)


def weights(kv, c, q, lse, table=None, lens=None):
    w, ws = start_weights(c.dims).cuda(), torch.zeros(64, dtype=torch.uint8, device="cuda")
    table, lens = c.block_table if table is None else table, c.seq_lens if lens is None else lens
    mla.mla_cache_weights(c.dims, FMT[kv], q.cuda(), c.cache.cuda(), table.cuda(), lens.cuda(), lse.cuda(), w, ws)
    return w.cpu(), status_of(ws)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("B,G", [(3, 1), (3, 4), (40, 1)])
def test_weights_leave_a_sequence_of_bad_length_alone(kv, B, G):
    """An idle place of the batch (length 0), a length below the new tokens',
    one past the table: that sequence's weights keep their bits, the others
    get what they get beside a good one."""
    lens = [100 + (37 * b) % 150 for b in range(B)]
    c, q = case_and_query(kv, B, 2, 16, G, lens)
    lse = lse_of(kv, c, q)
    good, st = weights(kv, c, q, lse)
    assert st == 0
    for bad in (0, 1, -7, c.dims["max_pages"] * 64 + 1):
        n = c.seq_lens.clone()
        n[1] = bad
        table = c.block_table.clamp(min=0)  # (a clamped length may walk over the unused entries)
        got, st = weights(kv, c, q, lse, table=table, lens=n)
        assert st == MLA_ERR_BAD_SEQLEN
        assert torch.equal(got[1], start_weights(c.dims)[1])
        got[1] = good[1]
        assert torch.equal(got, good)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("B,G,page", [(2, 1, 0), (2, 1, 1), (2, 4, 2), (34, 1, 3)])
def test_weights_leave_tokens_behind_a_bad_entry_alone(kv, B, G, page):
    lens = [230] + [100 + (37 * b) % 150 for b in range(1, B)]
    c, q = case_and_query(kv, B, 2, 16, G, lens)
    lse = lse_of(kv, c, q)
    good, st = weights(kv, c, q, lse)
    assert st == 0
    for entry in (-1, c.dims["num_pages"]):
        table = c.block_table.clone()
        table[0, page] = entry
        got, st = weights(kv, c, q, lse, table=table)
        assert st == MLA_ERR_BAD_TABLE
        at = slice(64 * page, 64 * page + 64)
        assert torch.equal(got[0, at], start_weights(c.dims)[0, at])
        got[0, at] = good[0, at]
        assert torch.equal(got, good)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("mp,n,budget,bad", [(4, 250, 100, 0), (4, 250, 100, 1), (4, 250, 100, 3), (70, 4400, 1000, 9), (70, 4400, 1000, 40)])
def test_evict_keeps_the_labels_of_rows_it_does_not_move(fmt, mp, n, budget, bad):
    """Where an entry of a move is bad the row stays, and so must the weight
    and the position that go with it."""
    table, num_pages = tables(1, mp, mp)
    S = mp * 64
    g = torch.Generator().manual_seed(budget)
    w, p = torch.rand(1, S, generator=g), torch.randperm(S, generator=g).int()[None]
    lens = torch.tensor([n], dtype=torch.int32)
    broken = table.clone()
    broken[0, bad] = num_pages if bad % 2 else -3
    raw, *got, st = evict(fmt, broken, num_pages, lens, w, p, budget, 10, 2)
    assert st == MLA_ERR_BAD_TABLE
    # the reference's moves, less those that touch the bad page
    rows, want_n, want_w, want_p = oc.evict(raw, table, lens, w, p, budget, 10, 2)
    moved_from = {int(x): i for i, x in enumerate(p[0, :n])}
    skipped = 0
    for to in range(budget):
        src = moved_from[int(want_p[0, to])]
        if src != to and bad in (to // 64, src // 64):
            want_w[0, to], want_p[0, to] = w[0, to], p[0, to]
            rows[int(table[0, to // 64]), to % 64] = raw[int(table[0, to // 64]), to % 64]
            skipped += 1
    assert skipped > 0
    same(got, (rows, want_n, want_w, want_p))
