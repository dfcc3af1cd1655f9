"""The serving loop that the front page prints, run as it stands: after every
step the cache holds the newest and the first text positions of each sequence.
On the CPU against the reference's calls, on the GPU against the library's."""
import os
import re
import types

import pytest
import torch

import mla_latent_kv_10_gb300 as mla
import oracle
from oracle import cache as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUDGET, RECENT, FIRST = 64, 16, 2
B, H, PAGES, STEPS, PROMPT = 2, 16, 2, 55, (90, 20)


def the_loop():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "mla_cache_evict" in c]
    assert len(code) == 1
    return code[0]


class Reference:
    """The calls of the loop by the fp64 reference, on CPU tensors."""
    KV_FP4 = mla.KV_FP4

    @staticmethod
    def DecodeBuffers(d):
        return types.SimpleNamespace(q_cat=None, lse=None)

    @staticmethod
    def CacheState(d):
        S = d["max_pages"] * 64
        return types.SimpleNamespace(weight=torch.zeros(d["B"], S), position=torch.zeros(d["B"], S, dtype=torch.int32),
                                     workspace=None)

    @staticmethod
    def mla_cache_append(d, fmt, c_kv, k_rope, table, lens, cache, ws, n_new=None, start_position=None, position=None):
        for b in range(d["B"]):
            m = d["Lq"] if n_new is None else int(n_new[b])
            rows = torch.from_numpy(oc.rows("fp4", c_kv[b, :m], k_rope[b, :m]))
            for l in range(m):
                at = int(lens[b]) - m + l
                cache[int(table[b, at // 64]), at % 64] = rows[l]
                position[b, at] = at if start_position is None else int(start_position[b]) + l

    @staticmethod
    def decode_step(d, bufs, q_nope, q_rope, W_UK, W_UV, cache, table, lens, fp4):
        out, _, lse = oracle.decode_fp4(d, q_nope, q_rope, W_UK, W_UV, cache, table, lens)
        q = torch.einsum("blhd,hdc->blhc", q_nope.double(), W_UK.double())
        bufs.q_cat, bufs.lse = torch.cat([q, q_rope.double()], -1).to(torch.bfloat16), lse
        return out

    @staticmethod
    def mla_cache_weights(d, fmt, q_cat, cache, table, lens, lse, weight, ws):
        weight += torch.from_numpy(oc.gathered_weights(d, "fp4", q_cat, cache, table, lens, lse)).float()

    @staticmethod
    def mla_cache_evict(d, fmt, budget, recent, first, table, cache, lens, weight, position, ws):
        new = oc.evict(cache.numpy(), table, lens, weight.numpy(), position.numpy(), budget, recent, first)
        for t, x in zip((cache, lens, weight, position), new):
            t.copy_(torch.from_numpy(x))


def run(calls, device, code):
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(device)
    d = dict(B=B, Lq=1, H=H, d_hc=128, d_c=512, d_R=64, G=1, page_size=64, max_pages=PAGES, num_pages=B * PAGES,
             scale=192.0 ** -0.5, causal=1)
    table = torch.randperm(B * PAGES, generator=g).view(B, PAGES).int().to(device)
    names = dict(mla=calls, dims=d, prompt_dims=dict(d, Lq=max(PROMPT)), table=table, budget=BUDGET, recent=RECENT,
                 first=FIRST, lens=torch.tensor(PROMPT, dtype=torch.int32, device=device),
                 cache=torch.zeros(B * PAGES, 64, 416, dtype=torch.uint8, device=device),
                 c_prompt=rnd(B, max(PROMPT), 512), k_prompt=rnd(B, max(PROMPT), 64),
                 W_UK=rnd(H, 128, 512) * 512 ** -0.5, W_UV=rnd(H, 128, 512) * 512 ** -0.5)

    def check(step):  # after that many steps
        lens, position = names["lens"].tolist(), names["state"].position.cpu()
        for b in range(B):
            text = PROMPT[b] + step
            assert lens[b] == min(text, BUDGET)
            held = position[b, :lens[b]].tolist()
            assert len(set(held)) == lens[b] and set(held) <= set(range(text)), (step, b)
            assert set(range(max(0, text - RECENT), text)) | set(range(FIRST)) <= set(held), (step, b)

    def steps():
        for i in range(STEPS):
            if i:
                check(i)
            yield rnd(B, 1, 512), rnd(B, 1, 64), rnd(B, 1, H, 128), rnd(B, 1, H, 64)

    names["steps"] = steps()
    exec(code, names)
    check(STEPS)
    return names


def test_newest_positions_stay_on_the_reference():
    run(Reference, "cpu", the_loop())


def test_the_check_sees_a_loop_without_text_positions():
    """Cached places instead of text positions: right until the first eviction."""
    code = re.sub(r"start_position=\w+,?", "", the_loop())
    with pytest.raises(AssertionError):
        run(Reference, "cpu", code)


@pytest.mark.gpu
def test_newest_positions_stay_on_the_device():
    from mla_latent_kv_10_gb300 import _build
    _build.build()
    names = run(mla, "cuda", the_loop())
    assert mla.mla_get_device_status(names["state"].workspace) == 0
    assert mla.mla_get_device_status(names["bufs"].workspace) == 0
