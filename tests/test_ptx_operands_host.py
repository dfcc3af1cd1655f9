"""Operands of the inline PTX wrappers that PTX restricts (no GPU): read from
the source."""
import os
import re

from mla_latent_kv_10_gb300 import _build


def test_phase_parity_is_zero_or_one():
    """mbarrier.try_wait.parity takes the parities 0 and 1 only; callers count
    phases, so each wrapper takes the low bit itself."""
    text = open(os.path.join(_build.CSRC, "ptx.cuh")).read()
    waits = re.findall(r'"mbarrier\.try_wait\.parity[^;]*;.*?\);', text, re.S)
    assert len(waits) == 2
    for w in waits:
        assert re.search(r'"r"\(parity & 1\)', w), w
    for name in os.listdir(_build.CSRC):  # nothing waits past the wrappers
        if name != "ptx.cuh":
            body = open(os.path.join(_build.CSRC, name)).read()
            assert "mbarrier.try_wait" not in body and "mbarrier.test_wait" not in body, name
