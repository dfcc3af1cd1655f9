"""The FP4 decode compiles without register spills in any of its forms (no
GPU): its softmax sits at the limit of 96 registers, and a spill there costs
more than any step it was won by."""
import os
import shutil

import pytest

from mla_latent_kv_10_gb300 import _build
from test_build_resources import NVCC, resource_report

pytestmark = pytest.mark.skipif(shutil.which(NVCC) is None and not os.path.exists(NVCC), reason="nvcc not found")


def test_no_form_spills(tmp_path):
    found = {n: r for n, r in resource_report(os.path.join(_build.CSRC, "mla_decode_fp4.cu"), tmp_path).items()
             if "decode_fp4_kernel" in n}
    assert len(found) == 12 and all(r.get("spill", 0) == 0 for r in found.values()), found
