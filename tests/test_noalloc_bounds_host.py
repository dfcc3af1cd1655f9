"""The allocation-free entry point's scratch and what its merge may read of it
(no GPU).  The merge clips every slot that the split plan names to a bound, so
that a plan spoilt by another call on the shared scratch leads to wrong numbers
and never past the array; the bound has to be the count the scratch was laid
out for.  The file is compiled with the host compiler against stand-ins for the
calls it makes, which record that bound."""
import os
import shutil
import subprocess

import pytest

from mla_latent_kv_10_gb300 import _build

CUDA_INCLUDE = os.path.join(os.path.dirname(os.path.dirname(shutil.which(_build.nvcc()) or _build.nvcc())), "include")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")),
                                reason="g++ or the CUDA headers not found")

HARNESS = r"""
#include "mla_noalloc.cu"
#include <cstdio>
#include <cstdlib>

static unsigned char* array;                 // stands for the scratch array on the device
static long long read_end;                   // bytes from its start that the merge may read up to
static int kUnits, kUnitsAnyFormat;

static void merge(const mla_dims* d, const float* o_part, const float* lse_part, int slots) {
  const long long rows = (long long)d->Lq * d->H;
  const long long o = reinterpret_cast<const unsigned char*>(o_part) - array + slots * rows * 512 * 4;
  const long long l = reinterpret_cast<const unsigned char*>(lse_part) - array + slots * rows * 4;
  read_end = o > l ? o : l;
}

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = array; return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
int mla_decode_workspace_size(const mla_dims* d, size_t* n) { *n = mla::ws_bytes_for(d->B); return MLA_OK; }
int mla_decode_num_slots(const mla_dims* d, int* n) { *n = d->B + kUnitsAnyFormat - 1; return MLA_OK; }
int mla_decode_paged(const mla_dims*, const void*, const void*, const int32_t*, const int32_t*, int, float*, float*,
                     void*, size_t, void*) { return MLA_OK; }
int mla_combine_splits(const mla_dims* d, const float* o, const float* l, const void*, size_t, void*, float*, void*) {
  merge(d, o, l, d->B + kUnitsAnyFormat - 1);  // the public merge: buffers sized by mla_decode_num_slots
  return MLA_OK;
}
}
namespace mla {
int decode_max_units(bool, bool, int, int* units) { *units = kUnits; return MLA_OK; }
cudaError_t launch_combine(const float* o, const float* l, const WsHeader*, void*, float*, int B, int Lq, int H, int G,
                           int slots, cudaStream_t) {
  mla_dims d = {};
  d.B = B, d.Lq = Lq, d.H = H, d.G = G;
  merge(&d, o, l, slots);
  return cudaSuccess;
}
}  // namespace mla

int main(int argc, char** argv) {
  mla_dims d = {};
  d.B = atoi(argv[1]), d.Lq = 1, d.H = atoi(argv[2]), d.G = 1;
  kUnits = atoi(argv[3]), kUnitsAnyFormat = atoi(argv[4]);
  array = static_cast<unsigned char*>(aligned_alloc(256, 256));  // an address; nothing is read
  void* p = array;
  const int rc = mla_decode_attend_noalloc(&d, p, p, static_cast<int32_t*>(p), static_cast<int32_t*>(p), p,
                                           static_cast<float*>(p), static_cast<int*>(p), nullptr);
  printf("%d %lld %zu\n", rc, read_end, mla::kNoAllocScratchBytes);
  free(array);
  return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    at = tmp_path_factory.mktemp("noalloc")
    src, exe = at / "harness.cpp", at / "harness"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O0", "-I", CUDA_INCLUDE, "-I", os.path.join(_build.ROOT, "include"),
                    "-I", _build.CSRC, str(src), "-o", str(exe), "-lpthread"], check=True, capture_output=True, text=True)
    return lambda *a: [int(x) for x in subprocess.run([str(exe), *map(str, a)], check=True, capture_output=True,
                                                      text=True).stdout.split()]


@pytest.mark.parametrize("units_any_format", [76, 152])
@pytest.mark.parametrize("B,H", [(1, 16), (900, 16), (940, 16), (1, 128), (50, 128)])
def test_the_merge_reads_inside_the_scratch(harness, B, H, units_any_format):
    """76 work units for the bf16 decode; another format may have more."""
    rc, read_end, size = harness(B, H, 76, units_any_format)
    assert rc == 0 and 0 < read_end <= size


def test_what_does_not_fit_is_refused(harness):
    assert harness(1024, 128, 76, 76)[0] == -4
