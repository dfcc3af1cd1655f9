"""Host-only checks of the Python binding."""
import types

import pytest

import mla_latent_kv_10_gb300 as mla


def fake_torch(names):
    c = types.SimpleNamespace(**{n: f for n, f in (("_cuda_getDevice", lambda: 3),
                                                   ("_cuda_getCurrentRawStream", lambda d: 100 + d)) if n in names})
    return types.SimpleNamespace(_C=c, cuda=types.SimpleNamespace(
        current_stream=lambda: types.SimpleNamespace(cuda_stream=77)))


@pytest.mark.parametrize("names,want", [
    (("_cuda_getDevice", "_cuda_getCurrentRawStream"), 103),
    (("_cuda_getDevice",), 77), (("_cuda_getCurrentRawStream",), 77), ((), 77),
])
def test_current_stream_without_the_private_names(names, want):
    """A torch without its private entry points is asked by the public one."""
    assert mla._current_stream_of(fake_torch(names))() == want


def test_streams_given():
    assert mla._stream(5) == 5 and mla._stream(types.SimpleNamespace(cuda_stream=9)) == 9
