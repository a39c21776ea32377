"""The stream that a call without one runs on (CPU only; torch's stream queries are stand-ins)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from prng_seeded_decode_amd import _binding  # noqa: E402


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(0x5000))
    return monkeypatch


def test_current_stream_without_torchs_private_query(current):
    current.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert _binding._stream_ptr(None).value == 0x5000


def test_current_stream_by_the_raw_query(current):
    asked = []
    current.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: asked.append(d) or 0x5000,
                    raising=False)
    assert _binding._stream_ptr(None).value == 0x5000 and asked == [3]


def test_given_streams():
    assert _binding._stream_ptr(0x7000).value == 0x7000
    assert _binding._stream_ptr(Stream(0x7000)).value == 0x7000
    assert isinstance(_binding._stream_ptr(0), ctypes.c_void_p)
