"""The quantised cache's Python calls with tensors of too few dimensions or no elements in a head:
ValueError, as for any other shape that does not fit (no GPU is touched)."""
import pytest

torch = pytest.importorskip("torch")


def _calls():
    import prng_seeded_decode_amd as S

    ints = torch.zeros(2, dtype=torch.int32)
    return {
        "append": lambda x, c, p: S.QCacheAppendCall(x, x, x, x, x, ints, ints, x, c, c, p, p),
        "read": lambda x, c, p: S.QCacheReadCall(c, c, p, p, ints, x, None),
        "attend": lambda x, c, p: S.QCacheAttendCall(x, c, c, p, p, ints.view(2, 1), ints, x),
    }


@pytest.mark.parametrize("call", ["append", "read", "attend"])
@pytest.mark.parametrize("shape", [(), (64,), (2, 64), (2, 2, 0), (0,), (1, 2, 2, 64)])
def test_a_shape_that_is_no_rows_of_heads(shape, call, monkeypatch):
    from prng_seeded_decode_amd import _serve

    monkeypatch.setattr(_serve, "_on_device", lambda tensors: 0)
    c = torch.zeros(3, 16, 2, 32, dtype=torch.uint8)
    p = torch.zeros(3, 16, 2, 1, 2, dtype=torch.float16)
    with pytest.raises(ValueError):
        _calls()[call](torch.zeros(shape, dtype=torch.float16), c, p)
