"""What the Python helpers of the serving operators refuse before an address
reaches the library: tensors that a kernel would read or write as something
else, or out of range (no GPU)."""
import pytest
import torch

import bit_plane_kv_encode_gb300 as pk

N, H, T, D = 2, 3, 5, 128


@pytest.fixture
def cache(monkeypatch):
    c = pk.Rows8(N, H, 4, 512, device="cpu")
    calls = []
    monkeypatch.setattr(pk, "bpkv_rows8_append", lambda *a: calls.append(a))
    c.calls = calls
    return c


def new(shape=(N, H, T, D), dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


BAD_ROWS = [
    new(dtype=torch.float32), new(dtype=torch.float16),                        # as other numbers
    new((N, T, H, D)).transpose(1, 2), new((N, H, T, 2 * D))[..., :D],         # other strides
    new((N - 1, H, T, D)), new((N, H - 1, T, D)), new((N, H, T, D // 2)),      # too few rows, short rows
    new((N, H, T - 1, D)), new((N + 1, H, T, D)),
    new((N * H, T, D)), torch.zeros((N, H, T, D), dtype=torch.bfloat16, device="meta"),
]


@pytest.mark.parametrize("bad", range(len(BAD_ROWS)))
def test_append_refuses_other_rows(cache, bad):
    x = BAD_ROWS[bad]
    for k, v in ((x, new()), (new(), x)):
        with pytest.raises(ValueError):
            cache.append(k, v, stream=0)
    assert not cache.calls


@pytest.mark.parametrize("kw", [
    dict(start=torch.zeros(N, dtype=torch.int32)), dict(start=torch.zeros(N - 1, dtype=torch.int64)),
    dict(start=torch.zeros(2 * N, dtype=torch.int64)[::2]), dict(start=torch.zeros(N, dtype=torch.int64, device="meta")),
    dict(status=torch.zeros(0, dtype=torch.int32)), dict(status=torch.zeros(1, dtype=torch.int32, device="meta"))])
def test_append_refuses_other_starts_and_status(cache, kw):
    with pytest.raises(ValueError):
        cache.append(new(), new(), stream=0, **kw)
    assert not cache.calls


def test_append_takes_what_fits(cache):
    k, v = new(), new()
    starts = (None, torch.zeros(N, dtype=torch.int64), 1 << 20)
    for start in starts:
        for status in (None, torch.zeros(1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8), 1 << 20):
            cache.append(k, v, start, status, 0)
    assert len(cache.calls) == 12 and all(a[1] is k and a[2] is v and a[3] == T for a in cache.calls)
    one = new((N, H, T + 4, D))[:, :, :1].contiguous()
    cache.append(one, one, stream=0)
    assert cache.calls[-1][3] == 1
