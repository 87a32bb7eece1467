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


def heads(G=4, **kw):
    """Arguments of qkv_args that fit, with those of kw in their place."""
    d = dict(qkv=new((N, T, (G + 2) * H * D)), q_out=torch.zeros((N, T, H, G, D)), n_kv_heads=H,
             pos=torch.zeros(N, dtype=torch.int64), inv_freq=torch.ones(D // 2), q_weight=torch.ones(D),
             k_weight=torch.ones(D), k_out=new(), v_out=new())
    d.update(kw)
    return d


def test_qkv_args_takes_what_fits():
    pk.qkv_args(**heads())
    pk.qkv_args(**heads(rows8=pk.Rows8(N, H, 4, 512, device="cpu"), status=torch.zeros(1, dtype=torch.int32)))
    pk.qkv_args(**heads(status=torch.zeros(256, dtype=torch.uint8), pos=None, q_weight=None, k_out=None, v_out=None,
                        rows8=pk.Rows8(N, H, 4, 512, device="cpu")))


@pytest.mark.parametrize("name", ["q_out", "pos", "inv_freq", "q_weight", "k_weight", "k_out", "v_out", "status", "rows8"])
def test_qkv_args_refuses_tensors_of_another_device(name):
    d = heads(status=torch.zeros(1, dtype=torch.int32), rows8=pk.Rows8(N, H, 4, 512, device="cpu"))
    if name == "rows8":
        d["rows8"].k8 = d["rows8"].k8.to("meta")
    else:
        d[name] = d[name].to("meta")
    with pytest.raises(ValueError):
        pk.qkv_args(**d)


@pytest.mark.parametrize("kw", [
    dict(inv_freq=torch.ones(D)[::2]), dict(inv_freq=torch.ones((D // 2, 1))), dict(pos=torch.zeros((N, 1), dtype=torch.int64)),
    dict(q_weight=torch.ones(2 * D)[::2]), dict(k_out=new((N, T, H, D)).transpose(1, 2)),
    dict(status=torch.zeros(0, dtype=torch.int32))])
def test_qkv_args_refuses_other_tensors(kw):
    with pytest.raises(ValueError):
        pk.qkv_args(**heads(**kw))


def test_n_max_is_the_callers_to_set():
    c = pk.Rows8(N, H, 4, 512, device="cpu")
    for n in (512, 0, 77):
        c.n_max = n
        assert c.n_max == n == c.c.n_max
    for n in (-1, 513):
        with pytest.raises(ValueError):
            c.n_max = n
    assert c.n_max == 77
