"""Refusals of the 8-bit rows, projected-heads and shared-prefix calls: every
argument error is found on the host before anything is enqueued (no GPU)."""
import ctypes

import pytest

EINVAL, ENOWS, EUNSUP = -1, -2, -4
FAKE = 1 << 20  # aligned, non-null, never read on these paths


@pytest.fixture(scope="module")
def L():
    from bit_plane_kv_encode_gb300 import build as B
    from bit_plane_kv_encode_gb300 import _binding
    B.build()
    return _binding.load()


def _rows8(**kw):
    from bit_plane_kv_encode_gb300 import bpkv_rows8
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, cap_tokens=1024, n_max=0, k8=FAKE, v8=FAKE, kexp=FAKE,
             vexp=FAKE, seq_len=FAKE)
    d.update(kw)
    return bpkv_rows8(**d)


def _cache(**kw):
    from bit_plane_kv_encode_gb300 import bpkv_cache
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, cap_tokens=1024, n_max=0, residency=0, reserved=0,
             planes=FAKE, scales=FAKE, k_rows=FAKE, v_rows=FAKE, seq_len=FAKE)
    d.update(kw)
    return bpkv_cache(**d)


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


BAD_ROWS8 = [(dict(head_dim=64), EUNSUP), (dict(n_seq=0), EINVAL), (dict(group=9), EINVAL), (dict(cap_tokens=1000), EINVAL),
             (dict(n_max=1025), EINVAL), (dict(k8=None), EINVAL), (dict(vexp=FAKE + 8), EINVAL),
             (dict(seq_len=FAKE + 4), EINVAL), (dict(n_kv_heads=70000), EUNSUP)]


@pytest.mark.parametrize("bad,rc", BAD_ROWS8)
def test_rows8_struct(L, bad, rc):
    c = _rows8(**bad)
    assert L.bpkv_rows8_append(ctypes.byref(c), FAKE, FAKE, 1, None, None, None) == rc
    assert L.bpkv_rows8_read(ctypes.byref(c), 0, 1, FAKE, FAKE, None) == rc
    assert L.bpkv_shared_attend8(None, None, ctypes.byref(c), FAKE, FAKE, FAKE, 1 << 40, None) == rc


@pytest.mark.parametrize("k,v,t,start,status,n_max", [
    (None, FAKE, 1, None, None, 0), (FAKE, None, 1, None, None, 0), (FAKE + 8, FAKE, 1, None, None, 0),
    (FAKE, FAKE, 0, None, None, 0), (FAKE, FAKE, 1025, FAKE * 2, None, 0), (FAKE, FAKE, 2, None, None, 1023),
    (FAKE, FAKE, 2, FAKE, None, 1023), (FAKE, FAKE, 1, FAKE * 2 + 4, None, 0), (FAKE, FAKE, 1, None, FAKE + 2, 0)])
def test_rows8_append(L, k, v, t, start, status, n_max):
    c = _rows8(n_max=n_max)
    assert L.bpkv_rows8_append(ctypes.byref(c), _p(k), _p(v), t, _p(start), _p(status), None) == EINVAL
    assert c.n_max == n_max


@pytest.mark.parametrize("t0,n,k,v", [(-1, 1, FAKE, FAKE), (0, 0, FAKE, FAKE), (1024, 1, FAKE, FAKE), (1, 1024, FAKE, FAKE),
                                      (0, 1, None, None), (0, 1, FAKE + 8, None), ((1 << 63) - 1, 1, FAKE, FAKE)])
def test_rows8_read(L, t0, n, k, v):
    assert L.bpkv_rows8_read(ctypes.byref(_rows8()), t0, n, _p(k), _p(v), None) == EINVAL


def _qkv(**kw):
    from bit_plane_kv_encode_gb300 import bpkv_qkv_args
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, t_new=1, rot_dim=128, flags=0, eps=1e-6, qkv=FAKE,
             ld=12 * 128, pos=FAKE * 2, inv_freq=FAKE, q_weight=None, k_weight=None, q_out=FAKE * 3, k_out=FAKE * 4,
             v_out=FAKE * 5)
    d.update(kw)
    return bpkv_qkv_args(**d)


@pytest.mark.parametrize("bad,rc", [
    (dict(head_dim=64), EUNSUP), (dict(n_seq=0), EINVAL), (dict(t_new=0), EINVAL), (dict(group=9), EINVAL),
    (dict(rot_dim=3), EINVAL), (dict(rot_dim=130), EINVAL), (dict(rot_dim=-2), EINVAL), (dict(inv_freq=None), EINVAL),
    (dict(flags=4), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(ld=12 * 128 - 8), EINVAL),
    (dict(ld=12 * 128 + 4), EINVAL), (dict(qkv=None), EINVAL), (dict(q_out=None), EINVAL), (dict(qkv=FAKE + 2), EINVAL),
    (dict(k_out=FAKE + 8), EINVAL), (dict(pos=None), EINVAL), (dict(pos=FAKE + 4), EINVAL),
    (dict(q_weight=FAKE + 2), EINVAL), (dict(n_seq=65536), EUNSUP), (dict(ld=1 << 61), EUNSUP),
    # outputs in the input (its last row), in one another
    (dict(q_out=FAKE + 12 * 128 * 2), EINVAL), (dict(k_out=FAKE + 2 * 12 * 128 * 2 - 16), EINVAL),
    (dict(v_out=FAKE), EINVAL), (dict(k_out=FAKE * 3 + 2 * 8 * 128 * 4 - 16), EINVAL), (dict(v_out=FAKE * 3 - 16), EINVAL),
    (dict(v_out=FAKE * 4 + 16), EINVAL)])
def test_qkv(L, bad, rc):
    a = _qkv(**bad)
    assert L.bpkv_qkv_rope(ctypes.byref(a), None) == rc


@pytest.mark.parametrize("bad,t,pos", [(dict(n_seq=3), 1, FAKE * 2), (dict(n_kv_heads=1), 1, FAKE * 2),
                                       (dict(k8=None), 1, FAKE * 2), (dict(), 1025, FAKE * 2), (dict(n_max=1024), 1, None),
                                       (dict(n_max=1024), 1, FAKE)])
def test_qkv_into_rows8(L, bad, t, pos):
    c = _rows8(**bad)
    a = _qkv(t_new=t, pos=pos, rows8=ctypes.pointer(c))
    assert L.bpkv_qkv_rope(ctypes.byref(a), None) == EINVAL


def test_null_structs(L):
    assert L.bpkv_qkv_rope(None, None) == EINVAL
    assert L.bpkv_rows8_append(None, FAKE, FAKE, 1, None, None, None) == EINVAL
    assert L.bpkv_rows8_read(None, 0, 1, FAKE, FAKE, None) == EINVAL
    assert L.bpkv_shared_attend(None, None, None, FAKE, FAKE, FAKE, 1 << 40, None) == EINVAL


def test_qkv_args_shapes():
    import torch

    import bit_plane_kv_encode_gb300 as pk
    qkv = torch.zeros((2, 3, 12 * 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 3, 2, 4, 128))
    a = pk.qkv_args(qkv, q, 2, pos=torch.zeros(2, dtype=torch.int64), inv_freq=torch.ones(32), pairs=True)
    assert (a.n_seq, a.t_new, a.n_kv_heads, a.group, a.rot_dim, a.flags, a.ld) == (2, 3, 2, 4, 64, pk.QKV_PAIRS, 12 * 128)
    for kw in (dict(pos=torch.zeros(2, dtype=torch.int32)), dict(pos=torch.zeros(3, dtype=torch.int64)),
               dict(k_out=torch.zeros((2, 2, 3, 128))), dict(inv_freq=torch.ones(32, dtype=torch.float64)),
               dict(q_weight=torch.ones(64))):
        with pytest.raises(ValueError):
            pk.qkv_args(qkv, q, 2, **{"pos": torch.zeros(2, dtype=torch.int64), **kw})
    with pytest.raises(ValueError):
        pk.qkv_args(qkv[:, :2], q[:, :2].contiguous(), 2, pos=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pk.qkv_args(qkv, q, 3)


def test_shared_workspace_size(L):
    f = L.bpkv_shared_workspace_size
    assert f(1, 0, 1, 1) > 256
    assert f(32, 1, 8, 4) > f(32, 0, 8, 4)
    for bad in [(0, 0, 1, 1), (513, 0, 1, 1), (1, 513, 1, 1), (1, -1, 1, 1), (1, 0, 0, 1), (1, 0, 1, 0), (1, 0, 1, 9)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_shared_attend(L, bits):
    fn, mk = (L.bpkv_shared_attend, _cache) if bits == 16 else (L.bpkv_shared_attend8, _rows8)
    c, p = mk(), mk(n_seq=1)
    ws, big = 1 << 20, 1 << 40

    def call(prefix=None, of=None, own=None, q=FAKE, out=FAKE, w=ws, n=big):
        own = c if own is None else own
        return fn(None if prefix is None else ctypes.byref(prefix), _p(of), ctypes.byref(own), _p(q), _p(out), _p(w), n,
                  None)

    assert call(q=None) == EINVAL and call(out=None) == EINVAL and call(q=FAKE + 8) == EINVAL
    assert call(of=FAKE + 2, prefix=p) == EINVAL
    assert call(prefix=mk(n_kv_heads=3)) == EINVAL and call(prefix=mk(group=2)) == EINVAL
    assert call(prefix=mk(cap_tokens=100)) == EINVAL
    assert call(own=mk(n_seq=513)) == EUNSUP and call(prefix=mk(n_seq=513)) == EUNSUP
    assert call(own=mk(cap_tokens=1 << 31)) == EUNSUP
    assert call(w=None) == ENOWS and call(w=FAKE + 128) == ENOWS and call(n=1000) == ENOWS
    need = L.bpkv_shared_workspace_size(2, 1, 2, 4)
    assert call(prefix=p, n=need - 1) == ENOWS
    size = 2 * 2 * 4 * 128 * 2
    assert call() == EINVAL and call(out=FAKE + size - 16) == EINVAL and call(q=FAKE + 16) == EINVAL
    if bits == 16:
        assert call(own=mk(residency=1)) == EUNSUP and call(prefix=mk(residency=1, n_seq=1)) == EUNSUP
