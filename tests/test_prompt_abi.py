"""Refusals of the calls for several new tokens of a sequence (prompts, trees,
accepted tokens): every argument error is found on the host before anything is
enqueued (no GPU)."""
import ctypes

import pytest
import torch

import bit_plane_kv_encode_gb300 as pk

EINVAL, ENOWS, EUNSUP = -1, -2, -4
FAKE = 1 << 40  # aligned, non-null, never read on these paths
STEP = 1 << 36  # far enough apart that nothing overlaps
D = 128


@pytest.fixture(scope="module")
def L():
    from bit_plane_kv_encode_gb300 import build as B
    from bit_plane_kv_encode_gb300 import _binding
    B.build()
    return _binding.load()


def _rows8(**kw):
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, cap_tokens=1024, n_max=0, k8=FAKE, v8=FAKE + STEP,
             kexp=FAKE + 2 * STEP, vexp=FAKE + 3 * STEP, seq_len=FAKE)
    d.update(kw)
    return pk.bpkv_rows8(**d)


def _cache(**kw):
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, cap_tokens=1024, n_max=0, residency=0, reserved=0,
             planes=FAKE, scales=FAKE, k_rows=FAKE, v_rows=FAKE + STEP, seq_len=FAKE)
    d.update(kw)
    return pk.bpkv_cache(**d)


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _prompt(**kw):
    d = dict(n_seq=2, n_kv_heads=2, group=4, head_dim=128, n_tokens=300, q_start=FAKE, q=FAKE + 4 * STEP, ld_q=8 * D,
             out=FAKE + 5 * STEP, k=FAKE + 6 * STEP, v=FAKE + 7 * STEP, ld_k=0, ld_v=0)
    d.update(kw)
    return pk.bpkv_prompt_args(**d)


def _cached(struct, **kw):
    a = _prompt(k=None, v=None, **kw)
    setattr(a, "cache" if isinstance(struct, pk.bpkv_cache) else "rows8", ctypes.pointer(struct))
    return a


QB, KB = 300 * 8 * D * 2, 300 * 2 * D * 2  # bytes of q, of k


@pytest.mark.parametrize("bad,rc", [
    (dict(head_dim=64), EUNSUP), (dict(n_seq=0), EINVAL), (dict(n_kv_heads=0), EINVAL), (dict(group=0), EINVAL),
    (dict(group=9), EINVAL), (dict(n_tokens=0), EINVAL), (dict(n_tokens=-5), EINVAL), (dict(n_seq=513), EUNSUP),
    (dict(n_kv_heads=65536), EUNSUP), (dict(n_tokens=(1 << 30) + 1), EUNSUP),
    (dict(n_tokens=1 << 29, n_kv_heads=4, ld_q=16 * D), EUNSUP), (dict(q_start=None), EINVAL),
    (dict(q_start=FAKE + 4), EINVAL), (dict(q=None), EINVAL), (dict(q=FAKE + 8), EINVAL), (dict(out=None), EINVAL),
    (dict(out=FAKE + 2), EINVAL), (dict(ld_q=8 * D - 8), EINVAL), (dict(ld_q=8 * D + 4), EINVAL),
    (dict(ld_q=(1 << 32) + 8), EUNSUP), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=None, v=None), EINVAL),
    (dict(k=FAKE + 8), EINVAL), (dict(v=FAKE + 8), EINVAL), (dict(ld_k=2 * D), EINVAL), (dict(ld_v=2 * D), EINVAL),
    (dict(ld_k=2 * D, ld_v=2 * D - 8), EINVAL), (dict(ld_k=2 * D + 4, ld_v=2 * D), EINVAL),
    (dict(ld_k=-2 * D, ld_v=2 * D), EINVAL), (dict(ld_k=1 << 33, ld_v=2 * D), EUNSUP),
    # out in q, in k, in v (their last rows)
    (dict(out=FAKE + 4 * STEP + QB - 16), EINVAL), (dict(out=FAKE + 4 * STEP - QB + 16), EINVAL),
    (dict(out=FAKE + 6 * STEP + KB - 16), EINVAL), (dict(out=FAKE + 7 * STEP + KB - 16), EINVAL),
    (dict(ld_k=4 * D, ld_v=2 * D, out=FAKE + 6 * STEP + 299 * 4 * D * 2), EINVAL)])
def test_prompt(L, bad, rc):
    a = _prompt(**bad)
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == rc


def test_prompt_units_that_do_not_count_in_32_bits(L):
    a = _prompt(n_tokens=1 << 21, n_kv_heads=8, ld_q=32 * D)
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 50, None) == EUNSUP


def test_prompt_workspace(L):
    a = _prompt()
    need = L.bpkv_prompt_workspace_size(300, 4)
    assert need > 256
    for ws, n in ((None, 1 << 40), (FAKE + 128, 1 << 40), (FAKE, need - 1)):
        assert L.bpkv_prompt_attend(ctypes.byref(a), _p(ws), n, None) == ENOWS
    assert L.bpkv_prompt_attend(None, FAKE, 1 << 40, None) == EINVAL
    for bad in ((0, 4), (1, 0), (1, 9), ((1 << 30) + 1, 1), (-1, 1)):
        assert L.bpkv_prompt_workspace_size(*bad) == 0
    assert L.bpkv_prompt_workspace_size(32, 4) < L.bpkv_prompt_workspace_size(33, 4)


BAD_SOURCES = [(dict(n_seq=3), EINVAL), (dict(n_kv_heads=3), EINVAL), (dict(group=2), EINVAL), (dict(head_dim=64), EUNSUP),
               (dict(cap_tokens=1000), EINVAL), (dict(seq_len=None), EINVAL), (dict(n_max=1025), EINVAL),
               (dict(cap_tokens=(1 << 30) + 512), EUNSUP)]


@pytest.mark.parametrize("bad,rc", BAD_SOURCES)
@pytest.mark.parametrize("make", [_cache, _rows8])
def test_prompt_over_a_cache(L, make, bad, rc):
    c = make(**bad)
    a = _cached(c)
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == rc


@pytest.mark.parametrize("make", [_cache, _rows8])
def test_prompt_takes_one_source(L, make):
    c = make()
    a = _cached(c, )
    a.k = a.v = FAKE
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == EINVAL
    a = _cached(_cache())
    a.rows8 = ctypes.pointer(_rows8())
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == EINVAL
    a = _cached(c, out=FAKE + 1024)  # in the rows
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == EINVAL
    a = _cached(_cache(residency=1))
    assert L.bpkv_prompt_attend(ctypes.byref(a), FAKE, 1 << 40, None) == EUNSUP


@pytest.mark.parametrize("bits", [16, 8])
def test_tree(L, bits):
    fn, make = (L.bpkv_tree_attend, _cache) if bits == 16 else (L.bpkv_tree_attend8, _rows8)
    q, out = FAKE + 4 * STEP, FAKE + 5 * STEP

    def call(c=None, t=8, tree=FAKE, q=q, out=out, ws=FAKE, n=1 << 40):
        c = make() if c is None else c
        return fn(ctypes.byref(c), t, _p(tree), _p(q), _p(out), _p(ws), n, None)

    assert call(t=0) == EINVAL and call(t=65) == EINVAL and call(t=-1) == EINVAL
    assert call(q=None) == EINVAL and call(out=None) == EINVAL and call(q=q + 8) == EINVAL and call(out=out + 8) == EINVAL
    assert call(tree=FAKE + 4) == EINVAL
    size = 2 * 8 * 2 * 4 * D * 2
    assert call(out=q) == EINVAL and call(out=q + size - 16) == EINVAL and call(out=FAKE) == EINVAL
    assert call(c=make(head_dim=64)) == EUNSUP and call(c=make(cap_tokens=100)) == EINVAL
    assert call(c=make(n_seq=513)) == EUNSUP and call(c=make(cap_tokens=(1 << 30) + 512)) == EUNSUP
    need = L.bpkv_prompt_workspace_size(8, 4)
    assert call(ws=None) == ENOWS and call(ws=FAKE + 64) == ENOWS and call(n=need - 1) == ENOWS
    if bits == 16:
        assert call(c=make(residency=1)) == EUNSUP
    assert fn(None, 8, None, q, out, FAKE, 1 << 40, None) == EINVAL


@pytest.mark.parametrize("bad,rc", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=FAKE + 8), EINVAL), (dict(v=FAKE + 8), EINVAL), (dict(t=0), EINVAL),
    (dict(t=1025), EINVAL), (dict(start=None), EINVAL), (dict(start=FAKE * 2 + 4), EINVAL), (dict(path=FAKE + 2), EINVAL),
    (dict(count=None), EINVAL), (dict(count=FAKE + 2), EINVAL), (dict(status=FAKE + 2), EINVAL),
    (dict(start=FAKE, n_max=1021), EINVAL), (dict(struct=dict(head_dim=64)), EUNSUP),
    (dict(struct=dict(vexp=None)), EINVAL), (dict(t=8, struct=dict(n_seq=65535, n_kv_heads=65535)), EUNSUP)])
def test_accept(L, bad, rc):
    d = dict(k=FAKE, v=FAKE, t=4, start=FAKE * 2, path=None, count=FAKE, status=None, n_max=0, struct={})
    d.update(bad)
    c = _rows8(n_max=d["n_max"], **d["struct"])  # start = FAKE is seq_len itself
    assert L.bpkv_rows8_accept(ctypes.byref(c), _p(d["k"]), _p(d["v"]), d["t"], _p(d["start"]), _p(d["path"]),
                               _p(d["count"]), _p(d["status"]), None) == rc
    assert c.n_max == d["n_max"]


def test_accept_null(L):
    assert L.bpkv_rows8_accept(None, FAKE, FAKE, 1, FAKE, None, FAKE, None, None) == EINVAL


# ------------------------------------------------------------------ the Python helpers

N, H, G, T = 2, 3, 4, 10


def bf(*shape, **kw):
    return torch.zeros(shape, dtype=torch.bfloat16, **kw)


def prompt(**kw):
    d = dict(q=bf(T, H, G, D), out=bf(T, H, G, D), q_start=torch.zeros(N + 1, dtype=torch.int64), k=bf(T, H, D),
             v=bf(T, H, D))
    d.update(kw)
    return pk.prompt_args(**d)


def test_prompt_args_takes_what_fits():
    a = prompt()
    assert (a.n_seq, a.n_kv_heads, a.group, a.n_tokens, a.ld_q, a.ld_k, a.ld_v) == (N, H, G, T, H * G * D, H * D, H * D)
    qkv = bf(T, (G + 2) * H * D)  # heads of a fused projection in place
    a = prompt(q=qkv[:, :G * H * D].unflatten(1, (H, G, D)), v=qkv[:, (G + 1) * H * D:].unflatten(1, (H, D)))
    assert (a.ld_q, a.ld_k, a.ld_v) == ((G + 2) * H * D, H * D, (G + 2) * H * D)
    for k in (bf(T * H, D), bf(N, H, T // N, D)):
        a = prompt(k=k, v=k.clone())
        assert (a.ld_k, a.ld_v) == (0, 0) and a.k == k.data_ptr()
    one = bf(1, H * G * D + 8)[:, :H * G * D].unflatten(1, (H, G, D))  # one token's stride is nobody's
    a = prompt(q=one, out=bf(1, H, G, D), k=bf(1, H, D), v=bf(1, H, D))
    assert (a.ld_q, a.ld_k) == (H * G * D, H * D)
    for c in (pk.Rows8(N, H, G, 512, device="cpu"), pk.Cache(N, H, G, 512, device="cpu")):
        a = prompt(k=None, v=None, cache=c)
        assert bool(a.rows8) == isinstance(c, pk.Rows8) and bool(a.cache) == isinstance(c, pk.Cache) and not a.k


@pytest.mark.parametrize("kw", [
    dict(q=bf(T, H, G, D).float()), dict(q=bf(T, H, G, 2 * D)[..., :D]), dict(q=bf(T, G, H, D).transpose(1, 2)),
    dict(q=bf(T, H, G * D)), dict(q=bf(0, H, G, D)), dict(out=bf(T, H, G, D).float()), dict(out=bf(T - 1, H, G, D)),
    dict(out=bf(T, H, G, 2 * D)[..., :D]), dict(out=bf(T, H, G, D, device="meta")),
    dict(q_start=torch.zeros(N + 1, dtype=torch.int32)), dict(q_start=torch.zeros(0, dtype=torch.int64)),
    dict(q_start=torch.zeros((N + 1, 1), dtype=torch.int64)), dict(q_start=torch.zeros(2 * N + 2, dtype=torch.int64)[::2]),
    dict(q_start=torch.zeros(N + 1, dtype=torch.int64, device="meta")), dict(k=None), dict(v=None), dict(k=None, v=None),
    dict(k=bf(T, H, D).float()), dict(k=bf(T, H + 1, D)), dict(k=bf(H, T, D).transpose(0, 1)), dict(k=bf(T * H, D)),
    dict(v=bf(T, H, D, device="meta")), dict(k=bf(T * H - 1, D), v=bf(T * H, D)), dict(k=bf(N, H, 5, D), v=bf(N, H, 6, D)),
    dict(k=bf(3, H, 3, D), v=bf(3, H, 3, D), q_start=torch.zeros(4, dtype=torch.int64))])
def test_prompt_args_refuses_other_tensors(kw):
    with pytest.raises(ValueError):
        prompt(**kw)


def test_prompt_args_refuses_other_caches():
    for shape in ((N + 1, H, G), (N, H + 1, G), (N, H, G + 1)):
        with pytest.raises(ValueError):
            prompt(k=None, v=None, cache=pk.Rows8(*shape, 512, device="cpu"))
    c = pk.Rows8(N, H, G, 512, device="cpu")
    with pytest.raises(ValueError):
        prompt(cache=c)
    c.k8 = c.k8.to("meta")
    with pytest.raises(ValueError):
        prompt(k=None, v=None, cache=c)


@pytest.mark.parametrize("kw", [
    dict(k_new=bf(N, H, 5, D).float()), dict(v_new=bf(N, H, 6, D)), dict(k_new=bf(N, 5, H, D).transpose(1, 2)),
    dict(start=torch.zeros(N, dtype=torch.int32)), dict(start=torch.zeros(N + 1, dtype=torch.int64)),
    dict(count=torch.zeros(N, dtype=torch.int64)), dict(count=torch.zeros(2 * N, dtype=torch.int32)[::2]),
    dict(path=torch.zeros((N, 4), dtype=torch.int32)), dict(path=torch.zeros((N, 5), dtype=torch.int64)),
    dict(path=torch.zeros((N, 5), dtype=torch.int32, device="meta")), dict(status=torch.zeros(0, dtype=torch.int32))])
def test_accept_refuses_other_tensors(kw, monkeypatch):
    c = pk.Rows8(N, H, G, 512, device="cpu")
    calls = []
    monkeypatch.setattr(pk, "bpkv_rows8_accept", lambda *a: calls.append(a))
    d = dict(k_new=bf(N, H, 5, D), v_new=bf(N, H, 5, D), start=torch.zeros(N, dtype=torch.int64),
             count=torch.zeros(N, dtype=torch.int32), path=torch.zeros((N, 5), dtype=torch.int32))
    c.accept(**d, stream=0)
    c.accept(**{**d, "path": None}, stream=0)
    assert len(calls) == 2 and calls[0][3] == 5
    with pytest.raises(ValueError):
        c.accept(**{**d, **kw}, stream=0)
    assert len(calls) == 2
