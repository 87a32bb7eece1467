"""What the Python helpers for several new tokens of a sequence make of tensors
whose strides or types the kernels would read as something else (no GPU)."""
import pytest
import torch

import bit_plane_kv_encode_gb300 as pk

N, H, G, T, D = 2, 3, 4, 10, 128


def bf(*shape, **kw):
    return torch.zeros(shape, dtype=torch.bfloat16, **kw)


def prompt(**kw):
    d = dict(q=bf(T, H, G, D), out=bf(T, H, G, D), q_start=torch.zeros(N + 1, dtype=torch.int64), k=bf(T, H, D),
             v=bf(T, H, D))
    d.update(kw)
    return pk.prompt_args(**d)


def one_for_all(*shape):
    """One token's heads as those of T tokens: a stride of 0, which in the struct says another layout."""
    return bf(1, *shape).expand(T, *shape)


def tokens(stride, *shape):
    """T tokens of dense heads, `stride` elements apart."""
    n = torch.Size(shape).numel()
    dense = tuple(torch.empty(shape).stride())
    return torch.as_strided(bf((T - 1) * stride + n), (T, *shape), (stride, *dense))


@pytest.mark.parametrize("kw", [
    dict(k=one_for_all(H, D), v=one_for_all(H, D)), dict(k=one_for_all(H, D)), dict(v=one_for_all(H, D)),
    dict(q=one_for_all(H, G, D)), dict(k=tokens(H * D - 8, H, D), v=tokens(H * D - 8, H, D)), dict(k=tokens(8, H, D)),
    dict(v=tokens(H * D + 4, H, D)), dict(q=tokens(D, H, G, D)), dict(q=tokens(H * G * D + 2, H, G, D))])
def test_tokens_that_overlap_or_lie_between_boundaries(kw):
    with pytest.raises(ValueError):
        prompt(**kw)


def test_what_the_strides_read_is_there():
    """Of a struct that is made, every element that the call may read lies in the tensor's storage."""
    for k in (bf(T, H, D), tokens(H * D + 8, H, D), bf(T, 2 * H, D)[:, H:], bf(T * H, D), bf(N, H, T // N, D)):
        a = prompt(k=k, v=k.clone() if k.is_contiguous() else k)
        ld = a.ld_k or H * D
        end = k.storage_offset() + (T - 1) * ld + H * D
        assert end * 2 <= k.untyped_storage().nbytes() and (a.ld_k == 0) == (k.dim() != 3)


def test_one_token_has_no_stride():
    one = bf(1, H, D).expand(1, H, D)
    a = prompt(q=bf(1, H, G, D), out=bf(1, H, G, D), k=one, v=one)
    assert (a.ld_q, a.ld_k, a.ld_v) == (H * G * D, H * D, H * D)


@pytest.mark.parametrize("shift", [-1, 1])
def test_accept_refuses_starts_that_share_some_of_the_lengths(shift):
    """Starts that are the lengths are read before these are set; those that lie one beside them would not be."""
    from bit_plane_kv_encode_gb300 import build
    build.build()
    base, far = 1 << 40, 1 << 36  # aligned, never read
    c = pk.bpkv_rows8(N, H, G, D, 512, 0, base, base + far, base + 2 * far, base + 3 * far, base + 4 * far)
    with pytest.raises(pk.BpkvError) as e:
        pk.bpkv_rows8_accept(c, base + 5 * far, base + 6 * far, 4, base + 4 * far + 8 * shift, None, base + 7 * far,
                             stream=0)
    assert e.value.status == -1 and c.n_max == 0


@pytest.mark.parametrize("make", [pk.Cache, pk.Rows8])
def test_the_bound_of_the_lengths_can_be_set(make):
    c = make(N, H, G, 512, device="cpu")
    for n in (512, 0, 77):
        c.n_max = n
        assert c.n_max == c.c.n_max == n
    for n in (-1, 513):
        with pytest.raises(ValueError):
            c.n_max = n
    assert c.n_max == 77


# ------------------------------------------------------------------ trees

t = 5


def tree_call(monkeypatch, make, **kw):
    """What tree_attend passes on, by the name of the call."""
    calls = []
    for name in ("bpkv_tree_attend", "bpkv_tree_attend8"):
        monkeypatch.setattr(pk, name, lambda *a, name=name: calls.append((name, a)))
    d = dict(q=bf(N, t, H, G, D), out=bf(N, t, H, G, D), tree=torch.zeros((N, t), dtype=torch.int64),
             ws=torch.zeros(1024, dtype=torch.uint8))
    d.update(kw)
    cache = make(N, H, G, 512, device="cpu")
    pk.tree_attend(cache, d["q"], d["out"], d["ws"], d["tree"], stream=0)
    (name, a), = calls
    assert a[0] is cache.c and a[1] == t and a[2] is d["tree"] and a[3] is d["q"] and a[4] is d["out"] and a[5] is d["ws"]
    assert a[6] == d["ws"].numel() * d["ws"].element_size() and a[7] == 0
    return name


@pytest.mark.parametrize("make,name", [(pk.Cache, "bpkv_tree_attend"), (pk.Rows8, "bpkv_tree_attend8")])
def test_tree_attend_takes_what_fits(monkeypatch, make, name):
    for tree in (torch.zeros((N, t), dtype=torch.int64), torch.zeros((N, t), dtype=torch.uint64), None):
        assert tree_call(monkeypatch, make, tree=tree) == name
    assert tree_call(monkeypatch, make, ws=torch.zeros(128, dtype=torch.int64)) == name


@pytest.mark.parametrize("make", [pk.Cache, pk.Rows8])
@pytest.mark.parametrize("kw", [
    dict(q=bf(N, t, H, G, D).float()), dict(q=bf(N, t, G, H, D).transpose(2, 3)), dict(q=bf(N * t, H, G, D)),
    dict(q=bf(N, 2 * t, H, G, D)[:, ::2]), dict(q=bf(N + 1, t, H, G, D)), dict(q=bf(N, t, H, G, D, device="meta")),
    dict(out=bf(N, t, H, G, D).float()), dict(out=bf(N, t + 1, H, G, D)), dict(out=bf(N, t, H, G, 2 * D)[..., :D]),
    dict(tree=torch.zeros((N, t), dtype=torch.int32)), dict(tree=torch.zeros((N, t, t), dtype=torch.bool)),
    dict(tree=torch.zeros((t, N), dtype=torch.int64).T), dict(tree=torch.zeros((N, 64), dtype=torch.int64)),
    dict(tree=torch.zeros((N, t), dtype=torch.int64, device="meta")), dict(ws=torch.zeros(1024, device="meta")),
    dict(ws=torch.zeros(2048, dtype=torch.uint8)[::2])])
def test_tree_attend_refuses_other_tensors(monkeypatch, make, kw):
    with pytest.raises(ValueError):
        tree_call(monkeypatch, make, **kw)
