"""The 8-bit rows (bpkv_rows8_append, bpkv_rows8_read) and the projected heads
(bpkv_qkv_rope) against their definitions in 64 bits.

Row codes and scales are defined exactly (a power-of-two scale, one rounding
to nearest even), so they are compared bit for bit, and so is the read-back.
Projected heads: float32 arithmetic on bf16 inputs.  The mean square is a sum
of 128 positive terms (relative 130 2^-24 at most), its reciprocal root 2^-22,
the norm's products 2 2^-24, the rotation's angle 2^-22 (half turns to 2^-32
rounded to float32, sincospi 2^-23), its two products and sum 3 2^-24 of |a| +
|b|: together below 2^-17 (|a| + |b|).  A bf16 output adds 2^-8 of itself."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import bit_plane_kv_encode_gb300 as m
    return m


def code_of(x):
    """(codes, exponent bytes) of bf16 rows, by search over the definition in 64 bits."""
    xd = x.double()
    a = xd.abs().amax(-1)
    e = torch.full(a.shape, 32.0, dtype=torch.float64, device=x.device)
    for k in range(31, -49, -1):
        e = torch.where(a <= 448 * 2.0 ** k, float(k), e)
    y = (xd / torch.exp2(e)[..., None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)) + 1e-12) - 3)
    y = torch.round(y / step) * step  # half to even, as the last bit of y / step is the code's
    return y, (e + 127).to(torch.uint8)


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def rows(g, shape):
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=g, device="cuda").float())
    x[..., 0, :] = 0
    if shape[-2] > 1:
        x[..., 1, :64] *= 2.0 ** -14  # steps below the smallest normal code
    if shape[-2] > 3:
        x[..., 2, :] = x[..., 2, :].sign() * 448.0
        x[..., 3, :] *= 2.0 ** -60   # below the scales' range
    if shape[-2] > 4:
        x[..., 4, :] *= 2.0 ** 30  # above it: saturates
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("N,H,t", [(1, 1, 1), (3, 2, 5), (2, 3, 600), (32, 8, 1), (1, 5, 1023)])
def test_append_and_read(pk, N, H, t):
    g = torch.Generator(device="cuda").manual_seed(t)
    cap = (t + 700 + 511) // 512 * 512
    c = pk.Rows8(N, H, 4, cap)
    for x in (c.k8, c.v8, c.kexp, c.vexp):
        x.fill_(0x55)
    k, v = rows(g, (N, H, t, D)), rows(g, (N, H, t, D))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.arange(N, device="cuda") * 13 % 100
    c.append(k, v, start, status)
    assert c.seq_len.tolist() == (start + t).tolist() and not status.any()
    assert c.n_max == t
    for x, codes, exps in ((k, c.k8, c.kexp), (v, c.v8, c.vexp)):
        y, e = code_of(x)
        for i in range(N):
            s = int(start[i])
            assert torch.equal(values(codes[i, :, s:s + t]), y[i])
            assert torch.equal(exps[i, :, s:s + t], e[i])
            # rows around them are as they were
            assert (codes[i, :, :s] == 0x55).all() and (codes[i, :, s + t:] == 0x55).all()
            assert (exps[i, :, :s] == 0x55).all() and (exps[i, :, s + t:] == 0x55).all()
    c.c.n_max = cap
    t0, n = 3, min(cap - 3, t + 100)
    kr, vr = c.read(t0, n)
    for got, codes, exps in ((kr, c.k8, c.kexp), (vr, c.v8, c.vexp)):
        want = values(codes[:, :, t0:t0 + n]) * torch.exp2((exps[:, :, t0:t0 + n].double() - 127).clamp(-48, 32))[..., None]
        there = (torch.arange(t0, t0 + n, device="cuda") < c.seq_len[:, None])[:, None, :, None]
        assert torch.equal(got.double(), torch.where(there, want, 0.0))


def test_append_behind_the_rows_and_overflow(pk):
    g = torch.Generator(device="cuda").manual_seed(3)
    N, H, cap = 3, 2, 512
    c = pk.Rows8(N, H, 1, cap)
    k, v = rows(g, (N, H, 200, D)), rows(g, (N, H, 200, D))
    c.append(k, v)
    c.append(k, v)
    assert c.seq_len.tolist() == [400] * 3 and c.n_max == 400
    y, _ = code_of(k)
    assert torch.equal(values(c.k8[:, :, 200:400]), y)
    with pytest.raises(pk.BpkvError) as e:
        c.append(k, v)
    assert e.value.status == -1
    # a start out of range leaves that sequence alone and is flagged; the others are written
    before = c.k8.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(k, v, torch.tensor([100, 313, -1], device="cuda"), status)
    assert c.seq_len.tolist() == [300, 400, 400] and status.tolist() == [pk.DEV_OVERFLOW]
    assert torch.equal(c.k8[1:], before[1:]) and torch.equal(values(c.k8[0, :, 100:300]), y[0])


@pytest.mark.parametrize("N,H,t", [(1, 1, 64), (3, 8, 8), (5, 13, 5), (2, 64, 1), (3, 65, 1), (7, 16, 1), (7, 17, 1)])
def test_append_raises_the_lengths_once(pk, N, H, t):
    """Rows of a sequence up to a CTA's 64 and above; one sequence that is full keeps its rows and its length."""
    g = torch.Generator(device="cuda").manual_seed(21)
    c = pk.Rows8(N, H, 2, 512)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([0 if i else 512 - t + 1 for i in range(N)], device="cuda")
    c.seq_len.copy_(lens)
    for x in (c.k8, c.v8):
        x.zero_()
    c.kexp.fill_(127)
    c.vexp.fill_(127)
    want = [torch.zeros((N, H, 512, D), dtype=torch.float64, device="cuda") for _ in range(2)]
    for step in range(3):
        kv = [torch.randn((N, H, t, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
        c.c.n_max = 0
        pk.bpkv_rows8_append(c.c, kv[0], kv[1], t, None, status)
        for i in range(1, N):
            for w, x in zip(want, kv):
                w[i, :, step * t:(step + 1) * t] = x[i].double()
    assert int(status) == pk.DEV_OVERFLOW
    lens[1:] = 3 * t
    assert torch.equal(c.seq_len, lens)
    c.seq_len.fill_(512)
    for got, w in zip(c.read(0, 512), want):
        # e4m3 after a scale that puts the row's largest at 224 or above: half a step is 2^-4 of a value, or 2^-10
        assert ((got.double() - w).abs() <= 2.0 ** -4 * w.abs() + 2.0 ** -10 * w.abs().amax(-1, keepdim=True) / 224).all()


@pytest.mark.parametrize("N,H,G", [(3, 8, 4), (2, 12, 2), (2, 7, 5), (700, 8, 5), (300, 2, 8)])
def test_qkv_raises_the_lengths_once(pk, N, H, G):
    """A token behind the stored ones, positions from the lengths: one CTA a token, several, and one by many tokens."""
    g = torch.Generator(device="cuda").manual_seed(22)
    c, d = pk.Rows8(N, H, G, 512), pk.Rows8(N, H, G, 512)
    start = torch.arange(N, device="cuda") * 7 % 513
    for x in (c, d):
        for y in (x.k8, x.v8, x.kexp, x.vexp):
            y.zero_()
        x.seq_len.copy_(start)
    inv = torch.logspace(0, -4, 64, device="cuda")
    pos = start.clone()
    for _ in range(2):
        qkv = torch.randn((N, 1, (G + 2) * H * D), generator=g, device="cuda").to(torch.bfloat16)
        q1, q2 = [torch.empty((N, 1, H, G, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for x, q, p in ((c, q1, None), (d, q2, pos)):
            x.c.n_max = 0
            pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, p, inv, rows8=x, status=status))
        pos = torch.where(pos < 512, pos + 1, pos)
        assert torch.equal(q1, q2)
    for a, b in ((c.k8, d.k8), (c.v8, d.v8), (c.kexp, d.kexp), (c.vexp, d.vexp), (c.seq_len, pos), (d.seq_len, pos)):
        assert torch.equal(a, b)


def test_captured_append(pk):
    g = torch.Generator(device="cuda").manual_seed(4)
    N, H = 2, 2
    c = pk.Rows8(N, H, 1, 512)
    k, v = rows(g, (N, H, 1, D)), rows(g, (N, H, 1, D))
    c.append(k, v)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        c.append(k, v)
    for _ in range(5):
        gr.replay()
    torch.cuda.synchronize()
    assert c.seq_len.tolist() == [6, 6]
    assert torch.equal(c.k8[:, :, 5], c.k8[:, :, 0])


def qkv_reference(qkv, N, t, H, G, pos, inv_freq, qw, kw, eps, pairs):
    """q, k, v in 64 bits and the scale of their float32 errors."""
    x = qkv[..., :(G + 2) * H * D].double().reshape(N, t, (G + 2) * H, D)
    rot = 2 * inv_freq.numel()
    u = (pos[:, None] + torch.arange(t, device="cuda")).double()[..., None] * inv_freq.double()
    cos, sin = u.cos()[:, :, None], u.sin()[:, :, None]

    def head(z, w):
        if w is not None:
            z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        scale = z.abs().clone()
        ia = torch.arange(0, rot, 2, device="cuda") if pairs else torch.arange(rot // 2, device="cuda")
        ib = ia + 1 if pairs else ia + rot // 2
        a, b = z[..., ia], z[..., ib]
        y = z.clone()
        y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
        scale[..., ia] = scale[..., ib] = a.abs() + b.abs()
        return y, scale * 2.0 ** -17

    q, qt = head(x[:, :, :G * H], qw)
    k, kt = head(x[:, :, G * H:(G + 1) * H], kw)
    q, qt = q.reshape(N, t, H, G, D), qt.reshape(N, t, H, G, D)
    return (q, qt), (k.transpose(1, 2), kt.transpose(1, 2)), x[:, :, (G + 1) * H:].transpose(1, 2)


def check(got, want, tol):
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((got.double() - want).abs() <= tol + 1e-30).all(), float(((got.double() - want).abs() / (tol + 1e-30)).max())


@pytest.mark.parametrize("rot,pairs", [(128, False), (128, True), (64, False), (66, False), (2, False), (34, True),
                                       (16, False), (48, False), (0, False)])
@pytest.mark.parametrize("N,t,H,G", [(1, 1, 8, 4), (3, 7, 2, 3), (2, 700, 1, 1)])
def test_qkv(pk, rot, pairs, N, t, H, G):
    g = torch.Generator(device="cuda").manual_seed(rot + t)
    ld = (G + 2) * H * D + 8 * (rot % 3)
    qkv = (2 * torch.randn((N, t, ld), generator=g, device="cuda")).to(torch.bfloat16)
    qkv[0, 0, :D] = 0
    pos = torch.tensor([1000003, 0, 77][:N], device="cuda")
    inv = (5e5 ** (-torch.arange(0, rot, 2, device="cuda").double() / max(rot, 1))).float()
    qw = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")) if rot != 64 else None
    kw = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")) if rot != 66 else None
    for qdt in (torch.float32, torch.bfloat16):
        q = torch.full((N, t, H, G, D), float("nan"), dtype=qdt, device="cuda")
        k = torch.full((N, H, t, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, float("nan"))
        pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, pos=pos, inv_freq=inv, q_weight=qw, k_weight=kw, eps=1e-6, pairs=pairs,
                                     k_out=k, v_out=v))
        (wq, tq), (wk, tk), wv = qkv_reference(qkv, N, t, H, G, pos, inv, qw, kw, 1e-6, pairs)
        check(q, wq, tq)
        check(k, wk, tk)
        assert torch.equal(v.double(), wv)


@pytest.mark.parametrize("N,t", [(1, 1), (32, 1), (3, 200)])
@pytest.mark.parametrize("behind", [False, True])
def test_qkv_into_rows8_is_the_two_calls(pk, N, t, behind):
    g = torch.Generator(device="cuda").manual_seed(N)
    H, G, cap = 3, 4, 1024
    qkv = torch.randn((N, t, (G + 2) * H * D), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(N, device="cuda") * 11 % 300
    inv = (1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    caches, outs = [], []
    for fused in (True, False):
        c = pk.Rows8(N, H, G, cap)
        for x in (c.k8, c.v8, c.kexp, c.vexp):
            x.zero_()
        c.seq_len.copy_(pos)
        c.c.n_max = 300
        q = torch.empty((N, t, H, G, D), dtype=torch.bfloat16, device="cuda")
        k = torch.empty((N, H, t, D), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        at = c.seq_len if behind else pos
        a = pk.qkv_args(qkv, q, H, pos=at, inv_freq=inv, q_weight=w, k_weight=w, k_out=k, v_out=v,
                        rows8=c if fused else None)
        pk.bpkv_qkv_rope(a)
        if not fused:
            c.append(k, v, None if behind else pos)
        assert c.seq_len.tolist() == (pos + t).tolist() and c.n_max == 300 + t
        caches.append(c)
        outs.append((q, k, v))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    a, b = caches
    for x, y in ((a.k8, b.k8), (a.v8, b.v8), (a.kexp, b.kexp), (a.vexp, b.vexp)):
        assert torch.equal(x, y)
