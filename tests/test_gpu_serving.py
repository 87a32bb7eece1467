"""The serving operators together, as a decode loop uses them: projected heads
go through bpkv_qkv_rope into a cache, and bpkv_shared_attend(8) reads it beside
a shared prefix, step after step; every step's output is checked against the
formula in 64 bits on the rows that the cache should hold."""
import pytest
import torch

from test_gpu_shared import D, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import bit_plane_kv_encode_gb300 as m
    return m


def heads(qkv, N, t, H, G, pos, inv, w, eps):
    """Normed and rotated queries and keys, and values, in 64 bits."""
    x = qkv.double().reshape(N, t, (G + 2) * H, D)
    u = (pos[:, None] + torch.arange(t, device="cuda")).double()[..., None] * inv.double()
    cos, sin = u.cos()[:, :, None], u.sin()[:, :, None]

    def head(z):
        z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        a, b = z[..., :D // 2], z[..., D // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    return (head(x[:, :, :G * H]).reshape(N, t, H, G, D), head(x[:, :, G * H:(G + 1) * H]).transpose(1, 2),
            x[:, :, (G + 1) * H:].transpose(1, 2))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("N,captured", [(3, False), (40, True)])
def test_decode_loop(pk, bits, N, captured):
    H, G, prompt, plen, steps, cap = 2, 4, 37, 300, 4, 512
    g = torch.Generator(device="cuda").manual_seed(11)
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    inv = (1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    row = (G + 2) * H * D

    def draw(n, t):
        return (1.5 * torch.randn((n, t, row), generator=g, device="cuda")).to(torch.bfloat16)

    if bits == 8:
        prefix, cache = pk.Rows8(1, H, G, cap), pk.Rows8(N, H, G, cap)
    else:
        prefix, cache = pk.Cache(1, H, G, cap), pk.Cache(N, H, G, cap)

    def fill(c, qkv, t, at, q):
        """qkv's keys and values behind the cache's rows: straight into 8-bit rows, through encode_append else."""
        n = qkv.shape[0]
        if bits == 8:
            pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, inv_freq=inv, q_weight=w, k_weight=w, rows8=c))
        else:
            k = torch.empty((n, H, t, D), dtype=torch.bfloat16, device="cuda")
            v = torch.empty_like(k)
            pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, pos=at, inv_freq=inv, q_weight=w, k_weight=w, k_out=k, v_out=v))
            c.append(k, v)

    def queries(n, t):
        return torch.empty((n, t, H, G, D), dtype=torch.bfloat16, device="cuda")

    # the shared prefix, then each session's own prompt behind it: positions go on from the prefix
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    base = torch.full((N,), plen, dtype=torch.int64, device="cuda")
    xp, xs = draw(1, plen), draw(N, prompt)
    fill(prefix, xp, plen, zero, queries(1, plen))
    if bits == 8:  # its positions are not the rows it fills: two calls
        k = torch.empty((N, H, prompt, D), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        pk.bpkv_qkv_rope(pk.qkv_args(xs, queries(N, prompt), H, pos=base, inv_freq=inv, q_weight=w, k_weight=w, k_out=k,
                                     v_out=v))
        cache.append(k, v)
    else:
        fill(cache, xs, prompt, base, queries(N, prompt))
    assert prefix.seq_len.tolist() == [plen] and cache.seq_len.tolist() == [prompt] * N

    ws = pk.shared_workspace(cache, prefix)
    qkv, q = draw(N, 1), queries(N, 1)
    kn = torch.empty((N, H, 1, D), dtype=torch.bfloat16, device="cuda")
    vn, out, pos = torch.empty_like(kn), torch.empty((N, H, G, D), dtype=torch.bfloat16, device="cuda"), base + prompt
    args = pk.qkv_args(qkv, q, H, pos=pos, inv_freq=inv, q_weight=w, k_weight=w, k_out=kn, v_out=vn)

    def step():
        pk.bpkv_qkv_rope(args)
        cache.append(kn, vn)
        (pk.bpkv_shared_attend8 if bits == 8 else pk.bpkv_shared_attend)(prefix.c, None, cache.c, q[:, 0], out, ws,
                                                                        ws.numel())
        pos.add_(1)

    def held(c):
        """The rows as the cache holds them, in 64 bits (and the scales of 8-bit values)."""
        if bits == 16:
            return c.k_rows.double(), c.v_rows.double(), None
        x = [codes.view(torch.float8_e4m3fn).double() * torch.exp2(e.double() - 127)[..., None]
             for codes, e in ((c.k8, c.kexp), (c.v8, c.vexp))]
        return (*x, torch.exp2(c.vexp.double() - 127))

    def check_rows(got, qkv, at, first):
        """Rows of new tokens against the formula.  bf16: 2^-8 of the value; 8-bit rows: the code's 2^-4 besides, or
        half a step of the smallest code, 2^-10 under a scale of at most max |x| / 224; float32 before it: 2^-17 of
        |a| + |b| <= 2 max |x|."""
        t = qkv.shape[1]
        for x, want in zip(got[:2], heads(qkv, qkv.shape[0], t, H, G, at, inv, w, 1e-6)[1:]):
            top = want.abs().amax(-1, keepdim=True)
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -16 * top
            if bits == 8:
                tol = tol + 2.0 ** -4 * 1.01 * want.abs() + 2.0 ** -10 / 224 * 1.01 * top
            assert ((x[:, :, first:first + t] - want).abs() <= tol).all()

    graph = None
    prows = held(prefix)
    check_rows(prows, xp, zero, 0)
    check_rows(held(cache), xs, base, 0)
    for i in range(steps):
        qkv.copy_(draw(N, 1))
        want_q, _, _ = heads(qkv, N, 1, H, G, base + prompt + i, inv, w, 1e-6)
        if captured and i == 1:
            graph = torch.cuda.CUDAGraph()
            before = (cache.seq_len.clone(), pos.clone())
            with torch.cuda.graph(graph):
                step()
            assert torch.equal(before[0], cache.seq_len) and torch.equal(before[1], pos)
        if graph is not None:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert pk.bpkv_read_status(ws) == 0
        n = prompt + i + 1
        assert cache.seq_len.tolist() == [n] * N
        mine = held(cache)
        check_rows(mine, qkv, base + prompt + i, n - 1)
        o, tol = reference(q[:, 0], mine, [n] * N, prows, [plen], [0] * N, bits)
        assert ((out.double() - o).abs() <= tol).all()
        assert ((q[:, 0].double() - want_q[:, 0]).abs() <= 2.0 ** -8 * want_q[:, 0].abs() + 2.0 ** -14).all()


@pytest.mark.parametrize("bits", [16, 8])
def test_two_calls_at_once(pk, bits):
    """Calls over the same caches on two streams, each with its own workspace, one of them replayed from a graph."""
    from test_gpu_shared import run_case
    r = run_case(pk, bits, 40, 2, 4, [(37 * i) % 300 for i in range(40)], [3001, 70], [i % 3 for i in range(40)],
                 bound=65536)
    outs = [torch.empty_like(r["out"]) for _ in range(2)]
    wss = [pk.shared_workspace(r["c"], r["pc"]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def call(i):
        r["fn"](r["pc"].c, r["of"], r["c"].c, r["q"], outs[i], wss[i], wss[i].numel())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(0)
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            call(1)
    torch.cuda.synchronize()
    for out, ws in zip(outs, wss):
        assert torch.equal(out, r["out"]) and pk.bpkv_read_status(ws) == 0


def test_first_calls_captured(pk):
    """A process whose first call of each operator is a captured one."""
    import subprocess
    import sys
    code = """
import torch, bit_plane_kv_encode_gb300 as pk
N, H, G = 40, 2, 4
c, p = pk.Rows8(N, H, G, 512), pk.Rows8(1, H, G, 65536)
for x in (c.k8, c.v8, p.k8, p.v8): x.fill_(0x38)
for x in (c.kexp, c.vexp, p.kexp, p.vexp): x.fill_(127)
p.seq_len.fill_(5000); p.c.n_max = 65536
ws = pk.shared_workspace(c, p)
qkv = torch.ones((N, 1, (G + 2) * H * 128), dtype=torch.bfloat16, device="cuda")
q = torch.empty((N, 1, H, G, 128), dtype=torch.bfloat16, device="cuda"); out = torch.empty_like(q)
a = pk.qkv_args(qkv, q, H, rows8=c)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pk.bpkv_qkv_rope(a)
    pk.bpkv_shared_attend8(p.c, None, c.c, q, out, ws, ws.numel())
for _ in range(3): g.replay()
torch.cuda.synchronize()
assert c.seq_len.tolist() == [3] * N and pk.bpkv_read_status(ws) == 0
assert (out == 1).all()
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("bits", [16, 8])
def test_host_bound_below_the_lengths(pk, bits):
    """n_max only sizes the launch: lengths it does not know of (a replayed graph's) are still attended to in full."""
    from test_gpu_shared import run_case
    r = run_case(pk, bits, 9, 2, 4, [700] * 9, [900], [0] * 9, given=False)
    first = r["out"].clone()
    for c in (r["c"], r["pc"]):
        c.c.n_max = 0
    r["out"].zero_()
    r["fn"](r["pc"].c, None, r["c"].c, r["q"], r["out"], r["ws"], r["ws"].numel())
    assert ((r["out"].double() - r["want"]).abs() <= r["tol"]).all()
    assert first.shape == r["out"].shape


def test_many_sequences_and_prefixes(pk):
    """The largest batch: 512 sequences over 512 prefixes in an order of their own, and one more is refused."""
    from test_gpu_shared import run_case
    N = 512
    of = [(i * 37) % N for i in range(N)]
    run_case(pk, 16, N, 1, 2, [(i * 7) % 90 for i in range(N)], [(i * 5) % 200 for i in range(N)], of)
    run_case(pk, 8, N, 1, 8, [(i * 7) % 90 for i in range(N)], [3001], [0] * N, given=False)
    big = pk.Rows8(513, 1, 1, 512)
    with pytest.raises(pk.BpkvError):
        pk.shared_workspace(big)
