"""Several new tokens of a sequence at once: what surrounds a call (streams,
graphs, other sequences, workspaces), and inputs at the ends of their ranges.
Bounds as in test_gpu_prompt."""
import math
import os
import subprocess
import sys

import pytest
import torch
from test_gpu_prompt import attention, causal, check, run_prompt, run_tree
from test_gpu_shared import draw_rows, make_cache, pk  # noqa: F401

pytestmark = pytest.mark.gpu
D = 128
BITS = [16, 8]


@pytest.mark.parametrize("rows", ["token", "seq"])
@pytest.mark.parametrize("new", [[70, 33, 129], [300, 1, 400], [20, 9, 30]])
def test_neighbours_that_hold_nan(pk, rows, new):
    """A sequence whose queries, keys and values are NaN or infinite says nothing about the others."""
    g = torch.Generator(device="cuda").manual_seed(4)
    H, G, T = 2, 4, sum(new)
    a0, a1 = new[0], new[0] + new[1]
    q = torch.randn((T, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (x[0] for x in draw_rows(g, 1, H, T))  # [H][T][D]
    q[a0:a1] = float("nan")
    k[:, a0:a1] = float("inf")
    v[:, a0:a1] = float("nan")
    out = torch.zeros_like(q)
    start = torch.tensor([0, a0, a1, T], device="cuda")
    if rows == "token":
        a = pk.prompt_args(q, out, start, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous())
    else:
        a = pk.prompt_args(q, out, start, *[torch.cat([x[:, i:j].reshape(-1, D) for i, j in ((0, a0), (a0, a1), (a1, T))])
                                            for x in (k, v)])
    ws = pk.prompt_workspace(a)
    pk.bpkv_prompt_attend(a, ws, ws.numel())
    for i, j in ((0, a0), (a1, T)):
        check(out[i:j], *attention(q[i:j], k[:, i:j], v[:, i:j], causal(j - i, j - i)))
    assert out[a0:a1].isnan().all() and pk.bpkv_read_status(ws) == 0


def test_starts_that_do_not_ascend(pk):
    """Values outside 0 .. T are taken as the nearest, and one below the last as that: rows of nobody stay."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for T in (90, 62):  # on the tensor cores, streamed
        starts_that_do_not_ascend(pk, g, T)


def starts_that_do_not_ascend(pk, g, T):
    H, G = 2, 2
    q = torch.randn((T, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (x[0].transpose(0, 1).contiguous() for x in draw_rows(g, 1, H, T))
    for start, parts in (([-7, 10, 4, 10 ** 12], [(0, 10), (10, T)]), ([5, 60, 0, 61], [(5, 60), (60, 61)]),
                         ([T, 3, 2, 1], []), ([1 << 62, -(1 << 62), 0, 5], [])):
        out = torch.full_like(q, 3.0)
        a = pk.prompt_args(q, out, torch.tensor(start, device="cuda"), k, v)
        ws = pk.prompt_workspace(a)
        pk.bpkv_prompt_attend(a, ws, ws.numel())
        nobody = torch.ones(T, dtype=torch.bool, device="cuda")
        for i, j in parts:
            check(out[i:j], *attention(q[i:j], k[i:j].transpose(0, 1), v[i:j].transpose(0, 1), causal(j - i, j - i)))
            nobody[i:j] = False
        assert (out[nobody] == 3.0).all() and pk.bpkv_read_status(ws) == 0


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t", [1, 8, 40])
def test_lengths_outside_the_cache(pk, bits, t):
    """Negative lengths are none, those past the capacity are the capacity."""
    got = run_tree(pk, bits, 3, t, 2, 4, [512, 512, 512], seed=t, tree="chain")
    c, want = got["c"], got["out"].clone()
    c.seq_len.copy_(torch.tensor([-5, 600, 1 << 40]))
    got["out"].fill_(7.0)
    got["fn"](c.c, t, None, got["q"], got["out"], got["ws"], got["ws"].numel())
    assert (got["out"][0] == 0).all() and torch.equal(got["out"][1:], want[1:])


@pytest.mark.parametrize("offset", [8, 16])
def test_outputs_on_16_bytes(pk, offset):
    """out starts on any 16-byte boundary."""
    for new in ([300, 5], [64], [1]):
        got = run_prompt(pk, "seq", new, None, 2, 4, seed=1)
        a = got["a"]
        n = got["out"].numel()
        flat = torch.full((n + 2 * offset,), 5.0, dtype=torch.bfloat16, device="cuda")
        a.out = flat.data_ptr() + 2 * offset
        pk.bpkv_prompt_attend(a, got["ws"], got["ws"].numel())
        assert torch.equal(flat[offset:offset + n].view_as(got["out"]), got["out"])
        assert (flat[:offset] == 5).all() and (flat[offset + n:] == 5).all()
    for bits in BITS:
        for t in (3, 60):
            got = run_tree(pk, bits, 2, t, 2, 4, [900, 4000])
            n = got["out"].numel()
            flat = torch.full((n + 2 * offset,), 5.0, dtype=torch.bfloat16, device="cuda")
            got["fn"](got["c"].c, t, got["mask"], got["q"], flat.data_ptr() + 2 * offset, got["ws"], got["ws"].numel())
            assert torch.equal(flat[offset:offset + n].view_as(got["out"]), got["out"])
            assert (flat[:offset] == 5).all() and (flat[offset + n:] == 5).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t,lens", [(2, [3000, 17]), (48, [9000, 300])])
def test_two_calls_at_once(pk, bits, t, lens):
    """Calls over the same cache on two streams, each with its own workspace, one of them replayed from a graph."""
    r = run_tree(pk, bits, 2, t, 2, 4, lens)
    outs = [torch.empty_like(r["out"]) for _ in range(2)]
    wss = [pk.tree_workspace(r["c"], t) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def call(i):
        r["fn"](r["c"].c, t, r["mask"], r["q"], outs[i], wss[i], wss[i].numel())

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


def test_calls_of_several_kinds_share_a_workspace(pk):
    """One after another on a stream: nothing is kept in it, and a captured prompt of other lengths is as good."""
    a = run_prompt(pk, "token", [2100, 40], None, 2, 4, seed=1)
    b = run_tree(pk, 16, 3, 64, 2, 4, [5000, 70, 64], seed=2)
    ws = torch.zeros(max(a["ws"].numel(), b["ws"].numel()), dtype=torch.uint8, device="cuda")
    want = [a["out"].clone(), b["out"].clone()]
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if i == 0:
                pk.bpkv_prompt_attend(a["a"], ws, ws.numel())
            else:
                b["fn"](b["c"].c, 64, b["mask"], b["q"], b["out"], ws, ws.numel())
        graphs.append(graph)
    for _ in range(3):
        for graph, out, w in zip(graphs, (a["out"], b["out"]), want):
            out.fill_(float("nan"))
            graph.replay()
            assert torch.equal(out, w)
    # other lengths, read on the device
    a["q_start"].copy_(torch.tensor([0, 1000, 2140]))
    graphs[0].replay()
    k, v = a["a"].keep[3], a["a"].keep[4]
    for i, j in ((0, 1000), (1000, 2140)):
        check(a["out"][i:j], *attention(a["q"][i:j], k[i:j].transpose(0, 1), v[i:j].transpose(0, 1), causal(j - i, j - i)))


def test_first_calls_captured(pk):
    """A process whose first call of each operator is a captured one."""
    code = """
import torch, bit_plane_kv_encode_gb300 as pk
N, H, G, t = 3, 2, 4, 5
c, big = pk.Rows8(N, H, G, 512), pk.Rows8(1, H, G, 65536)
for x in (c.k8, c.v8, big.k8, big.v8): x.fill_(0x38)
for x in (c.kexp, c.vexp, big.kexp, big.vexp): x.fill_(127)
big.seq_len.fill_(60000); big.c.n_max = 60000
k = torch.ones((N, H, t, 128), dtype=torch.bfloat16, device="cuda")
q = torch.ones((N, t, H, G, 128), dtype=torch.bfloat16, device="cuda"); out = torch.zeros_like(q)
far, far_out = torch.ones((1, 64, H, G, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 64, H, G, 128), dtype=torch.bfloat16, device="cuda")
flat, kv = q.view(N * t, H, G, 128), torch.ones((N * t * H, 128), dtype=torch.bfloat16, device="cuda")
a_out = torch.zeros_like(flat)
a = pk.prompt_args(flat, a_out, torch.arange(0, N * t + 1, t, device="cuda"), kv, kv)
w = [pk.prompt_workspace(a), pk.tree_workspace(c, t), pk.tree_workspace(big, 64)]
start, count = torch.full((N,), 9, device="cuda"), torch.full((N,), t, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.accept(k, k, start, count)
    pk.bpkv_tree_attend8(c.c, t, None, q, out, w[1], w[1].numel())
    pk.bpkv_tree_attend8(big.c, 64, None, far, far_out, w[2], w[2].numel())
    pk.bpkv_prompt_attend(a, w[0], w[0].numel())
for _ in range(3): g.replay()
torch.cuda.synchronize()
assert c.seq_len.tolist() == [9 + t] * N and all(pk.bpkv_read_status(x) == 0 for x in w)
assert (out == 1).all() and (far_out == 1).all() and (a_out == 1).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t", [2, 20, 64])
def test_maxima_that_rise(pk, bits, t):
    """Keys that grow along the rows: the running maximum moves at every tile, in every part of it."""
    g = torch.Generator(device="cuda").manual_seed(t)
    N, H, G, n = 1, 2, 4, 2500
    cap = 32768
    k, v = draw_rows(g, N, H, cap, 0.3, sink=False)
    k = (k.float() * (0.1 + 0.012 * torch.arange(cap, device="cuda"))[:, None]).to(torch.bfloat16)
    c, rows = make_cache(pk, bits, G, cap, [n], k, v)
    q = torch.randn((N, t, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = pk.tree_workspace(c, t)
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    for n_max in (n, 0, cap):
        c.c.n_max = n_max
        fn(c.c, t, None, q, out, ws, ws.numel())
        check(out[0], *attention(q[0], rows[0][0, :, :n], rows[1][0, :, :n], causal(t, n),
                                 None if bits == 16 else rows[2][0, :, :n]))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t", [2, 64])
def test_values_of_any_size(pk, bits, t):
    """Values (and 8-bit rows' scales) over the whole range, row by row."""
    g = torch.Generator(device="cuda").manual_seed(t)
    N, H, G, n, cap = 1, 2, 4, 700, 32768
    k, v = draw_rows(g, N, H, cap, 0.3, sink=False)
    v = (v.float() * torch.exp2(torch.randint(-30, 36, (N, H, cap, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    c, rows = make_cache(pk, bits, G, cap, [n], k, v)
    q = torch.randn((N, t, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = pk.tree_workspace(c, t)
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    for n_max in (n, cap):
        c.c.n_max = n_max
        fn(c.c, t, None, q, out, ws, ws.numel())
        check(out[0], *attention(q[0], rows[0][0, :, :n], rows[1][0, :, :n], causal(t, n),
                                 None if bits == 16 else rows[2][0, :, :n]))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t,n_max", [(1, 1900), (16, 1900), (64, 1900), (64, 32768)])
@pytest.mark.parametrize("rise", [[0, 15], [0, 15, 15, 30, 31, 62], [15, 0], [0, 5, 10, 15, 20]])
def test_values_near_the_bound(pk, bits, t, n_max, rise):
    """Values up to 2^80 under weights that are far above those of the first tile: logits rise by 1.02 `rise` powers of
    two, by which the sums may be above their size before they are taken back.  All is positive, so the output's error
    is that of its terms: a weight's rounding 2^-8, a sum of n 2^-23 n, the exponent's float32 2^-17 or less, the output
    2^-8."""
    g = torch.Generator(device="cuda").manual_seed(sum(rise))
    H, G, n, cap = 2, 4, 1900, 32768 if n_max > 2048 else 2048
    q = torch.ones((1, t, H, G, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    # rows in as many parts as there are in `rise`, the first of a tile
    part = torch.arange(cap, device="cuda").sub(128).clamp(min=-1).div(1800 / max(1, len(rise) - 1), rounding_mode="floor")
    part = (part + 1).clamp(0, len(rise) - 1).long()
    k = (torch.tensor(rise, device="cuda", dtype=torch.float32)[part] / 16)[None, None, :, None].expand(1, H, cap, D)
    v = ((torch.rand((1, H, cap, D), generator=g, device="cuda") + 1) * 2.0 ** 79).to(torch.bfloat16)
    c, (k64, v64, *_) = make_cache(pk, bits, G, cap, [n], k.to(torch.bfloat16), v)
    assert float(v64.abs().max()) <= 2.0 ** 80
    c.c.n_max = n_max
    ws = pk.tree_workspace(c, t)
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    fn(c.c, t, torch.zeros((1, t), dtype=torch.int64, device="cuda"), q, out, ws, ws.numel())
    torch.cuda.synchronize()
    assert pk.bpkv_read_status(ws) == 0
    w = torch.softmax(k64[0, :, :n - t].double().sum(-1) / math.sqrt(D), -1)
    want = torch.einsum("hn,hnd->hd", w, v64[0, :, :n - t].double())[None, None, :, None]
    err = ((out.double() - want).abs() / want).max()
    assert float(err) <= 2.0 ** -7 + n * 2.0 ** -23 + 2.0 ** -17, float(err)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t,n_max", [(1, 1900), (4, 1900), (16, 1900), (64, 1900), (64, 32768)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_logits(pk, bits, t, n_max, sign):
    """Logits of 2^14 to 2^28, of one sign: the rows whose keys have the largest share the weight evenly.  Weights are
    bf16 (2^-8; 8-bit rows where they are streamed: halves, whose base-2 exponent is a multiple of 2, 4, ... from 2^24 on, so that the
    output is only known to lie between the values it can take), a sum of n terms 2^-23 n, the output 2^-8."""
    g = torch.Generator(device="cuda").manual_seed(9)
    H, G, n, cap = 2, 4, 1900, 32768 if n_max > 2048 else 2048
    q = torch.full((1, t, H, G, D), float(sign), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    j = torch.arange(cap, device="cuda")
    step = torch.tensor([1.0, 1.125, 1.25], device="cuda")[j // 7 % 3]
    v = (torch.rand((1, H, cap, D), generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    best = (step[:n - t] == (1.25 if sign > 0 else 1.0)).double()
    mask = torch.zeros((1, t), dtype=torch.int64, device="cuda")  # the rows before the tree
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    for e in range(10, 25):
        k = (2.0 ** e * step)[None, None, :, None].expand(1, H, cap, D).to(torch.bfloat16)
        c, (_, v64, _) = make_cache(pk, bits, G, cap, [n], k, v)
        c.c.n_max = n_max
        ws = pk.tree_workspace(c, t)
        fn(c.c, t, mask, q, out, ws, ws.numel())
        assert pk.bpkv_read_status(ws) == 0
        mine = v64[0, :, :n - t]
        top = math.sqrt(D) * 2.0 ** e * 1.25 * math.log2(math.e)
        if bits == 16 or n_max > n or top < 2 ** 23:
            want = ((best[:, None] * mine).sum(1) / best.sum())[None, None, :, None]
            rel = (2.0 ** -8 if bits == 16 or n_max > n else 2.0 ** -11 + top * 2.0 ** -23) + n * 2.0 ** -23 + 2.0 ** -8
            err = (out.double() - want).abs() / want
            assert float(err.max()) <= rel, f"2^{e}: {float(err.max())}"
        else:
            few = mine[:, best > 0]
            lo, hi = few.amin(1)[None, None, :, None], few.amax(1)[None, None, :, None]
            assert ((out.double() >= lo * (1 - 2.0 ** -5)) & (out.double() <= hi * (1 + 2.0 ** -5))).all(), f"2^{e}"


@pytest.mark.parametrize("bits", BITS)
def test_many_sequences(pk, bits):
    """The largest batch, and one more is refused."""
    N = 512
    lens = [(37 * i) % 700 for i in range(N)]
    run_tree(pk, bits, N, 3, 1, 4, lens)  # streamed
    run_tree(pk, bits, N, 20, 1, 4, lens)  # tensor cores
    new = [(11 * i) % 40 for i in range(N)]
    run_prompt(pk, "token", new, None, 1, 4)
    run_prompt(pk, "cache", new, [(29 * i) % 300 for i in range(N)], 1, 4, bits=bits)
    c = (pk.Cache if bits == 16 else pk.Rows8)(513, 1, 1, 512)
    q = torch.zeros((513, 1, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    ws = pk.tree_workspace(c, 1)
    with pytest.raises(pk.BpkvError):
        (pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8)(c.c, 1, None, q, torch.zeros_like(q), ws, ws.numel())


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("t", [2, 64])
def test_rows_past_32_bits(pk, bits, t):
    """The last head of a cache whose rows pass 2^32 bytes."""
    cap, H, G = 262144, 66 if bits == 16 else 132, 1
    c = (pk.Cache if bits == 16 else pk.Rows8)(1, H, G, cap)
    g = torch.Generator(device="cuda").manual_seed(t)
    k, v = draw_rows(g, 1, 1, cap)
    part, rows = make_cache(pk, bits, G, cap, [cap], k, v)
    names = ("k_rows", "v_rows") if bits == 16 else ("k8", "v8", "kexp", "vexp")
    for name in names:
        getattr(c, name)[:, :-1].zero_()
        getattr(c, name)[:, -1:].copy_(getattr(part, name))
    assert getattr(c, names[0]).numel() * getattr(c, names[0]).element_size() > 1 << 32
    c.seq_len.fill_(cap)
    c.c.n_max = cap
    q = torch.randn((1, t, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = pk.tree_workspace(c, t)
    (pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8)(c.c, t, None, q, out, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    check(out[0, :, -1:], *attention(q[0, :, -1:], rows[0][0], rows[1][0], causal(t, cap), None if bits == 16 else rows[2][0]))
    assert (out[0, :, :-1] == 0).all()


@pytest.mark.parametrize("bits", BITS)
def test_drafting_loop(pk, bits):
    """A prompt, then rounds of drafted trees of which some tokens are kept, as a serving loop runs them: heads, rows,
    attention and acceptance together, each round's attention against the formula on the rows that the cache holds."""
    H, G, prompt, t, rounds, N, cap = 2, 4, 70, 12, 4, 3, 512
    g = torch.Generator(device="cuda").manual_seed(3)
    inv = (1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")

    def heads(n, pos):
        qkv = torch.randn((N, n, (G + 2) * H * D), generator=g, device="cuda").to(torch.bfloat16)
        q = torch.empty((N, n, H, G, D), dtype=torch.bfloat16, device="cuda")
        k = torch.empty((N, H, n, D), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, pos, inv, w, w, k_out=k, v_out=v))
        return q, k, v

    c = (pk.Cache if bits == 16 else pk.Rows8)(N, H, G, cap)

    def rows(n):
        if bits == 16:
            return c.k_rows[:, :, :n], c.v_rows[:, :, :n]
        return c.read(0, n)

    # the prompt: its attention over its own keys, as bpkv_qkv_rope leaves them
    q, k, v = heads(prompt, torch.zeros(N, dtype=torch.int64, device="cuda"))
    c.append(k, v)
    flat = q.view(N * prompt, H, G, D)
    out = torch.empty_like(flat)
    start = torch.arange(0, N * prompt + 1, prompt, device="cuda")
    a = pk.prompt_args(flat, out, start, k, v)
    ws = pk.prompt_workspace(a)
    pk.bpkv_prompt_attend(a, ws, ws.numel())
    for i in range(N):
        check(out[i * prompt:(i + 1) * prompt], *attention(q[i], k[i], v[i], causal(prompt, prompt)), f"prompt {i}")
    tw = pk.tree_workspace(c, t)
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    lens = [prompt] * N
    for r in range(rounds):
        at = torch.tensor(lens, device="cuda")
        q, k, v = heads(t, at)
        if bits == 8:
            c.append(k, v, at)
            c.n_max = max(lens) + t
        else:
            c.append(k, v)
        up = (torch.rand((N, t), generator=g, device="cuda") * torch.arange(t, device="cuda")).long().tolist()
        masks = [[0] * t for _ in range(N)]
        for i in range(N):
            for j in range(t):
                masks[i][j] = (masks[i][up[i][j]] if j else 0) | 1 << j
        mask = torch.tensor(masks, device="cuda")
        out = torch.empty_like(q)
        fn(c.c, t, mask, q, out, tw, tw.numel())
        for i in range(N):
            n = lens[i] + t
            kk, vv = rows(n)
            sees = torch.ones((t, n), dtype=torch.bool, device="cuda")
            sees[:, lens[i]:] = (mask[i][:, None] >> torch.arange(t, device="cuda")) & 1 > 0
            check(out[i], *attention(q[i], kk[i, :, :n], vv[i, :, :n], sees), f"round {r}, sequence {i}")
        # a way down each tree is kept, of another length for each sequence (bf16 rows: the first of them, as many for all)
        if bits == 8:
            ways = []
            for i in range(N):
                j, way = t - 1 - i, []
                while True:
                    way.insert(0, j)
                    if j == 0:
                        break
                    j = up[i][j]
                ways.append(way[:len(way) - (r + i) % 2])
            path = torch.zeros((N, t), dtype=torch.int32, device="cuda")
            for i, way in enumerate(ways):
                path[i, :len(way)] = torch.tensor(way, dtype=torch.int32)
            before = [x.clone() for x in c.read(0, max(lens) + t)]
            c.accept(k, v, at, torch.tensor([len(x) for x in ways], dtype=torch.int32, device="cuda"), path)
            for i, way in enumerate(ways):
                for x, old in zip(c.read(0, max(lens) + t), before):
                    assert torch.equal(x[i, :, :lens[i]], old[i, :, :lens[i]])
                    for j, node in enumerate(way):
                        assert torch.equal(x[i, :, lens[i] + j], old[i, :, lens[i] + node])
                lens[i] += len(way)
            c.n_max = max(lens)
        else:
            lens = [x + 3 for x in lens]
            c.seq_len.copy_(torch.tensor(lens))
            c.c.n_max = max(lens)
        assert c.seq_len.tolist() == lens and pk.bpkv_read_status(tw) == 0


def test_drafted_tokens_rolled_back(pk):
    """A Cache whose length is set back behind drafted tokens, and appended to again, holds what one does that never saw
    them: rows, planes and scales."""
    H, n, t, keep, more = 2, 100, 40, 3, 50
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = draw_rows(g, 1, H, n + t + more)
    c, want = pk.Cache(1, H, 4, 512), pk.Cache(1, H, 4, 512)
    c.append(k[:, :, :n].contiguous(), v[:, :, :n].contiguous())
    c.append(k[:, :, n:n + t].contiguous() * 8, v[:, :, n:n + t].contiguous())  # larger keys: other scales
    c.seq_len.fill_(n + keep)
    c.c.n_max = n + keep
    rest = [x[:, :, n + t:].contiguous() for x in (k, v)]
    c.append(*rest)
    want.append(torch.cat((k[:, :, :n], k[:, :, n:n + keep] * 8), 2), v[:, :, :n + keep].contiguous())
    want.append(*rest)
    end, nb = n + keep + more, (n + keep + more + 63) // 64
    assert c.seq_len.tolist() == want.seq_len.tolist() == [end]
    assert torch.equal(c.k_rows[:, :, :end], want.k_rows[:, :, :end]) and torch.equal(c.v_rows[:, :, :end], want.v_rows[:, :, :end])
    assert torch.equal(c.planes[..., :nb], want.planes[..., :nb]) and torch.equal(c.scales[..., :nb], want.scales[..., :nb])
