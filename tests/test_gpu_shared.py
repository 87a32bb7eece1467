"""Decode attention over shared prefixes (bpkv_shared_attend over bf16 rows,
bpkv_shared_attend8 over 8-bit rows) against the formula in 64 bits.

Bounds.  With p the exact softmax weights, A = sum p |v| and o = sum p v:
  - weights enter the product rounded: bf16 by at most 2^-8 of themselves (half
    of finfo.eps); two e5m2 pieces by 2^-3 of the 2^-3 that the first leaves,
    2^-6, after a half's 2^-11.  Their unit is set by the largest p 2^e (e: the
    row's scale exponent), which they hold as 2^11 or more; the smallest step is
    2^-16, so a token's code (at most 448) loses half of that at most: together
    n 448 2^-17 2^-11 < n 2^-19 of the largest p 2^e.  A row of zeros counts here
    too, with its 2^-48: what lies 67 binary orders below it is lost;
  - logits are float32 sums of 128 products, off by B <= 130 2^-24 sum_j |q_j k_j|
    / sqrt(D) at most (8-bit rows: q is off by 2^-16 of its largest channel
    besides), which moves a weight by B and the sum by B: 2 B A;
  - sums over n tokens in float32, n 2^-23 A; exp2 2^-21;
  - the output is bf16: 2^-8 |o|."""
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


def quantise(x):
    """Rows as the 8-bit cache holds them: codes, exponent bytes and the values they stand for."""
    xf = x.double()
    a = xf.abs().amax(-1)
    m, e = torch.frexp(a)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-48, 32)
    e = torch.where(a > 0, e, torch.full_like(e, -48))
    c = (xf * torch.exp2(-e.double())[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return c.view(torch.uint8), (e + 127).to(torch.uint8), c.double() * torch.exp2(e.double())[..., None]


def make_cache(pk, bits, G, cap, lens, k, v):
    """A cache of len(lens) sequences and its rows in 64 bits; rows past the lengths hold NaN."""
    N = len(lens)
    H = k.shape[1]
    if bits == 16:
        c = pk.Cache(N, H, G, cap)
        c.k_rows.copy_(k)
        c.v_rows.copy_(v)
        rows = (k.double(), v.double(), None)
    else:
        c = pk.Rows8(N, H, G, cap)
        vals = []
        for x, codes, exps in ((k, c.k8, c.kexp), (v, c.v8, c.vexp)):
            q, e, val = quantise(x)
            codes.copy_(q)
            exps.copy_(e)
            vals.append(val)
        rows = (*vals, torch.exp2(c.vexp.double() - 127))
    for i, n in enumerate(lens):
        if bits == 16:
            c.k_rows[i, :, n:] = float("nan")
            c.v_rows[i, :, n:] = float("nan")
        else:
            for x in (c.k8, c.v8):
                x[i, :, n:] = 0x7f  # NaN
            for x in (c.kexp, c.vexp):
                x[i, :, n:] = 255
    c.seq_len.copy_(torch.tensor(lens))
    c.c.n_max = max(lens)
    return c, rows


def draw_rows(g, N, H, cap, spread=0.75, sink=True):
    k = torch.randn((N, H, cap, D), generator=g, device="cuda")
    k *= torch.exp(spread * torch.randn((N, H, 1, D), generator=g, device="cuda"))
    v = torch.randn((N, H, cap, D), generator=g, device="cuda")
    # rows of very different size, as the scales of 8-bit rows must carry
    v *= torch.exp2(torch.randint(-6, 5, (N, H, cap, 1), generator=g, device="cuda").float())
    if sink:
        k[:, :, 0] *= 3
        v[:, :, 0] = 0
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def reference(q, rows, lens, prows, plens, prefix_of, bits):
    """(o, bound) in 64 bits."""
    N, H, G, _ = q.shape
    o = torch.zeros((N, H, G, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    for i in range(N):
        p = prefix_of[i]
        k, v, s = [None if r is None else r[i, :, :lens[i]] for r in rows]
        if prows is not None and 0 <= p < len(plens):
            pk, pv, ps = [None if r is None else r[p, :, :plens[p]] for r in prows]
            k, v, s = torch.cat((pk, k), 1), torch.cat((pv, v), 1), None if s is None else torch.cat((ps, s), 1)
        n = k.shape[1]
        if n == 0:
            continue
        qd = q[i].double()
        x = qd @ k.transpose(-1, -2) / math.sqrt(D)
        w = torch.softmax(x, -1)
        o[i] = w @ v
        A = w @ v.abs()
        B = 130 * 2.0 ** -24 * (qd.abs() @ k.abs().transpose(-1, -2)).amax(-1) / math.sqrt(D)
        if bits == 16:
            w_off = 2.0 ** -8
            floor = 0.0
        else:
            w_off = 2.0 ** -6 + 2.0 ** -11
            B = B + 2.0 ** -16 * qd.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None] / math.sqrt(D)
            floor = n * 2.0 ** -19 * (w * s[:, None]).amax(-1)[..., None]
        tol[i] = (w_off + 2 * B[..., None] + n * 2.0 ** -23 + 2.0 ** -21) * A + 2.0 ** -8 * o[i].abs() + floor
    return o, tol + 1e-30


def run_case(pk, bits, N, H, G, lens, plens, prefix_of, seed=1, spread=0.75, sink=True, given=True, bound=None):
    """One call against the formula.  bound: what the host knows of the prefixes' lengths (a cache of that size), which
    decides whether a CTA takes each sequence with its prefix (none given and short), they are streamed by 16 query rows
    (3000) or taken by the tensor cores (65536)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cap = max(512, (max(lens) + 511) // 512 * 512)
    q = torch.randn((N, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = draw_rows(g, N, H, cap, spread, sink)
    c, rows = make_cache(pk, bits, G, cap, lens, k, v)
    pc, prows = None, None
    if plens:
        pcap = max(512, ((bound or max(plens)) + 511) // 512 * 512)
        k, v = draw_rows(g, len(plens), H, pcap, spread, sink)
        pc, prows = make_cache(pk, bits, G, pcap, plens, k, v)
        pc.c.n_max = bound or max(plens)
    ws = pk.shared_workspace(c, pc)
    out = torch.full((N, H, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    of = torch.tensor(prefix_of, dtype=torch.int32, device="cuda") if given else None
    fn = pk.bpkv_shared_attend if bits == 16 else pk.bpkv_shared_attend8
    fn(pc.c if pc else None, of, c.c, q, out, ws, ws.numel())
    torch.cuda.synchronize()
    assert pk.bpkv_read_status(ws) == 0
    want, tol = reference(q, rows, lens, prows, plens, prefix_of, bits)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    worst = float((err / tol).max())
    assert worst <= 1, f"worst error {worst:.3g} of the bound"
    return dict(pk=pk, fn=fn, c=c, pc=pc, of=of, q=q, ws=ws, out=out, want=want, tol=tol)


BITS = [16, 8]


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("n", [1, 127, 128, 129, 500, 1000])
def test_own_rows_only(pk, bits, n):
    run_case(pk, bits, 1, 2, 4, [n], [], [0], given=False)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N,H,G,longest", [(1, 1, 1, 1024), (76, 2, 8, 300), (77, 2, 5, 700), (305, 2, 4, 512),
                                           (305, 2, 2, 513), (76, 2, 4, 2048), (76, 2, 4, 2049), (77, 2, 3, 1025), (1, 1, 8, 599),
                                           (4, 3, 8, 600), (2, 1, 5, 32768), (1, 1, 1, 32769), (13, 1, 4, 601),
                                           (8, 4, 3, 16384), (8, 4, 3, 16385), (33, 1, 4, 600), (36, 2, 8, 4096),
                                           (36, 2, 8, 4097)])
def test_short_sequences(pk, bits, N, H, G, longest):
    """Own rows by whole units of 8, 4 and 2 warps and of clusters of 8, 4 and 2 CTAs, and past these lengths planned;
    then with a bound below the lengths."""
    lens = [(longest - 89 * i) % (longest + 1) for i in range(N)]
    lens[N // 2:N // 2 + 3] = [0, 1, 17][:len(lens[N // 2:N // 2 + 3])]
    lens[0] = longest
    r = run_case(pk, bits, N, H, G, lens, [], [0] * N, given=False)
    r["c"].c.n_max = 1
    r["out"].fill_(float("nan"))
    r["fn"](None, None, r["c"].c, r["q"], r["out"], r["ws"], r["ws"].numel())
    assert ((r["out"].double() - r["want"]).abs() <= r["tol"]).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("G", [1, 3, 8])
def test_ragged_batch_with_empty_sequences(pk, bits, G):
    lens = [0, 1, 700, 0, 129, 1500, 128]
    run_case(pk, bits, 7, 3, G, lens, [], [0] * 7, given=False)


def test_nothing_at_all(pk):
    r = run_case(pk, 16, 3, 2, 4, [0, 0, 0], [], [0] * 3, given=False)
    assert (r["out"] == 0).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("bound", [None, 3000, 65536])
@pytest.mark.parametrize("N,G", [(1, 4), (5, 3), (4, 8), (9, 4), (16, 4), (31, 4), (32, 4), (33, 4), (43, 3), (64, 4),
                                 (65, 4), (70, 8)])
def test_one_prefix(pk, bits, N, G, bound):
    """Rows below, at and past 16 (streamed), 32 and 64 (copies), 128 (one stream's worth) and 256 (a unit's)."""
    lens = [(37 * i) % 300 for i in range(N)]
    for plen in (1000, 1):
        run_case(pk, bits, N, 2, G, lens, [plen], [0] * N, given=False, bound=bound)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N,H,G,plens,longest", [(38, 4, 3, [900], 4096), (40, 8, 5, [5000], 2048), (77, 8, 2, [300], 600),
                                                 (160, 4, 8, [2000], 469), (44, 8, 8, [700, 0, 1, 200], 300), (44, 8, 1, [700, 0, 1, 200], 300),
                                                 (500, 2, 1, [130, 900], 1024), (38, 4, 7, [900], 4097), (40, 4, 7, [900], 2049),
                                                 (20, 1, 1, [9000], 50), (70, 1, 1, [9000], 50), (24, 3, 2, [3000], 70)])
def test_own_rows_behind_the_wide_kernel(pk, bits, N, H, G, plens, longest):
    """Joined with the prefix's partials in units of 8, 4 and 2 warps; prefixes of few sequences and of none; and one
    token more than that takes."""
    lens = [(89 * i) % (longest + 1) for i in range(N)]
    lens[1] = longest
    P = len(plens)
    of = [(0, 0, 0, 0, 1, 0, 0, 2, 3, -1)[i % 10] for i in range(N)] if P > 2 else [i % P for i in range(N)]
    run_case(pk, bits, N, H, G, lens, plens, of, bound=65536)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("bound", [None, 3000, 65536])
@pytest.mark.parametrize("plens,of", [([0], 0), ([0, 0], 1), ([900], -1), ([900, 5], 2)])
def test_prefixes_that_give_nothing(pk, bits, bound, plens, of):
    """Only empty prefixes, or prefixes that no sequence has, every way; also with no rows of their own."""
    for lens in ([(37 * i) % 300 for i in range(40)], [0] * 40):
        r = run_case(pk, bits, 40, 4, 4, lens, plens, [of] * 40, bound=bound)
    assert (r["out"] == 0).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N,H,plen,longest", [(3, 4, 30000, 2000), (8, 4, 12000, 4000), (18, 4, 4000, 4000), (5, 1, 20000, 0)])
def test_clusters_over_prefixes(pk, bits, N, H, plen, longest):
    """Units of 8, 4 and 2 CTAs over a prefix, an empty one and none, with and without rows of their own."""
    lens = [(997 * i) % (longest + 1) for i in range(N)]
    lens[-1] = longest
    run_case(pk, bits, N, H, 4, lens, [plen, 0], [(0, 0, 1, 5)[i % 4] for i in range(N)])


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("bound", [None, 3000, 65536])
def test_several_prefixes(pk, bits, bound):
    """Mixed order, sequences without a prefix, an empty prefix and one nobody has."""
    N = 41
    of = [(0, 2, 1, 0, -1, 3, 7, 2)[i % 8] for i in range(N)]
    lens = [(53 * i) % 400 for i in range(N)]
    run_case(pk, bits, N, 2, 8, lens, [777, 1, 513, 0, 900], of, bound=bound)


@pytest.mark.parametrize("bits", BITS)
def test_long_prefix_and_peaked_weights(pk, bits):
    """Many tiles for each CTA, a maximum that rises often, and one that sits in the first token."""
    run_case(pk, bits, 40, 4, 4, [(211 * i) % 900 for i in range(40)], [40001], [0] * 40, spread=1.3)
    run_case(pk, bits, 9, 1, 4, [5] * 9, [70000], [0] * 9, spread=0.2, sink=False, given=False)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N,bound", [(1, 1900), (1, 2000), (40, 1900), (40, 2000), (17, 65536), (40, 65536)])
def test_rising_maximum_of_a_prefix(pk, bits, N, bound):
    """Logits that climb along a prefix's rows, in whole units, streamed, and on the tensor cores with 68 and 160 query rows."""
    g = torch.Generator(device="cuda").manual_seed(8)
    H, G, n, cap = 1, 4, 2000, 65536
    q = (1 + 0.1 * torch.randn((N, H, G, D), generator=g, device="cuda")).to(torch.bfloat16)
    ramp = torch.linspace(-4, 4, n, device="cuda")[None, None, :, None]
    ramp = torch.cat((ramp, torch.zeros((1, 1, cap - n, 1), device="cuda")), 2)
    k = (ramp + 0.05 * torch.randn((1, H, cap, D), generator=g, device="cuda")).to(torch.bfloat16)
    v = torch.randn((1, H, cap, D), generator=g, device="cuda").to(torch.bfloat16)
    own = [(5 * i) % 70 for i in range(N)]
    ko, vo = draw_rows(g, N, H, 512)
    c, rows = make_cache(pk, bits, G, 512, own, ko, vo)
    pc, prows = make_cache(pk, bits, G, cap, [n], k, v)
    pc.c.n_max = bound
    ws = pk.shared_workspace(c, pc)
    out = torch.empty((N, H, G, D), dtype=torch.bfloat16, device="cuda")
    (pk.bpkv_shared_attend if bits == 16 else pk.bpkv_shared_attend8)(pc.c, None, c.c, q, out, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    want, tol = reference(q, rows, own, prows, [n], [0] * N, bits)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("n", [2000, 1023])
def test_rising_maximum(pk, bits, n):
    """Logits that climb along the rows: O is rescaled tile after tile."""
    g = torch.Generator(device="cuda").manual_seed(7)
    N, H, G = 3, 1, 4
    q = torch.ones((N, H, G, D), device="cuda").to(torch.bfloat16)
    ramp = torch.linspace(-4, 4, n, device="cuda")[None, None, :, None]
    k = (ramp + 0.05 * torch.randn((N, H, n, D), generator=g, device="cuda")).to(torch.bfloat16)
    v = torch.randn((N, H, n, D), generator=g, device="cuda").to(torch.bfloat16)
    cap = 2048
    pad = torch.zeros((N, H, cap - n, D), dtype=torch.bfloat16, device="cuda")
    lens = [n, n * 11 // 20, 64]
    c, rows = make_cache(pk, bits, G, cap, lens, torch.cat((k, pad), 2), torch.cat((v, pad), 2))
    ws = pk.shared_workspace(c)
    out = torch.empty((N, H, G, D), dtype=torch.bfloat16, device="cuda")
    (pk.bpkv_shared_attend if bits == 16 else pk.bpkv_shared_attend8)(None, None, c.c, q, out, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    want, tol = reference(q, rows, lens, None, [], [0] * N, bits)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("bound", [None, 3000, 65536])
def test_repeats_streams_and_graphs(pk, bits, bound):
    """The same bits from every call, on another stream, and from two captured graphs that share the workspace."""
    r = run_case(pk, bits, 33, 2, 4, [(37 * i) % 300 for i in range(33)], [3001], [0] * 33, given=False, bound=bound)
    args = (r["pc"].c, r["of"], r["c"].c, r["q"])
    first = r["out"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = torch.empty_like(first)
    with torch.cuda.stream(s):
        for _ in range(3):
            r["fn"](*args, out2, r["ws"], r["ws"].numel())
    s.synchronize()
    assert torch.equal(out2, first)
    outs = [torch.empty_like(first), torch.empty_like(first)]
    graphs = []
    for o in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r["fn"](*args, o, r["ws"], r["ws"].numel())
        graphs.append(gr)
    for gr in (graphs[0], graphs[1], graphs[0]):
        for o in outs:
            o.zero_()
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and not outs[1].any()
    # lengths are read on the device: a replay follows them
    r["c"].seq_len.zero_()
    r["pc"].seq_len.zero_()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert not outs[1].any()
