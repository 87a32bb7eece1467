"""Longer uses of the serving operators: drafted tokens that are rejected,
prompts of many turns, device lengths above the host's bound."""
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


def test_drafted_tokens_overwritten_again_and_again(pk):
    """Far more tokens drafted than the cache holds; one a step stays.  With n_max kept at what the host knows, the
    cache takes tokens behind its rows to its end."""
    g = torch.Generator(device="cuda").manual_seed(31)
    N, H, t, cap, steps = 3, 2, 6, 512, 120
    c = pk.Rows8(N, H, 4, cap)
    first = torch.tensor([0, 40, 300], device="cuda")
    start = first.clone()
    want = torch.zeros((N, H, cap, D), dtype=torch.float64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for x in (c.k8, c.v8):
        x.zero_()
    c.kexp.fill_(127)
    c.vexp.fill_(127)
    for i in range(steps):
        # small whole numbers: codes hold them exactly
        k = torch.randint(-8, 9, (N, H, t, D), generator=g, device="cuda").to(torch.bfloat16)
        c.append(k, -k, start, status)
        c.n_max = 300 + i + t
        for s in range(N):
            at = int(first[s]) + i
            want[s, :, at:at + t] = k[s].double()
        start += 1
    assert torch.equal(c.seq_len, start - 1 + t)
    more = cap - c.n_max
    k = torch.randint(-8, 9, (N, H, more, D), generator=g, device="cuda").to(torch.bfloat16)
    for s in range(N):
        n = int(c.seq_len[s])
        want[s, :, n:n + more] = k[s].double()
    lens = c.seq_len + more
    c.append(k, -k, None, status)
    assert c.n_max == cap and torch.equal(c.seq_len, lens) and not status.any()
    there = (torch.arange(cap, device="cuda") < lens[:, None])[:, None, :, None]
    kr, vr = c.read(0, cap)
    assert torch.equal(kr.double(), torch.where(there, want, 0.0))
    assert torch.equal(vr.double(), torch.where(there, -want, 0.0))


@pytest.mark.parametrize("N,t,H,G,rot,pairs", [(10, 8001, 1, 1, 128, False), (5, 8001, 2, 8, 64, True),
                                               (3, 13337, 1, 1, 18, False)])
def test_projected_heads_of_many_turns(pk, N, t, H, G, rot, pairs):
    """A CTA's second and third turn: more tokens than the grid's 4864 CTAs take at once, eight each."""
    from test_gpu_rows8 import check, qkv_reference
    assert N * t > 8 * 4864
    g = torch.Generator(device="cuda").manual_seed(t)
    cap = (t + 1100 + 511) // 512 * 512
    qkv = torch.randn((N, t, (G + 2) * H * D), generator=g, device="cuda").to(torch.bfloat16)
    pos = 1000 - 97 * torch.arange(N, device="cuda")
    inv = (1e4 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float()
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    c, d = pk.Rows8(N, H, G, cap), pk.Rows8(N, H, G, cap)
    for x in (c, d):
        for y in (x.k8, x.v8, x.kexp, x.vexp):
            y.zero_()
    q = torch.full((N, t, H, G, D), float("nan"), device="cuda")
    k = torch.full((N, H, t, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    q2 = torch.empty((N, t, H, G, D), dtype=torch.bfloat16, device="cuda")
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, pos, inv, w, w, pairs=pairs, k_out=k, v_out=v))
    pk.bpkv_qkv_rope(pk.qkv_args(qkv, q2, H, pos, inv, w, w, pairs=pairs, k_out=k2, v_out=v2, rows8=c))
    (wq, tq), (wk, tk), wv = qkv_reference(qkv, N, t, H, G, pos, inv, w, w, 1e-6, pairs)
    for got, want, tol in ((q, wq, tq), (q2, wq, tq), (k, wk, tk), (k2, wk, tk)):
        check(got, want, tol)
    assert torch.equal(v.double(), wv) and torch.equal(v2, v)
    # into the 8-bit rows: as the append of the bf16 rows does it
    d.append(k2, v2, pos)
    for a, b in ((c.k8, d.k8), (c.v8, d.v8), (c.kexp, d.kexp), (c.vexp, d.vexp), (c.seq_len, d.seq_len)):
        assert torch.equal(a, b)
    assert torch.equal(c.seq_len, pos + t)


LOW = [
    # prefix on the tensor cores; own rows behind it in whole units; the same, joined by the streaming kernel's join
    (40, 2, 4, 900, [60001], 900, 20000), (40, 2, 4, 5000, [60001], 300, 20000), (40, 2, 4, 5600, [30001], 5000, 20000),
    # no prefix, planned; a prefix that is streamed by 16 query rows; with several
    (1, 2, 4, 60000, [], 40000, 0), (40, 2, 4, 700, [9001], 300, 3000), (41, 2, 8, 400, [5003, 0, 2000], 300, 1800),
    # clusters of 8 and 2 CTAs; whole units of 8, 4 and 2 warps
    (2, 2, 5, 9000, [7001], 2000, 3000), (9, 4, 4, 2500, [6001], 700, 1000), (20, 4, 8, 3000, [2001], 300, 1000),
    (40, 4, 3, 3000, [900], 900, 300), (200, 4, 2, 700, [300], 300, 100),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("N,H,G,longest,plens,own_bound,prefix_bound", LOW)
def test_lengths_above_the_hosts_bound(pk, bits, N, H, G, longest, plens, own_bound, prefix_bound):
    """n_max chooses the way and sizes its launches; longer sequences and prefixes are attended to in full, every way."""
    from test_gpu_shared import run_case
    lens = [(longest - 89 * i) % (longest + 1) for i in range(N)]
    r = run_case(pk, bits, N, H, G, lens, plens, [i % len(plens) if plens else 0 for i in range(N)])
    r["c"].c.n_max = own_bound
    if plens:
        r["pc"].c.n_max = prefix_bound
    r["out"].fill_(float("nan"))
    r["fn"](r["pc"].c if plens else None, r["of"], r["c"].c, r["q"], r["out"], r["ws"], r["ws"].numel())
    assert ((r["out"].double() - r["want"]).abs() <= r["tol"]).all()
    assert pk.bpkv_read_status(r["ws"]) == 0


def turns(p, f):
    """p f / (2 pi) modulo one, from whole numbers of 200 bits (pi by Machin's formula)."""
    one = 1 << 200

    def arctan_of_inverse(x):
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    a, b = float(f).as_integer_ratio()
    return p * a * one * one // (b * two_pi) % one / one


@pytest.mark.parametrize("first", [1 << 31, (1 << 36) + 12345, (1 << 40) + 7, (1 << 50) + 1, -3, -(1 << 35)])
def test_far_positions(pk, first):
    """The angle's bound: |p| (1 + f) 2^-64 turns, the fixed point's last bit (2^-32 turns), the float's rounding (2^-25
    half turns); then sincospi 2^-23, and the two products and the sum 3 2^-24 of |a| + |b|."""
    import math
    H, G, t = 1, 1, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn((1, t, 3 * D), generator=g, device="cuda").to(torch.bfloat16)
    inv = (5e5 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float()
    inv[1] = 3.0
    q = torch.empty((1, t, H, G, D), device="cuda")
    pk.bpkv_qkv_rope(pk.qkv_args(qkv, q, H, torch.tensor([first], device="cuda"), inv))
    x, y = qkv[0, :, :D].double().cpu(), q[0, :, 0, 0].double().cpu()
    for i in range(t):
        p = first + i
        for j, f in enumerate(inv.tolist()):
            u = 2 * math.pi * turns(p, f)
            a, b = float(x[i, j]), float(x[i, j + D // 2])
            off = 2 * math.pi * (abs(p) * (1 + f) * 2.0 ** -64 + 2.0 ** -32) + math.pi * 2.0 ** -25
            tol = (off + 2.0 ** -23 + 3 * 2.0 ** -24) * (abs(a) + abs(b))
            assert abs(float(y[i, j]) - (a * math.cos(u) - b * math.sin(u))) <= tol
            assert abs(float(y[i, j + D // 2]) - (b * math.cos(u) + a * math.sin(u))) <= tol
