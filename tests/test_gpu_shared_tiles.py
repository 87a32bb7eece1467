"""Attention over shared prefixes: that every tile counts, as often as it should
and under its own scales (bpkv_shared_attend, bpkv_shared_attend8)."""
import math

import pytest
import torch

import test_gpu_shared
from test_gpu_shared import make_cache, run_case

pytestmark = pytest.mark.gpu
D = 128
TILE = 128


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import bit_plane_kv_encode_gb300 as m
    return m


def marked_rows(g, P, H, cap):
    """Keys of nearly equal logits whose scales differ from tile to tile, values that name their tile: channel (tile mod
    128) alone is set, to a power of two of the channel's own, so that a channel's sum is its few tiles' and the scales of
    neighbouring tiles differ by several binary orders."""
    tile = torch.arange(cap, device="cuda") // TILE
    k = 0.25 * torch.randn((P, H, cap, D), generator=g, device="cuda")
    k[..., 0] += 0.5
    k[..., 64:] = 0
    k[..., 127] = torch.exp2((tile * 5 % 8 - 3).float())  # sets the row's scale; q has nothing there
    v = torch.zeros((P, H, cap, D), device="cuda")
    mark = tile % D
    v[:, :, torch.arange(cap, device="cuda"), mark] = torch.exp2((mark * 7 % 12 - 6).float())
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("behind", [0, 5000])
@pytest.mark.parametrize("N,G,H,plens", [
    (5, 4, 1, [250001]), (12, 4, 1, [250001]), (25, 4, 1, [250001]), (40, 5, 1, [250001]),  # copies 4, 2, 1; both streams
    (5, 4, 4, [65001]), (9, 7, 4, [65001]), (32, 4, 3, [90112]), (70, 4, 4, [65001]),       # heads that a CTA goes on to
    (37, 4, 2, [66000, 131, 47001, 90001]), (75, 8, 1, [120001, 64, 130001]),
    (75, 8, 1, [120001, 90064])])
def test_every_tile_counts(pk, bits, behind, N, G, H, plens):
    """Twelve tiles and more for each CTA of the wide kernel, with and without rows that end inside a tile; joined in
    whole units (behind 0) and by the join behind the streaming kernel (what the host knows of own rows: 5000).

    Every value is positive, so that a channel's error is relative to itself.  A weight: 2^-8 as bf16; 8-bit rows 2^-6 +
    2^-11 as two e5m2 pieces, and n 2^-19 of the largest w 2^e for what their smallest step loses.  Logits: B as in
    test_gpu_shared, over the channels that q has; in the base-2 exponent at most 64, three roundings of it, 2^-17.  Sums:
    no term passes through more additions than a CTA has tokens, plus its parts and the join's.  A channel has at most
    sixteen tiles of nearly equal weight: one of them lost or counted twice is 6% and more of it."""
    g = torch.Generator(device="cuda").manual_seed(N + G)
    P = len(plens)
    pcap = (max(plens) + 511) // 512 * 512
    q = torch.zeros((N, H, G, D), device="cuda")
    q[..., :64] = torch.randn((N, H, G, 64), generator=g, device="cuda")
    q[..., 0] = 8
    q = q.to(torch.bfloat16)
    k, v = marked_rows(g, P, H, pcap)
    pc, (pk64, pv64, scale) = make_cache(pk, bits, G, pcap, plens, k, v)
    c = (pk.Cache if bits == 16 else pk.Rows8)(N, H, G, 5120 if behind else 512)
    c.c.n_max = behind
    of = [i * 3 % P for i in range(N)]
    ws = pk.shared_workspace(c, pc)
    out = torch.full((N, H, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fn = pk.bpkv_shared_attend if bits == 16 else pk.bpkv_shared_attend8
    fn(pc.c, torch.tensor(of, dtype=torch.int32, device="cuda"), c.c, q, out, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    chain = (sum(math.ceil(n / TILE) * math.ceil(sum(i == p for i in of) * G / 256) for p, n in enumerate(plens)) * H //
             152 + 2) * TILE + 2 * 152
    worst = 0.0
    for p in range(P):
        mine = [i for i in range(N) if of[i] == p]
        if not mine:
            continue
        n = plens[p]
        for h in range(H):
            qd, kd, vd = q[mine, h].double().reshape(-1, D), pk64[p, h, :n], pv64[p, h, :n]
            w = torch.softmax(qd @ kd.T / math.sqrt(D), -1)
            o = w @ vd
            B = 130 * 2.0 ** -24 * (qd.abs() @ kd.abs().T).amax(-1) / math.sqrt(D)
            rel, floor = 2.0 ** -8, torch.zeros(len(mine) * G, dtype=torch.float64, device="cuda")
            if bits == 8:
                rel = 2.0 ** -6 + 2.0 ** -11
                B = B + 2.0 ** -16 * 8 * kd[:, :64].abs().sum(-1).amax() / math.sqrt(D)
                floor = n * 2.0 ** -19 * (w * scale[p, h, :n]).amax(-1)
            tol = (rel + 2.0 ** -8 + 2 * B[:, None] + 2.0 ** -17 + chain * 2.0 ** -23) * o + floor[:, None]
            if n >= 40000:  # the bound tells one tile of a channel's
                assert float((tol / o.clamp(min=1e-30)).max()) < 0.04
            err = (out[mine, h].double().reshape(-1, D) - o).abs()
            worst = max(worst, float((err / (tol + 1e-30)).max()))
    assert worst <= 1, f"worst error {worst:.3g} of the bound"


def halves_reference(q, rows, lens, prows, plens, prefix_of, bits):
    """As test_gpu_shared.reference for 8-bit rows, with what the ways beside the tensor-core kernel hold: weights as
    halves (2^-11; their smallest step 2^-24 under a largest of 2^11 at least: 448 2^-25 2^-11 < 2^-27 a token), q as
    halves under its row's scale (off by 2^-25 at most where the largest is 2^7: 2^-32 of it); the base-2 exponent, at
    most 64, rounded three times, 2^-17."""
    assert bits == 8
    N, H, G, _ = q.shape
    o = torch.zeros((N, H, G, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    for i in range(N):
        p = prefix_of[i]
        k, v, s = [r[i, :, :lens[i]] for r in rows]
        if prows is not None and 0 <= p < len(plens):
            k, v, s = [torch.cat((r[p, :, :plens[p]], x), 1) for r, x in zip(prows, (k, v, s))]
        n = k.shape[1]
        if n == 0:
            continue
        qd = q[i].double()
        w = torch.softmax(qd @ k.transpose(-1, -2) / math.sqrt(D), -1)
        o[i] = w @ v
        B = (130 * 2.0 ** -24 * (qd.abs() @ k.abs().transpose(-1, -2)).amax(-1) +
             2.0 ** -32 * qd.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None]) / math.sqrt(D)
        tol[i] = ((2.0 ** -11 + 2 * B[..., None] + 2.0 ** -17 + n * 2.0 ** -23 + 2.0 ** -21) * (w @ v.abs()) +
                  2.0 ** -8 * o[i].abs() + n * 2.0 ** -27 * (w * s[:, None]).amax(-1)[..., None])
    return o, tol + 1e-30


@pytest.mark.parametrize("N,H,G,longest,plens,bound", [
    (1, 2, 4, 500, [], None), (77, 2, 5, 700, [], None), (305, 2, 4, 512, [], None), (4, 3, 8, 6000, [], None),  # whole
    (36, 2, 8, 5000, [], None), (1, 1, 1, 32769, [], None),                                                      # planned
    (16, 2, 4, 300, [900], None), (5, 4, 3, 1000, [12000], None),                           # whole, over a prefix
    (40, 2, 4, 300, [2900], 3000), (33, 2, 8, 200, [1000, 0, 700], 3000)])                  # streamed by 16 rows
def test_weights_are_halves_beside_the_tensor_cores(pk, monkeypatch, N, H, G, longest, plens, bound):
    monkeypatch.setattr(test_gpu_shared, "reference", halves_reference)
    lens = [(longest - 89 * i) % (longest + 1) for i in range(N)]
    run_case(pk, 8, N, H, G, lens, plens, [i % len(plens) if plens else 0 for i in range(N)], bound=bound)
