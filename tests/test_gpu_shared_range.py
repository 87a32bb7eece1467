"""Attention over shared prefixes at logits far beyond a softmax's usual range
(bpkv_shared_attend, bpkv_shared_attend8)."""
import math

import pytest
import torch

from test_gpu_shared import make_cache

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import bit_plane_kv_encode_gb300 as m
    return m


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("N,bound", [(1, 1900), (1, 40000), (40, 1900), (40, 3000), (17, 65536), (40, 65536)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_logits(pk, bits, N, bound, sign):
    """Logits of 2^14 to 2^29, of one sign: the tokens whose keys have the largest share the weight evenly, and any other
    is thousands below it.  Equal rows have equal logits, so that those of float32 do not count here; what counts is that
    a maximum of such size, less the shift of the weights and plus the rise that is let pass, leaves them in range.  Values
    grow by powers of two along the rows, which 8-bit rows' scales add to the exponent.

    Weights: 2^-8 as bf16, 2^-6 + 2^-11 as pieces (a sum of n terms 2^-23 n, the output 2^-8).  8-bit rows: from 2^24 on
    the base-2 exponent is a whole number of 2, 4, ... and a scale's power of two is rounded into it: by half of that
    number at most, so parts joined after that may weigh 2^16 of one another.  There the output has to lie between the
    values it can take."""
    g = torch.Generator(device="cuda").manual_seed(9)
    H, G, n, cap = 2, 4, 1900, 65536
    fn = pk.bpkv_shared_attend if bits == 16 else pk.bpkv_shared_attend8
    q = torch.full((N, H, G, D), float(sign), dtype=torch.bfloat16, device="cuda")
    j = torch.arange(cap, device="cuda")
    step = torch.tensor([1.0, 1.125, 1.25], device="cuda")[j // 7 % 3]
    v = torch.rand((1, H, cap, D), generator=g, device="cuda") + 0.5
    v = (v * torch.exp2((j * 9 // n % 9 - 2).float())[:, None]).to(torch.bfloat16)
    none = torch.zeros((N, H, 512, D), dtype=torch.bfloat16, device="cuda")
    c, _ = make_cache(pk, bits, G, 512, [0] * N, none, none)
    best = (step[:n] == (1.25 if sign > 0 else 1.0)).double()
    for e in range(10, 26):
        k = (2.0 ** e * step)[None, None, :, None].expand(1, H, cap, D).to(torch.bfloat16)
        pc, (_, v64, _) = make_cache(pk, bits, G, cap, [n], k, v)
        pc.c.n_max = bound
        ws = pk.shared_workspace(c, pc)
        out = torch.full((N, H, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        fn(pc.c, None, c.c, q, out, ws, ws.numel())
        assert pk.bpkv_read_status(ws) == 0
        mine = v64[0, :, :n]
        top = math.sqrt(D) * 2.0 ** e * 1.25 * math.log2(math.e)
        if bits == 16 or top < 2 ** 23:
            want = ((best[:, None] * mine).sum(1) / best.sum())[None, :, None]
            rel = (2.0 ** -8 if bits == 16 else 2.0 ** -6 + 2.0 ** -11 + top * 2.0 ** -23) + n * 2.0 ** -23 + 2.0 ** -8
            err = (out.double() - want).abs() / want
            assert float(err.max()) <= rel, f"2^{e}: {float(err.max())}"
        else:
            few = mine[:, best > 0]
            lo, hi = few.amin(1)[None, :, None], few.amax(1)[None, :, None]
            within = bool(((out.double() >= lo * (1 - 2.0 ** -5)) & (out.double() <= hi * (1 + 2.0 ** -5))).all())
            assert within, f"2^{e}"
