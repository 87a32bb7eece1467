"""Longer uses of the serving operators: drafted tokens that are rejected."""
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
