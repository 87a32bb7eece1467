"""Calls of few tokens behind long rows of many sequences, some of which are idle: one
sequence may have all of the tokens, which the host does not know.  Where its rows would
be streamed again and again the tensor cores take the call, else it is streamed; either
way gives its own bits, by which the tests tell the two apart.  Bounds as in
test_gpu_prompt."""
import pytest
import torch
from test_gpu_prompt import attention, causal, check, run_prompt, run_tree
from test_gpu_shared import draw_rows, make_cache, pk  # noqa: F401

pytestmark = pytest.mark.gpu
D, H, G, ROWS = 128, 2, 4, 20000
BITS = [16, 8]


def cache(pk, bits, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = draw_rows(g, N, H, ROWS // 512 * 512 + 512)
    return make_cache(pk, bits, G, k.shape[2], [ROWS] * N, k, v)


def one_of(pk, c, i):
    """Sequence i of a cache as a cache of its own."""
    names = ("k_rows", "v_rows") if isinstance(c, pk.Cache) else ("k8", "v8", "kexp", "vexp")
    one = type(c)(1, H, G, c.c.cap_tokens)
    for name in (*names, "seq_len"):
        getattr(one, name).copy_(getattr(c, name)[i:i + 1])
    one.c.n_max = c.c.n_max
    return one


def args(pk, q, new, c):
    out = torch.full_like(q, 7.0)
    start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], device="cuda")
    a = pk.prompt_args(q, out, start, cache=c)
    ws = pk.prompt_workspace(a)
    ws[256:].fill_(0xff)
    return a, ws, out, start


def attend(pk, q, new, c):
    a, ws, out, _ = args(pk, q, new, c)
    pk.bpkv_prompt_attend(a, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    return out


def draw_q(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, H, G, D), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N,i,t", [(64, 0, 64), (64, 63, 64), (33, 17, 33), (40, 39, 60)])
def test_one_sequence_has_all_tokens(pk, bits, N, i, t):
    """As if the others were not there: on the tensor cores."""
    c, rows = cache(pk, bits, N, i)
    q = draw_q(t, N)
    out = attend(pk, q, [t if j == i else 0 for j in range(N)], c)
    check(out, *attention(q, rows[0][i, :, :ROWS], rows[1][i, :, :ROWS], causal(t, ROWS)))
    assert torch.equal(out, attend(pk, q, [t], one_of(pk, c, i)))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("N", [64, 20])
def test_every_sequence_has_one(pk, bits, N):
    """Streamed, as a tree of one node."""
    c, rows = cache(pk, bits, N, N)
    q = draw_q(N, 1)
    out = attend(pk, q, [1] * N, c)
    tree = torch.empty_like(q)
    ws = pk.tree_workspace(c, 1)
    (pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8)(c.c, 1, None, q, tree, ws, ws.numel())
    assert torch.equal(out, tree)
    for i in (0, N - 1):
        check(out[i:i + 1], *attention(q[i:i + 1], rows[0][i, :, :ROWS], rows[1][i, :, :ROWS], causal(1, ROWS),
                                       None if bits == 16 else rows[2][i, :, :ROWS]))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("new,past", [([1] * 31 + [32], [100] * 31 + [15000]), ([1] * 31 + [32], [15000] * 31 + [10]),
                                      ([0, 9, 0, 1] * 6, [9000] * 24), ([2] * 32, [100, 16000] * 16),
                                      ([4] * 16, [12000] * 16), ([3, 60, 0] + [0] * 30, [17000, 3, 5] + [0] * 30)])
def test_tokens_in_any_proportion(pk, bits, new, past):
    run_prompt(pk, "cache", new, past, 2, 4, seed=len(new), bits=bits, pad=1, n_max=17024)


@pytest.mark.parametrize("bits", BITS)
def test_a_captured_call_with_other_starts(pk, bits):
    """What takes the call is found on the device, also in a replayed graph."""
    N = T = 64
    c, _ = cache(pk, bits, N, 3)
    q = draw_q(T, 3)
    one, all_ = [1] * N, [0] * 9 + [T] + [0] * (N - 10)
    want = {k: attend(pk, q, new, c) for k, new in (("one", one), ("all", all_))}
    a, ws, out, start = args(pk, q, one, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.bpkv_prompt_attend(a, ws, ws.numel())
    for k, new in (("one", one), ("all", all_), ("one", one), ("none", [0] * N)):
        start.copy_(torch.tensor([sum(new[:i]) for i in range(N + 1)]))
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out, want[k]) if k in want else (out == 7.0).all(), k
    # starts outside the tokens and before the last one, as everywhere
    start.copy_(torch.tensor([-5, 60, 10, 1 << 40] + [0] * (N - 3)))
    out.fill_(7.0)
    graph.replay()
    assert torch.equal(out, attend(pk, q, [60, 0, 4] + [0] * (N - 3), c)) and pk.bpkv_read_status(ws) == 0


@pytest.mark.parametrize("bits", BITS)
def test_the_checked_call(pk, bits):
    """tree_attend is the call of the cache's kind."""
    got = run_tree(pk, bits, 3, 9, 2, 4, [700, 9, 4000])
    out = torch.empty_like(got["out"])
    pk.tree_attend(got["c"], got["q"], out, pk.tree_workspace(got["c"], 9), got["mask"])
    assert torch.equal(out, got["out"])
    with pytest.raises(ValueError):
        pk.tree_attend(got["c"], got["q"].float(), out, got["ws"], got["mask"])
