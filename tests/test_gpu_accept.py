"""Accepted tokens into 8-bit rows (bpkv_rows8_accept): the same bytes that
bpkv_rows8_append writes for the same tokens, and nothing else."""
import pytest
import torch
from test_gpu_shared import draw_rows, pk  # noqa: F401

pytestmark = pytest.mark.gpu
D = 128
NAMES = ("k8", "v8", "kexp", "vexp")


def mark(c):
    for n in NAMES:
        getattr(c, n).fill_(0xa5)


def run(pk, N, H, t, start, count, path=None, cap=1024, at_len=False, refused=()):
    g = torch.Generator(device="cuda").manual_seed(N * t)
    k, v = draw_rows(g, N, H, t)
    c, want = pk.Rows8(N, H, 4, cap), pk.Rows8(N, H, 4, cap)
    mark(c)
    mark(want)
    old = torch.tensor(start if at_len else [7] * N, device="cuda")
    c.seq_len.copy_(old)
    c.n_max = min(cap, max(0, max(start))) if at_len else 9
    n_max = c.n_max
    one = pk.Rows8(1, H, 4, cap)
    for i in range(N):
        if i in refused or count[i] == 0:
            continue
        nodes = path[i][:count[i]] if path else list(range(count[i]))
        nodes = torch.tensor([min(max(x, 0), t - 1) for x in nodes], device="cuda")
        one.append(k[i:i + 1, :, nodes].contiguous(), v[i:i + 1, :, nodes].contiguous(),
                   torch.zeros(1, dtype=torch.int64, device="cuda"))
        for n in NAMES:
            getattr(want, n)[i, :, start[i]:start[i] + count[i]] = getattr(one, n)[0, :, :count[i]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = c.seq_len if at_len else torch.tensor(start, device="cuda")
    p = torch.tensor([(x + [-9] * t)[:t] for x in path], dtype=torch.int32, device="cuda") if path else None
    c.accept(k, v, s, torch.tensor(count, dtype=torch.int32, device="cuda"), p, status)
    torch.cuda.synchronize()
    for n in NAMES:
        assert torch.equal(getattr(c, n), getattr(want, n)), n
    lens = [int(old[i]) if i in refused else start[i] + count[i] for i in range(N)]
    assert c.seq_len.tolist() == lens
    assert c.n_max == min(n_max + t, cap)
    return int(status)


@pytest.mark.parametrize("at_len", [False, True])
@pytest.mark.parametrize("N,H,t", [(1, 1, 1), (3, 2, 5), (7, 8, 16), (2, 3, 64), (40, 8, 33)])
def test_first_tokens(pk, N, H, t, at_len):
    start = [(17 * i) % 900 for i in range(N)]
    count = [(5 * i + t) % (t + 1) for i in range(N)]
    assert run(pk, N, H, t, start, count, at_len=at_len) == 0


@pytest.mark.parametrize("at_len", [False, True])
def test_paths(pk, at_len):
    """Ways down a tree, a token more than once, tokens in any order."""
    path = [[0, 2, 5], [7, 7, 7, 7], [6, 5, 4, 3, 2, 1, 0], [], [3]]
    assert run(pk, 5, 3, 8, [0, 63, 64, 5, 1000], [3, 4, 7, 0, 1], path, at_len=at_len) == 0


def test_many_rows(pk):
    assert run(pk, 16, 8, 700, [300 - 3 * i for i in range(16)], [(211 * i) % 701 for i in range(16)]) == 0


@pytest.mark.parametrize("at_len", [False, True])
def test_what_does_not_fit_is_refused(pk, at_len):
    cap = 1024
    start, count = [cap - 4, cap - 5, cap, 0, 0], [5, 5, 0, 9, -1]
    if at_len:
        # the host's bound keeps the lengths within the cache; counts may still be wrong
        assert run(pk, 3, 2, 8, [4, 0, 0], [5, 9, -1], at_len=True, refused=(1, 2)) == pk.DEV_OVERFLOW
    else:
        assert run(pk, 5, 2, 8, start, count, cap=cap, refused=(0, 3, 4)) == pk.DEV_OVERFLOW
        assert run(pk, 1, 2, 8, [-1], [2], cap=cap, refused=(0,)) == pk.DEV_OVERFLOW


def test_path_outside_the_tokens(pk):
    assert run(pk, 2, 2, 4, [0, 0], [3, 2], [[0, 9, 1], [-4, 2]]) == pk.DEV_OVERFLOW
    # past the count it says nothing
    assert run(pk, 1, 2, 4, [0], [1], [[2, 99, -1, 77]]) == 0
