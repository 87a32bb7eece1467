"""Attention of several new tokens of a sequence at once (bpkv_prompt_attend over
packed keys or a cache, bpkv_tree_attend over bf16 rows, bpkv_tree_attend8 over
8-bit rows) against the formula in 64 bits.

Bounds.  With p the exact softmax weights, A = sum p |v| and o = sum p v:
  - weights enter the product as bf16, off by at most 2^-8 of themselves;
  - logits are float32 sums of 128 products, off by B <= 130 2^-24 sum_j |q_j k_j|
    / sqrt(D) at most, which moves a weight by B and the sum by B: 2 B A;
  - sums over n keys in float32, n 2^-23 A; exp2 2^-21;
  - the output is bf16: 2^-8 |o|.
8-bit rows count as the values they stand for, which bf16 holds exactly; where they are
streamed, a weight times its row's scale 2^e is a half in which the largest is 2^11 or
more: off by 2^-11 of itself, and by 2^-25 (half the smallest step) of a code of 448 at
most, together n 2^-27 of the largest p 2^e."""
import math

import pytest
import torch
from test_gpu_shared import draw_rows, make_cache, pk  # noqa: F401

pytestmark = pytest.mark.gpu
D = 128
WAYS = [None, 32768]  # what the host knows of the lengths


def attention(q, k, v, sees, scale=None):
    """(o, bound) in 64 bits of q [t][H][G][D] over k, v [H][n][D], sees [t][n]; scale [H][n]: of 8-bit rows of v."""
    n = k.shape[1]
    if n == 0:
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        return o, o + 1e-30
    qd, k, v = q.double().permute(1, 2, 0, 3), k.double()[:, None], v.double()[:, None]  # [H][G][t][D]
    x = qd @ k.transpose(-1, -2) / math.sqrt(D)
    x = x.masked_fill(~sees, -math.inf)
    w = torch.where(sees.any(-1)[:, None], torch.softmax(x, -1), 0.0)
    o, A = w @ v, w @ v.abs()
    B = 130 * 2.0 ** -24 * ((qd.abs() @ k.abs().transpose(-1, -2)) * sees).amax(-1, keepdim=True) / math.sqrt(D)
    tol = (2.0 ** -8 + 2 * B + n * 2.0 ** -23 + 2.0 ** -21) * A + 2.0 ** -8 * o.abs() + 1e-30
    if scale is not None:
        tol = tol + n * 2.0 ** -27 * (w * scale[:, None, None]).amax(-1, keepdim=True)
    return o.permute(2, 0, 1, 3), tol.permute(2, 0, 1, 3)


def check(out, want, tol, what=""):
    assert torch.isfinite(out).all(), what
    err = (out.double() - want).abs() / tol
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 1, f"{what}: worst error {worst:.3g} of the bound"


def causal(t, n, device="cuda"):
    return torch.arange(n, device=device) <= torch.arange(n - t, n, device=device)[:, None]


def run_prompt(pk, rows, new, past, H, G, seed=0, lens=None, spread=0.75, pad=0, ld=0, bits=16, n_max=None):
    """One call against the formula.  new: tokens of each sequence, past: rows before them (a cache); pad: rows of q and
    out behind the last sequence; ld: elements between tokens beyond the dense ones."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, T = len(new), sum(new) + pad
    start = [sum(new[:i]) for i in range(N + 1)]
    q = torch.randn((T, H * G * D + ld), generator=g, device="cuda").to(torch.bfloat16)[:, :H * G * D]
    q = torch.as_strided(q, (T, H, G, D), (H * G * D + ld, G * D, D, 1))
    out = torch.full((T, H, G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q_start = torch.tensor(start, dtype=torch.int64, device="cuda")
    if rows == "cache":
        lens = lens or [a + b for a, b in zip(new, past)]
        cap = max(512, (max(max(lens), n_max or 0) + 511) // 512 * 512)
        k, v = draw_rows(g, N, H, cap, spread)
        c, vals = make_cache(pk, bits, G, cap, lens, k, v)
        if n_max is not None:
            c.c.n_max = n_max
        a = pk.prompt_args(q, out, q_start, cache=c)
        kv = [(vals[0][i, :, :lens[i]], vals[1][i, :, :lens[i]]) for i in range(N)]
    else:
        k, v = draw_rows(g, 1, H, T, spread)
        k, v = k[0], v[0]  # [H][T][D]
        kv = [(k[:, a:b], v[:, a:b]) for a, b in zip(start, start[1:])]
        if rows == "token":
            x = torch.empty((2, T, H * D + ld), dtype=torch.bfloat16, device="cuda")[..., :H * D].unflatten(-1, (H, D))
            x[0].copy_(k.transpose(0, 1))
            x[1].copy_(v.transpose(0, 1))
            x[:, start[-1]:] = float("nan")  # behind the last sequence
            ks, vs = x[0], x[1]
        else:
            ks, vs = [torch.cat([x[:, a:b].reshape(-1, D) for a, b in zip(start, start[1:])] +
                                [torch.full((pad * H, D), float("nan"), dtype=torch.bfloat16, device="cuda")])
                      for x in (k, v)]
        a = pk.prompt_args(q, out, q_start, ks, vs)
        lens = new
    ws = pk.prompt_workspace(a)
    ws[256:].fill_(0xff)  # nothing in it counts
    pk.bpkv_prompt_attend(a, ws, ws.numel())
    torch.cuda.synchronize()
    assert pk.bpkv_read_status(ws) == 0
    for i in range(N):
        at = slice(start[i], start[i + 1])
        want, tol = attention(q[at], *kv[i], causal(new[i], lens[i]))
        check(out[at], want, tol, f"sequence {i}")
    assert (out[start[-1]:] == 7.0).all(), "rows behind the last sequence"
    return dict(a=a, ws=ws, out=out, q=q, q_start=q_start)


LAYOUTS = ["token", "seq"]


@pytest.mark.parametrize("rows", LAYOUTS)
@pytest.mark.parametrize("t", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_short_prompts(pk, rows, t):
    run_prompt(pk, rows, [t], None, 2, 4, seed=t)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("t", [1, 41, 300])
def test_groups(pk, G, t):
    run_prompt(pk, "seq", [t], None, 3, G, seed=G + t)


@pytest.mark.parametrize("rows", LAYOUTS)
@pytest.mark.parametrize("new", [[5, 0, 1, 130, 64, 257], [0, 0, 3], [700, 1, 800, 0], [1] * 40, [129] * 9])
def test_packed_prompts(pk, rows, new):
    run_prompt(pk, rows, new, None, 2, 4, seed=len(new), pad=3, ld=8)


@pytest.mark.parametrize("G,t", [(1, 2500), (3, 1100), (4, 1025), (7, 801), (8, 2049)])
def test_prompts_that_are_cut(pk, G, t):
    run_prompt(pk, "token", [t, 17, t // 2], None, 2, G, seed=t)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [511]), ([1, 1, 1], [0, 128, 4000]), ([7, 0, 130], [100, 9, 1000]),
                                      ([64, 33], [4090, 127]), ([300, 2], [700, 9000])])
@pytest.mark.parametrize("n_max", WAYS)
def test_behind_cached_rows(pk, bits, new, past, n_max):
    run_prompt(pk, "cache", new, past, 2, 4, seed=sum(new), bits=bits, pad=2, n_max=n_max)


# Runs of 64 tokens: eight, two and four of each sequence, mixtures of them, numbers that are no power of two, one
# token more or less than whole runs, sequences without any.
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,past", [([512] * 4, [3000, 2900, 3100, 0]), ([128, 127, 65, 128], [511, 2000, 8000, 1]),
                                      ([256, 200, 193, 256], [4000, 4500, 100, 777]), ([512, 128, 256, 384], [4096, 3072, 2048, 1024]),
                                      ([320] * 4, [3000] * 4), ([512, 0, 1000, 30], [2000, 0, 5000, 9000]),
                                      ([0, 0, 1025, 0], [5, 0, 6000, 0]), ([512, 512], [30000, 32000]),
                                      ([64, 513, 64, 449], [128, 128, 128, 128])])
def test_runs_side_by_side(pk, bits, new, past):
    """As many rows as sequences may have make runs of a sequence go side by side, however many they do have."""
    run_prompt(pk, "cache", new, past, 2, 4, seed=sum(new) + sum(past), bits=bits, pad=3,
               n_max=(1 << 19) // (2 * len(new)))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("H,G,new,past", [(1, 8, [16] * 8 + [256] * 8, [2000] * 16), (5, 3, [336, 300], [9000, 4000]),
                                          (8, 1, [1024, 700], [3000, 5000]), (3, 7, [216], [70000])])
def test_runs_of_other_groups_side_by_side(pk, bits, H, G, new, past):
    run_prompt(pk, "cache", new, past, H, G, seed=G, bits=bits, n_max=(1 << 19) // (len(new) * H))


def test_runs_side_by_side_give_equal_bits(pk):
    got = run_prompt(pk, "cache", [512, 500, 384], [9000, 8000, 7000], 2, 4, n_max=1 << 16)
    first = got["out"].clone()
    for _ in range(3):
        got["out"].zero_()
        pk.bpkv_prompt_attend(got["a"], got["ws"], got["ws"].numel())
        torch.cuda.synchronize()
        assert torch.equal(got["out"], first)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,n_max", [([40, 3, 200, 5], None), ([40, 3, 2, 5], None), ([40, 3, 2, 5], 32768)])
def test_more_new_tokens_than_rows(pk, bits, new, n_max):
    """Tokens without a row see nothing: zeros."""
    got = run_prompt(pk, "cache", new, None, 2, 4, lens=[10, 0, 150, 600], bits=bits, n_max=n_max)
    assert (got["out"][:30] == 0).all() and (got["out"][40:43] == 0).all()


@pytest.mark.parametrize("rows", LAYOUTS)
@pytest.mark.parametrize("new", [[0, 1, 0, 0, 2, 60], [1] * 33 + [0] * 40 + [1] * 30, [5, 0, 17, 3], [64]])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_few_tokens_of_many_prompts(pk, rows, new, G):
    """Prompts of 64 tokens together at most, which are streamed; empty ones among them."""
    run_prompt(pk, rows, new, None, 3, G, seed=len(new), pad=1, ld=16)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n_max", [0, 100, 2048])
def test_any_bound_of_the_lengths(pk, bits, n_max):
    """n_max sizes the launch and chooses the way, never the result."""
    run_prompt(pk, "cache", [50, 70], [1500, 2000], 2, 4, seed=3, bits=bits, n_max=n_max)


def run_tree(pk, bits, N, t, H, G, lens, seed=0, tree="random", n_max=None):
    """One call against the formula.  n_max: what the host knows of the lengths, which decides whether a cluster streams
    a tree's rows or, above 16 rows, the tensor cores take it (32768)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cap = max(512, (max(max(lens), n_max or 0) + 511) // 512 * 512)
    k, v = draw_rows(g, N, H, cap)
    c, vals = make_cache(pk, bits, G, cap, lens, k, v)
    if n_max is not None:
        c.c.n_max = n_max
    q = torch.randn((N, t, H, G, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((N, t, H, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    if tree == "chain":
        mask, bit = None, torch.ones((t, t), dtype=torch.bool, device="cuda").tril().expand(N, t, t)
    else:
        p = dict(random=0.4, full=1.1, none=-1.0)[tree]
        bit = torch.rand((N, t, t), generator=g, device="cuda") < p
        weight = torch.tensor([1 << j if j < 63 else -(1 << 63) for j in range(t)], device="cuda")
        mask = (bit.long() * weight).sum(-1)
        if t < 64:  # bits past the tree say nothing
            mask |= torch.tensor(-1, device="cuda") << t
    ws = pk.tree_workspace(c, t)
    ws[256:].fill_(0xff)
    fn = pk.bpkv_tree_attend if bits == 16 else pk.bpkv_tree_attend8
    fn(c.c, t, mask, q, out, ws, ws.numel())
    torch.cuda.synchronize()
    assert pk.bpkv_read_status(ws) == 0
    for i in range(N):
        n = lens[i]
        sees = torch.ones((t, max(n, t)), dtype=torch.bool, device="cuda")
        sees[:, max(n, t) - t:] = bit[i]
        sees = sees[:, max(n, t) - n:]  # a short sequence's first nodes have no rows
        want, tol = attention(q[i], vals[0][i, :, :n], vals[1][i, :, :n], sees, None if bits == 16 else vals[2][i, :, :n])
        check(out[i], want, tol, f"sequence {i}")
    return dict(c=c, mask=mask, q=q, out=out, ws=ws, fn=fn)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("tree", ["chain", "random", "full", "none"])
@pytest.mark.parametrize("t", [1, 2, 8, 32, 33, 64])
@pytest.mark.parametrize("n_max", WAYS)
def test_trees(pk, bits, tree, t, n_max):
    run_tree(pk, bits, 3, t, 2, 4, [t, 500, 130 + t], seed=t, tree=tree, n_max=n_max)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("G,t", [(1, 64), (2, 64), (3, 50), (5, 64), (6, 7), (7, 64), (8, 64), (8, 16), (8, 17)])
@pytest.mark.parametrize("n_max", WAYS)
def test_tree_groups(pk, bits, G, t, n_max):
    run_tree(pk, bits, 2, t, 1, G, [1000, 4097], seed=G, n_max=n_max)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n_max", WAYS)
def test_tree_at_every_place_of_a_tile(pk, bits, n_max):
    """The tree begins and ends inside tiles, on their edges and across them."""
    t = 40
    lens = [t + x for x in (0, 1, 23, 63, 64, 65, 87, 88, 89, 90, 127, 128, 129, 200, 216, 217)]
    run_tree(pk, bits, len(lens), t, 1, 4, lens, seed=5, n_max=n_max)
    run_tree(pk, bits, len(lens), 3, 1, 4, [x - t + 3 for x in lens], seed=6, n_max=n_max)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n_max", WAYS)
def test_trees_of_short_sequences(pk, bits, n_max):
    """Fewer rows than nodes: the first nodes have none."""
    run_tree(pk, bits, 5, 20, 2, 4, [0, 1, 19, 20, 21], seed=7, n_max=n_max)
    run_tree(pk, bits, 4, 64, 1, 8, [0, 1, 63, 65], seed=8, n_max=n_max)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("t,lens", [(8, [20000]), (64, [30001, 64]), (3, [5, 9000, 700]), (16, [3000] * 20)])
def test_trees_that_are_cut(pk, bits, t, lens):
    run_tree(pk, bits, len(lens), t, 2, 4, lens, seed=t)


@pytest.mark.parametrize("bits", [16, 8])
def test_equal_calls_give_equal_bits(pk, bits):
    got = run_tree(pk, bits, 3, 30, 2, 4, [9000, 40, 5000], seed=2)
    first = got["out"].clone()
    for _ in range(5):
        got["out"].fill_(float("nan"))
        got["fn"](got["c"].c, 30, got["mask"], got["q"], got["out"], got["ws"], got["ws"].numel())
        assert torch.equal(got["out"], first)
