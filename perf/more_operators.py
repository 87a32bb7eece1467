"""The measured cases of the attention of several new tokens of a sequence at once.

Three operators, as a serving loop uses them around a KV cache:

  prompt   causal attention of whole prompts of different lengths, packed one
           behind the other, over their own keys and values (rows "token":
           [T][H][D], "seq": each prompt's [H][t][D] as bpkv_qkv_rope leaves
           it), or of a prompt's next tokens over the rows of a cache that
           they end (rows "cache", of bf16 or 8 bits): bpkv_prompt_attend;
  tree     attention of a tree of drafted tokens, the last t rows of each
           sequence of a cache: a node sees all rows before the tree, and of
           the tree those that its mask names: bpkv_tree_attend over bf16
           rows, bpkv_tree_attend8 over 8-bit rows;
  accept   of the drafted tokens those that were accepted, as many as each
           sequence has, quantised behind its rows: bpkv_rows8_accept.

Where ``own`` is false the operators are computed in elementary torch
operations in 32 bits; where it is true by the library's calls.
"""
import math

import torch

own = False
DEVICE = "cuda"

D = 128          # channels of a head
E4M3_MAX = 448.0
E_MIN, E_MAX = -48, 32  # exponents of a row's scale


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a short question to one session: latency
        dict(name="prompt_short", op="prompt", N=1, t=17, H=8, G=4, rows="seq", bits=16, past=0),
        # one prompt of 8191 tokens
        dict(name="prompt_8191", op="prompt", N=1, t=8191, H=8, G=4, rows="token", bits=16, past=0),
        # sixteen prompts of 251 to 4001 tokens, packed
        dict(name="prompt_packed", op="prompt", N=16, t=4001, H=8, G=4, rows="seq", bits=16, past=0),
        # two key heads with seven query heads each, which do not divide a tile
        dict(name="prompt_group7", op="prompt", N=3, t=1365, H=2, G=7, rows="token", bits=16, past=0),
        # a long document at once
        dict(name="prompt_16383", op="prompt", N=1, t=16383, H=8, G=4, rows="seq", bits=16, past=0),
        # the next 512 tokens of four prompts, 32256 tokens of each in the cache before them
        dict(name="chunk_cache", op="prompt", N=4, t=512, H=8, G=4, rows="cache", bits=16, past=32256),
        # a question of 1000 tokens behind a context of 100000 in 8-bit rows
        dict(name="chunk_cache8", op="prompt", N=1, t=1000, H=8, G=4, rows="cache", bits=8, past=100000),
        # eight drafted tokens of one session: latency
        dict(name="tree_small", op="tree", N=1, t=8, H=8, G=4, smax=2000, bits=16),
        # trees of 32 nodes of sixteen sessions
        dict(name="tree_batch", op="tree", N=16, t=32, H=8, G=4, smax=8192, bits=16),
        # wide trees behind long contexts in 8-bit rows
        dict(name="tree8_long", op="tree", N=4, t=64, H=8, G=4, smax=131071, bits=8),
        # the accepted ones of 16 drafted tokens of each of 32 sessions
        dict(name="accept_step", op="accept", N=32, t=16, H=8, start=4095),
        # prompts of different lengths, padded, appended at once
        dict(name="accept_prompts", op="accept", N=16, t=2047, H=8, start=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "chunk", "chunk", "tree", "tree", "tree", "accept"])
    if op == "accept":
        N = _log_int(rng, 1, 64)
        return dict(op=op, N=N, t=_log_int(rng, 1, 32768 // N), H=rng.randint(1, 8), start=rng.randint(0, 3000))
    H, G = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8)
    if op == "tree":
        N, t = _log_int(rng, 1, 64), rng.randint(1, 64)
        # at most a million rows of a KV head in all
        return dict(op=op, N=N, t=t, H=H, G=G, smax=max(t, _log_int(rng, 1, min(131072, 1000000 // (N * H)))),
                    bits=rng.choice([16, 8]))
    N = _log_int(rng, 1, 24)
    if op == "prompt":
        t = _log_int(rng, 1, 16383)
        case = dict(op="prompt", N=N, t=t, H=H, G=G, rows=rng.choice(["token", "seq"]), bits=16, past=0)
    else:
        t = _log_int(rng, 1, 2048)
        case = dict(op="prompt", N=N, t=t, H=H, G=G, rows="cache", bits=rng.choice([16, 8]),
                    past=_log_int(rng, 1, min(131072, 1000000 // (N * H))))
    # no more products than the largest listed case
    while work(case)["flops"] > 2 * D * 32 * 16383 * 16384:
        case["t"] = max(1, case["t"] // 2)
        case["past"] //= 2
    return case


def _cap(n):
    return max(512, (n + 511) // 512 * 512)


def _prompts(case):
    """New tokens of each sequence, and the rows of it before them (ragged in a batch)."""
    N, t, past = case["N"], case["t"], case["past"]
    if N == 1:
        return [t], [past]
    new = [max(1, t * (1 + (5 * i + N - 1) % N) // N) for i in range(N)]
    return new, [past * (1 + (3 * i + N - 1) % N) // N for i in range(N)]


def _trees(case):
    """Rows of each sequence, the tree's among them."""
    N, t, smax = case["N"], case["t"], case["smax"]
    return [smax if N == 1 else t + (smax - t) * ((5 * i + N - 1) % N) // (N - 1) for i in range(N)]


def _accepted(case):
    """Where each sequence's accepted tokens go, and how many they are."""
    N, t = case["N"], case["t"]
    return [max(0, case["start"] - i) for i in range(N)], [t if N == 1 else t * ((5 * i + N - 1) % N) // (N - 1)
                                                            for i in range(N)]


def work(case):
    op = case["op"]
    H = case["H"]
    row8 = 2 * D + 2
    if op == "accept":
        n = sum(_accepted(case)[1])
        return {"bytes": n * H * (4 * D + row8) + n * 4, "flops": n * H * 4 * D}
    G = case["G"]
    row = 4 * D if case["bits"] == 16 else row8
    if op == "prompt":
        new, past = _prompts(case)
        pairs = sum(t * p + t * (t + 1) // 2 for t, p in zip(new, past))
        return {"bytes": H * row * (sum(new) + sum(past)) + 2 * sum(new) * H * G * D * 2, "flops": 4 * D * H * G * pairs}
    lens, t, N = _trees(case), case["t"], case["N"]
    # every node over the rows before the tree and, of a random tree, some three nodes above it
    pairs = sum((n - t) * t for n in lens) + N * t * min(t, 4)
    return {"bytes": H * row * sum(lens) + 2 * N * t * H * G * D * 2 + N * t * 8, "flops": 4 * D * H * G * pairs}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _quantise(x):
    """bf16 rows [..., D] -> e4m3 codes and one power-of-two scale for each row, as its biased exponent (e8m0)."""
    xf = x.float()
    a = xf.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(E_MIN, E_MAX)  # 448 = 0.875 * 2^9
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN))
    y = torch.ldexp(xf, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _keys(g, shape):
    """Rows [..., n, D] of keys: channels of different widths, a few tokens with large keys among them."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    x *= torch.exp(0.75 * torch.randn(D, generator=g, device=DEVICE))
    n = max(1, shape[-2] // 997)
    at = torch.randint(0, shape[-2], (n,), generator=g, device=DEVICE)
    x[..., at, :] *= 2.5
    return x.to(torch.bfloat16)


def _values(g, shape):
    return torch.randn(shape, generator=g, device=DEVICE).to(torch.bfloat16)


def _ints(x, dtype=torch.int64):
    return torch.tensor(x, device=DEVICE, dtype=dtype)


def _prepare_cache(s, case, g, lens, group):
    """Rows of a cache of bf16 or 8-bit rows, in the framework's own cache where it runs."""
    N, H, cap = len(lens), case["H"], _cap(max(lens))
    s["len"] = _ints(lens)
    rows = [_keys(g, (N, H, cap, D)), _values(g, (N, H, cap, D))]
    if case["bits"] == 8:
        rows = [x.view(torch.uint8) for r in rows for x in _quantise(r)]  # k8, kexp, v8, vexp
    s["rows"] = rows
    if own:
        import bit_plane_kv_encode_gb300 as pk
        c = s["cache"] = (pk.Rows8 if case["bits"] == 8 else pk.Cache)(N, H, group, cap)
        for dst, src in zip((c.k8, c.kexp, c.v8, c.vexp) if case["bits"] == 8 else (c.k_rows, c.v_rows), rows):
            dst.copy_(src)
        c.seq_len.copy_(s["len"])
        c.c.n_max = max(lens)


def prepare(case, seed):
    g = _gen(seed)
    op, N, t, H = case["op"], case["N"], case["t"], case["H"]
    s = dict(case=case)
    if own:
        import bit_plane_kv_encode_gb300 as pk
    if op == "prompt":
        G = case["G"]
        new, past = _prompts(case)
        T = sum(new)
        start = [sum(new[:i]) for i in range(N + 1)]
        s["q"] = torch.randn((T, H, G, D), generator=g, device=DEVICE).to(torch.bfloat16)
        s["out"] = torch.zeros((T, H, G, D), dtype=torch.bfloat16, device=DEVICE)
        s["q_start"] = _ints(start)
        if case["rows"] == "cache":
            _prepare_cache(s, case, g, [a + b for a, b in zip(new, past)], G)
        else:
            k, v = _keys(g, (H, T, D)), _values(g, (H, T, D))
            if case["rows"] == "token":
                s["k"], s["v"] = k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()
            else:
                s["k"], s["v"] = [torch.cat([x[:, a:b].reshape(-1, D) for a, b in zip(start, start[1:])])
                                  for x in (k, v)]
        if own:
            s["args"] = pk.prompt_args(s["q"], s["out"], s["q_start"], s.get("k"), s.get("v"), cache=s.get("cache"))
            s["ws"] = pk.prompt_workspace(s["args"])
        return s
    if op == "tree":
        G = case["G"]
        s["q"] = torch.randn((N, t, H, G, D), generator=g, device=DEVICE).to(torch.bfloat16)
        s["out"] = torch.zeros((N, t, H, G, D), dtype=torch.bfloat16, device=DEVICE)
        _prepare_cache(s, case, g, _trees(case), G)
        # a random tree: every node but the roots hangs on one before it, and sees itself and what is above it
        up = (torch.rand((N, t), generator=g, device=DEVICE) * torch.arange(t, device=DEVICE)).long().tolist()
        masks = []
        for n in range(N):
            m = []
            for j in range(t):
                m.append((m[up[n][j]] if j else 0) | 1 << j)
            masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        s["tree"] = _ints(masks)
        if own:
            s["ws"] = pk.tree_workspace(s["cache"], t)
        return s
    start, count = _accepted(case)
    s["k"], s["v"] = _keys(g, (N, H, t, D)), _values(g, (N, H, t, D))
    s["start"], s["count"] = _ints(start), _ints(count, torch.int32)
    # accepted tokens in their order, one way down the tree
    s["path"] = torch.zeros((N, t), dtype=torch.int32, device=DEVICE)
    for i, n in enumerate(count):
        if n:
            s["path"][i, :n] = torch.randperm(t, generator=g, device=DEVICE)[:n].sort().values
    cap = _cap(case["start"] + t)
    if own:
        c = s["cache"] = pk.Rows8(N, H, 1, cap)
        s["k8"], s["kexp"], s["v8"], s["vexp"], s["seq_len"] = c.k8, c.kexp, c.v8, c.vexp, c.seq_len
    else:
        for name in ("k8", "v8"):
            s[name] = torch.empty((N, H, cap, D), dtype=torch.uint8, device=DEVICE)
        for name in ("kexp", "vexp"):
            s[name] = torch.empty((N, H, cap), dtype=torch.uint8, device=DEVICE)
        s["seq_len"] = torch.empty(N, dtype=torch.int64, device=DEVICE)
    for name in ("k8", "v8", "kexp", "vexp", "seq_len"):
        s[name].zero_()
    return s


# ----------------------------------------------------------------------- run

def _rows8_out(s):
    return dict(k8=s["k8"].view(torch.float8_e4m3fn), kscale=s["kexp"].view(torch.float8_e8m0fnu),
                v8=s["v8"].view(torch.float8_e4m3fn), vscale=s["vexp"].view(torch.float8_e8m0fnu),
                seq_len=s["seq_len"])


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import bit_plane_kv_encode_gb300 as pk
        if op == "prompt":
            pk.bpkv_prompt_attend(s["args"], s["ws"], s["ws"].numel())
            return s["out"]
        if op == "tree":
            attend = pk.bpkv_tree_attend8 if c["bits"] == 8 else pk.bpkv_tree_attend
            attend(s["cache"].c, c["t"], s["tree"], s["q"], s["out"], s["ws"], s["ws"].numel())
            return s["out"]
        pk.bpkv_rows8_accept(s["cache"].c, s["k"], s["v"], c["t"], s["start"], s["path"], s["count"])
        return _rows8_out(s)
    if op == "accept":
        return _plain_accept(s, c)
    out = []
    for i in range(c["N"]):
        if op == "prompt":
            new, past = _prompts(c)
            t, n = new[i], new[i] + past[i]
            a = sum(new[:i])
            q = s["q"][a:a + t]
            k, v = _plain_rows(s, c, i, a, n)
            # new token j sees the rows up to its own
            sees = torch.arange(n, device=DEVICE) <= torch.arange(n - t, n, device=DEVICE)[:, None]
        else:
            n, t = _trees(c)[i], c["t"]
            q = s["q"][i]
            k, v = _plain_rows(s, c, i, 0, n)
            bits = (s["tree"][i][:, None] >> torch.arange(t, device=DEVICE)) & 1
            sees = torch.cat((torch.ones((t, n - t), dtype=torch.bool, device=DEVICE), bits > 0), 1)
        out.append(_plain_attend(q, k, v, sees, op == "prompt"))
    return torch.cat(out) if op == "prompt" else torch.stack(out)


def _plain_rows(s, c, i, first, n):
    """Keys and values of sequence i, [H][n][D] in 32 bits; first: its first token among the packed ones."""
    if "rows" not in s:
        if c["rows"] == "token":
            return [s[x][first:first + n].transpose(0, 1).float() for x in "kv"]
        return [s[x][first * c["H"]:(first + n) * c["H"]].view(c["H"], n, D).float() for x in "kv"]
    r = s["rows"]
    if c["bits"] == 16:
        return [x[i, :, :n].float() for x in r]
    return [torch.ldexp(r[j][i, :, :n].view(torch.float8_e4m3fn).float(), r[j + 1][i, :, :n].int()[..., None] - 127)
            for j in (0, 2)]


def _plain_attend(q, k, v, sees, causal):
    """q [t][H][G][D] over k, v [H][n][D], token j over the rows sees[j]; some tokens at a time."""
    t, H, G, _ = q.shape
    n = k.shape[1]
    step = max(1, (1 << 29) // (H * G * n))
    out = torch.empty_like(q)
    for a in range(0, t, step):
        b = min(t, a + step)
        m = n - t + b if causal else n  # rows that any of them sees
        x = q[a:b].permute(1, 0, 2, 3).reshape(H, (b - a) * G, D).float() / math.sqrt(D) @ k[:, :m].transpose(1, 2)
        x = torch.where(sees[a:b, None, :m], x.view(H, b - a, G, m), -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        norm = x.sum(-1, keepdim=True)
        o = (x.view(H, (b - a) * G, m) @ v[:, :m]).view(H, b - a, G, D)
        out[a:b] = torch.where(norm > 0, o / norm, 0.0).permute(1, 0, 2, 3).to(q.dtype)
    return out


def _plain_accept(s, c):
    N, H, t = c["N"], c["H"], c["t"]
    n, h, j = torch.arange(N, device=DEVICE)[:, None, None], torch.arange(H, device=DEVICE)[:, None], \
        torch.arange(t, device=DEVICE)
    there = j < s["count"][:, None, None]  # [N, 1, t]
    # what is not accepted goes nowhere: to the row it has already
    at = torch.where(there, s["start"][:, None, None] + j, 0)
    node = s["path"].long()[:, None].expand(N, H, t)
    where = [x.expand(N, H, t)[there.expand(N, H, t)] for x in (n, h, at)]
    for x, codes, exps in ((s["k"], "k8", "kexp"), (s["v"], "v8", "vexp")):
        y, e = _quantise(x[n, h, node][there.expand(N, H, t)])
        s[codes][tuple(where)] = y.view(torch.uint8)
        s[exps][tuple(where)] = e
    s["seq_len"].copy_(s["start"] + s["count"])
    return _rows8_out(s)


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits."""
    s, c = prepare(case, seed), case
    if c["op"] == "accept":
        return _exact_accept(s, c)
    H, G, N = c["H"], c["G"], c["N"]
    got = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    scale = D ** -0.5
    lens = s["len"].tolist() if "len" in s else None
    for i in range(N):
        for h in range(H):
            if c["op"] == "prompt":
                a, b = (int(x) for x in s["q_start"][i:i + 2])
                dst, q = got[a:b, h], s["q"][a:b, h].double()
            else:
                dst, q = got[i, :, h], s["q"][i, :, h].double()
            t = q.shape[0]
            n = lens[i] if lens else t
            if lens is None and c["rows"] == "token":
                k, v = s["k"][a:b, h].double(), s["v"][a:b, h].double()
            elif lens is None:
                k, v = (s[x][H * a + h * t:H * a + h * t + t].double() for x in "kv")
            elif c["bits"] == 16:
                k, v = (x[i, h, :n].double() for x in s["rows"])
            else:
                r = s["rows"]
                k, v = (r[j][i, h, :n].view(torch.float8_e4m3fn).double()
                        * torch.exp2(r[j + 1][i, h, :n].double() - 127)[:, None] for j in (0, 2))
            for x in range(0, t, 512):
                y = min(t, x + 512)
                m = n - t + y if c["op"] == "prompt" else n
                logit = torch.einsum("tgd,nd->gtn", q[x:y], k[:m]) * scale
                hide = torch.zeros((y - x, m), dtype=torch.bool, device=DEVICE)
                if c["op"] == "prompt":
                    hide[:, n - t + x:] = torch.triu(torch.ones((y - x, y - x), dtype=torch.bool, device=DEVICE), 1)
                else:
                    for j in range(t):
                        hide[:, n - t + j] = (s["tree"][i, x:y] >> j) % 2 == 0
                p = torch.softmax(logit.masked_fill(hide, -math.inf), -1)
                dst[x:y] = torch.einsum("gtn,nd->tgd", p, v[:m])
    return got


def _exact_accept(s, c):
    N, H, t = c["N"], c["H"], c["t"]
    got = {}
    start, count = s["start"].tolist(), s["count"].tolist()
    for name in "kv":
        codes = torch.zeros(s["k8"].shape, dtype=torch.float64, device=DEVICE)
        scale = torch.full(s["kexp"].shape, 2.0 ** -127, dtype=torch.float64, device=DEVICE)  # of the zero byte
        for i in range(N):
            x = s[name][i][:, s["path"][i, :count[i]].long()].double()
            a = x.abs().amax(-1)
            a = torch.where(a > 0, a, 2.0 ** E_MIN)
            e = torch.round(torch.log2(a / E4M3_MAX))  # the smallest e with a <= 448 2^e is this one or the next
            e = torch.where(a <= E4M3_MAX * torch.exp2(e), e, e + 1)
            e = torch.where(a <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
            y = x / torch.exp2(e)[..., None]
            # e4m3: three bits after the leading one, down to steps of 2^-9
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            at = slice(start[i], start[i] + count[i])
            codes[i, :, at] = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
            scale[i, :, at] = torch.exp2(e)
        got[name + "8"], got[name + "scale"] = codes, scale
    return dict(got, seq_len=s["start"] + s["count"])
