"""The measured cases of the serving operators around the exact rows of a KV cache.

Three operators, as one decode step uses them in turn:

  qkv      the projected query, key and value heads of new tokens: RMS norm of
           every query and key head, position rotation, and the rows laid out
           for the caches (bpkv_qkv_rope); with a cache of 8-bit rows the keys
           and values are quantised into it by the same call;
  append8  rows quantised to 8 bits as they are written (bpkv_rows8_append),
  read8    and read back (bpkv_rows8_read);
  attend   decode attention of a batch whose sequences share long prefixes:
           every prefix row is read once for all of its sequences
           (bpkv_shared_attend over bf16 rows, bpkv_shared_attend8 over 8-bit
           rows); without a prefix it is the plain attention of each sequence
           over its own rows.

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
        # one token of one session: latency of a launch
        dict(name="qkv_token", op="qkv", N=1, t=1, H=8, G=4, rot=128, pairs=False, norm=True, q16=False, q8=False,
             pos=32767),
        # one token of each of 32 sessions, straight into the 8-bit rows
        dict(name="qkv_batch_rows8", op="qkv", N=32, t=1, H=8, G=4, rot=128, pairs=False, norm=True, q16=True,
             q8=True, pos=65535),
        # a prompt of 8191 tokens
        dict(name="qkv_prompt", op="qkv", N=1, t=8191, H=8, G=4, rot=128, pairs=False, norm=True, q16=True, q8=False,
             pos=0),
        # rotation of half the channels in neighbouring pairs, no norm, far positions, float queries for the scans
        dict(name="qkv_partial", op="qkv", N=3, t=1365, H=2, G=7, rot=64, pairs=True, norm=False, q16=False, q8=False,
             pos=1000003),
        # one token of each of 32 sessions
        dict(name="append8_step", op="append8", N=32, t=1, H=8, start=4095),
        # a whole context written at once
        dict(name="append8_prompt", op="append8", N=1, t=32768, H=8, start=0),
        # four sessions' rows read back, e.g. to be encoded into another cache
        dict(name="read8_rows", op="read8", N=4, n=8191, H=8, t0=257),
        # one short session: latency
        dict(name="attend_short", op="attend", N=1, H=8, G=4, P=0, plen=0, smax=500, bits=16),
        # 32 sessions over one shared context of 32768 tokens
        dict(name="attend_prefix", op="attend", N=32, H=8, G=4, P=1, plen=32768, smax=1000, bits=16),
        # 128 sessions over a context of 131072 tokens: more products than bytes
        dict(name="attend_wide", op="attend", N=128, H=8, G=4, P=1, plen=131072, smax=512, bits=16),
        # 8-bit rows, two shared contexts, 8 query heads for each KV head
        dict(name="attend8_prefixes", op="attend", N=16, H=4, G=8, P=2, plen=131071, smax=2000, bits=8),
        # 8-bit rows, ragged sessions that share nothing
        dict(name="attend8_ragged", op="attend", N=32, H=8, G=4, P=0, plen=0, smax=16384, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qkv", "qkv", "append8", "read8", "attend", "attend", "attend", "attend"])
    if op == "qkv":
        N = _log_int(rng, 1, 64)
        t = _log_int(rng, 1, 8192 // N)
        pairs, norm = rng.random() < 0.5, rng.random() < 0.7
        q16, q8 = rng.random() < 0.5, rng.random() < 0.4
        return dict(op=op, N=N, t=t, H=rng.choice([1, 2, 5, 8]), G=rng.randint(1, 4), rot=2 * rng.randint(0, 64),
                    pairs=pairs, norm=norm, q16=q16, q8=q8, pos=_log_int(rng, 1, 1 << 20) - 1)
    if op == "append8":
        N = _log_int(rng, 1, 64)
        return dict(op=op, N=N, t=_log_int(rng, 1, 32768 // N), H=rng.randint(1, 8), start=rng.randint(0, 3000))
    if op == "read8":
        N = _log_int(rng, 1, 64)
        return dict(op=op, N=N, n=_log_int(rng, 1, 32768 // N), H=rng.randint(1, 8), t0=rng.randint(0, 3000))
    N = _log_int(rng, 1, 96)
    H, G = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8)
    P = rng.choice([0, 1, 1, 1, 2, 3])
    plen = _log_int(rng, 1, 131072 // max(P, 1)) if P else 0
    # own rows: at most half a million rows of a KV head in all
    smax = _log_int(rng, 1, max(2, min(20000, 500000 // (N * H))))
    # no more products than the largest listed case
    while P and N * G * H * plen > 128 * 4 * 8 * 131072 // 2:
        plen //= 2
    return dict(op=op, N=N, H=H, G=G, P=P, plen=plen, smax=smax, bits=rng.choice([16, 8]))


def _cap(n):
    return max(512, (n + 511) // 512 * 512)


def _lengths(case):
    """Tokens of each sequence's own (ragged, one of them empty in a batch) and of each prefix."""
    N, smax = case["N"], case["smax"]
    own_len = [smax if N == 1 else smax * ((5 * i + N - 1) % N) // (N - 1) for i in range(N)]
    return own_len, [max(1, case["plen"] - 101 * p) for p in range(case["P"])]


def work(case):
    op = case["op"]
    if op == "qkv":
        tok = case["N"] * case["t"]
        H, G = case["H"], case["G"]
        row = 2 * D + 2 if case["q8"] else 4 * D
        q = H * G * D * (2 if case["q16"] else 4)
        return {"bytes": tok * ((G + 2) * H * D * 2 + q + H * row), "flops": tok * (G + 1) * H * D * 7}
    if op in ("append8", "read8"):
        rows = case["N"] * case["H"] * (case["t"] if op == "append8" else case["n"])
        return {"bytes": rows * (4 * D + 2 * D + 2), "flops": rows * 4 * D}
    own_len, plen = _lengths(case)
    N, H, G, P = case["N"], case["H"], case["G"], case["P"]
    row = 4 * D if case["bits"] == 16 else 2 * D + 2
    tokens = sum(own_len) + sum(plen[i % P] for i in range(N)) if P else sum(own_len)
    return {"bytes": H * row * (sum(own_len) + sum(plen[:N])) + 2 * N * H * G * D * 2,
            "flops": 4 * tokens * H * G * D}


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


def _rows(g, shape, spread):
    """Rows of keys (channels of different widths) or values, a few tokens with large keys among them."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    if spread:
        x *= torch.exp(0.75 * torch.randn((shape[0], shape[1], 1, D), generator=g, device=DEVICE))
        n = max(1, shape[2] // 997)
        at = torch.randint(0, shape[2], (n,), generator=g, device=DEVICE)
        x[:, :, at] *= 2.5
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "qkv":
        N, t, H, G, rot = case["N"], case["t"], case["H"], case["G"], case["rot"]
        heads = (G + 2) * H
        s["qkv"] = torch.randn((N, t, heads * D), generator=g, device=DEVICE).mul_(1.5).to(torch.bfloat16)
        s["pos"] = case["pos"] - torch.arange(N, device=DEVICE).clamp(max=case["pos"])
        s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, device=DEVICE, dtype=torch.float64) / max(rot, 1))).float()
        s["qw"] = 1 + 0.3 * torch.randn(D, generator=g, device=DEVICE) if case["norm"] else None
        s["kw"] = 1 + 0.3 * torch.randn(D, generator=g, device=DEVICE) if case["norm"] else None
        s["q_out"] = torch.zeros((N, t, H, G, D), dtype=torch.bfloat16 if case["q16"] else torch.float32, device=DEVICE)
        if case["q8"]:
            _prepare_rows8(s, N, H, _cap(case["pos"] + t))
        else:
            s["k_out"] = torch.zeros((N, H, t, D), dtype=torch.bfloat16, device=DEVICE)
            s["v_out"] = torch.zeros((N, H, t, D), dtype=torch.bfloat16, device=DEVICE)
        if own:
            import bit_plane_kv_encode_gb300 as pk
            s["args"] = pk.qkv_args(s["qkv"], s["q_out"], H, pos=s["pos"], inv_freq=s["inv_freq"], q_weight=s["qw"],
                                    k_weight=s["kw"], eps=1e-6, pairs=case["pairs"], k_out=s.get("k_out"),
                                    v_out=s.get("v_out"), rows8=s.get("cache"))
        return s
    if op == "append8":
        N, t, H = case["N"], case["t"], case["H"]
        s["k"], s["v"] = _rows(g, (N, H, t, D), True), _rows(g, (N, H, t, D), False)
        s["start"] = case["start"] - torch.arange(N, device=DEVICE).clamp(max=case["start"])
        _prepare_rows8(s, N, H, _cap(case["start"] + t))
        return s
    if op == "read8":
        N, n, H = case["N"], case["n"], case["H"]
        cap = _cap(case["t0"] + n)
        _prepare_rows8(s, N, H, cap, _rows(g, (N, H, cap, D), True), _rows(g, (N, H, cap, D), False))
        s["seq_len"].copy_(case["t0"] + n - torch.arange(N, device=DEVICE).clamp(max=n - 1))
        s["k_out"] = torch.zeros((N, H, n, D), dtype=torch.bfloat16, device=DEVICE)
        s["v_out"] = torch.zeros((N, H, n, D), dtype=torch.bfloat16, device=DEVICE)
        return s
    N, H, G, P = case["N"], case["H"], case["G"], case["P"]
    own_len, plen = _lengths(case)
    cap, pcap = _cap(case["smax"]), _cap(case["plen"])
    s["q"] = torch.randn((N, H, G, D), generator=g, device=DEVICE).to(torch.bfloat16)
    s["len"] = torch.tensor(own_len, device=DEVICE, dtype=torch.int64)
    s["rows"] = [_rows(g, (N, H, cap, D), True), _rows(g, (N, H, cap, D), False)]
    s["prefix_of"] = None
    if P:
        s["plen"] = torch.tensor(plen, device=DEVICE, dtype=torch.int64)
        s["prows"] = [_rows(g, (P, H, pcap, D), True), _rows(g, (P, H, pcap, D), False)]
        if P > 1:
            s["prefix_of"] = (torch.arange(N, device=DEVICE) % P).to(torch.int32)
    if case["bits"] == 8:
        for name in ("rows", "prows") if P else ("rows",):
            s[name] = [x for r in s[name] for x in _quantise(r)]  # k8, kexp, v8, vexp
    s["out"] = torch.zeros((N, H, G, D), dtype=torch.bfloat16, device=DEVICE)
    if own:
        import bit_plane_kv_encode_gb300 as pk

        def cache(n, capacity, rows, lengths, longest):
            if case["bits"] == 8:
                c = pk.Rows8(n, H, G, capacity)
                for dst, src in zip((c.k8, c.kexp, c.v8, c.vexp), rows):
                    dst.copy_(src.view(torch.uint8))
            else:
                c = pk.Cache(n, H, G, capacity)
                c.k_rows.copy_(rows[0])
                c.v_rows.copy_(rows[1])
            c.seq_len.copy_(lengths)
            c.c.n_max = longest
            return c

        s["cache"] = cache(N, cap, s["rows"], s["len"], case["smax"])
        s["prefix"] = cache(P, pcap, s["prows"], s["plen"], case["plen"]) if P else None
        s["ws"] = pk.shared_workspace(s["cache"], s["prefix"])
    return s


def _prepare_rows8(s, N, H, cap, k=None, v=None):
    """The buffers of a cache of 8-bit rows: the framework's own where it runs, plain ones else."""
    if own:
        import bit_plane_kv_encode_gb300 as pk
        c = s["cache"] = pk.Rows8(N, H, 1 if s["case"]["op"] != "qkv" else s["case"]["G"], cap)
        s["k8"], s["kexp"], s["v8"], s["vexp"], s["seq_len"] = c.k8, c.kexp, c.v8, c.vexp, c.seq_len
    else:
        for name in ("k8", "v8"):
            s[name] = torch.empty((N, H, cap, D), dtype=torch.uint8, device=DEVICE)
        for name in ("kexp", "vexp"):
            s[name] = torch.empty((N, H, cap), dtype=torch.uint8, device=DEVICE)
        s["seq_len"] = torch.empty(N, dtype=torch.int64, device=DEVICE)
    s["seq_len"].zero_()
    for x, codes, exps in ((k, "k8", "kexp"), (v, "v8", "vexp")):
        if x is None:
            s[codes].zero_()
            s[exps].zero_()
        else:
            c, e = _quantise(x)
            s[codes].copy_(c.view(torch.uint8))
            s[exps].copy_(e)


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
        if op == "qkv":
            pk.bpkv_qkv_rope(s["args"])
            if c["q8"]:
                return dict(q=s["q_out"], **_rows8_out(s))
            return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
        if op == "append8":
            pk.bpkv_rows8_append(s["cache"].c, s["k"], s["v"], c["t"], s["start"])
            return _rows8_out(s)
        if op == "read8":
            pk.bpkv_rows8_read(s["cache"].c, c["t0"], c["n"], s["k_out"], s["v_out"])
            return dict(k=s["k_out"], v=s["v_out"])
        attend = pk.bpkv_shared_attend8 if c["bits"] == 8 else pk.bpkv_shared_attend
        attend(s["prefix"].c if s["prefix"] else None, s["prefix_of"], s["cache"].c, s["q"], s["out"], s["ws"],
               s["ws"].numel())
        return s["out"]
    if op == "qkv":
        q, k, v = _plain_qkv(s, c)
        if c["q8"]:
            _plain_append(s, k, v, s["pos"])
            return dict(q=q, **_rows8_out(s))
        return dict(q=q, k=k, v=v)
    if op == "append8":
        _plain_append(s, s["k"], s["v"], s["start"])
        return _rows8_out(s)
    if op == "read8":
        return dict(k=_plain_read(s, c, "k8", "kexp"), v=_plain_read(s, c, "v8", "vexp"))
    return _plain_attend(s, c)


def _plain_qkv(s, c):
    N, t, H, G, rot = c["N"], c["t"], c["H"], c["G"], c["rot"]
    x = s["qkv"].view(N, t, (G + 2) * H, D).float()
    q, k, v = x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:]
    # angles in 64 bits: positions reach a million, where 32 bits leave no fraction of a turn
    at = (s["pos"][:, None] + torch.arange(t, device=DEVICE)).double()
    angle = at[..., None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    q, k = _plain_head(q, s["qw"], cos, sin, rot, c["pairs"]), _plain_head(k, s["kw"], cos, sin, rot, c["pairs"])
    q = q.view(N, t, H, G, D)
    return (q.to(torch.bfloat16) if c["q16"] else q, k.to(torch.bfloat16).transpose(1, 2).contiguous(),
            v.to(torch.bfloat16).transpose(1, 2).contiguous())


def _plain_head(x, w, cos, sin, rot, pairs):
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s, k, v, start):
    N, H, t, _ = k.shape
    at = start[:, None, None] + torch.arange(t, device=DEVICE)
    n, h = torch.arange(N, device=DEVICE)[:, None, None], torch.arange(H, device=DEVICE)[:, None]
    for x, codes, exps in ((k, "k8", "kexp"), (v, "v8", "vexp")):
        y, e = _quantise(x)
        s[codes][n, h, at] = y.view(torch.uint8)
        s[exps][n, h, at] = e
    s["seq_len"].copy_(start + t)


def _values(codes, exps):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps.int()[..., None] - 127)


def _plain_read(s, c, codes, exps):
    at = slice(c["t0"], c["t0"] + c["n"])
    x = _values(s[codes][:, :, at], s[exps][:, :, at])
    there = torch.arange(c["t0"], c["t0"] + c["n"], device=DEVICE) < s["seq_len"][:, None]
    return torch.where(there[:, None, :, None], x, 0.0).to(torch.bfloat16)


def _plain_rows(rows, n):
    if len(rows) == 2:
        return rows[0][:, :, :n].float(), rows[1][:, :, :n].float()
    return _values(rows[0][:, :, :n], rows[1][:, :, :n]), _values(rows[2][:, :, :n], rows[3][:, :, :n])


def _plain_attend(s, c):
    N, H, G, P = c["N"], c["H"], c["G"], c["P"]
    q = s["q"].float() / math.sqrt(D)
    k, v = _plain_rows(s["rows"], c["smax"])
    x = q @ k.transpose(-1, -2)  # [N, H, G, smax]
    there = torch.arange(c["smax"], device=DEVICE) < s["len"][:, None]
    x = torch.where(there[:, None, None], x, -math.inf)
    if P:
        pk, pv = _plain_rows(s["prows"], c["plen"])
        n = s["plen"]
        if P == 1:  # all sequences' heads against the one prefix
            y = q.permute(1, 0, 2, 3).reshape(H, N * G, D) @ pk[0].transpose(-1, -2)
            y = y.view(H, N, G, -1).transpose(0, 1)
            n = n.expand(N)
        else:
            of = s["prefix_of"].long()
            pv, n = pv[of], n[of]
            y = q @ pk[of].transpose(-1, -2)
        there = torch.arange(c["plen"], device=DEVICE) < n[:, None]
        x = torch.cat((torch.where(there[:, None, None], y, -math.inf), x), -1)
        del y
    m = x.amax(-1, keepdim=True)
    x = torch.where(m == -math.inf, 0.0, torch.exp(x - m))
    norm = x.sum(-1, keepdim=True)
    o = x[..., c["plen"]:] @ v
    if P == 1:
        y = x[..., :c["plen"]].transpose(0, 1).reshape(H, N * G, -1) @ pv[0]
        o += y.view(H, N, G, D).transpose(0, 1)
    elif P:
        o += x[..., :c["plen"]] @ pv
    return torch.where(norm > 0, o / norm, 0.0).to(torch.bfloat16)


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits."""
    s, c = prepare(case, seed), case
    if c["op"] == "qkv":
        return _exact_qkv(s, c)
    if c["op"] == "append8":
        return _exact_append(s, s["k"].double(), s["v"].double(), s["start"])
    if c["op"] == "read8":
        return _exact_read(s, c)
    return _exact_attend(s, c)


def _exact_qkv(s, c):
    N, t, H, G, rot = c["N"], c["t"], c["H"], c["G"], c["rot"]
    x = s["qkv"].double().reshape(N, t, G * H + 2 * H, D)
    where = s["pos"].double().reshape(N, 1) + torch.arange(t, device=DEVICE, dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                       where[:, :, None, None] * s["inv_freq"].double())

    def head(z, w):
        if w is not None:
            z = z / torch.sqrt(z.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        first = torch.arange(0, rot, 2, device=DEVICE) if c["pairs"] else torch.arange(rot // 2, device=DEVICE)
        second = first + 1 if c["pairs"] else first + rot // 2
        r = torch.complex(z[..., first], z[..., second]) * turn
        z = z.clone()
        z[..., first], z[..., second] = r.real, r.imag
        return z

    q = head(x[:, :, :G * H], s["qw"]).reshape(N, t, H, G, D)
    k = head(x[:, :, G * H:G * H + H], s["kw"]).permute(0, 2, 1, 3)
    v = x[:, :, G * H + H:].permute(0, 2, 1, 3)
    if not c["q8"]:
        return dict(q=q, k=k, v=v)
    # a code is the rounding of a rounded key: the exact key has none of its own
    return dict(q=q, k8=None, kscale=None, seq_len=s["pos"] + t,
                **{n: x for n, x in _exact_append(s, k, v, s["pos"]).items() if n[0] == "v"})


def _exact_append(s, k, v, start):
    N, H, t, _ = k.shape
    got = {}
    for name, x in (("k", k), ("v", v)):
        a = x.abs().amax(-1)
        a = torch.where(a > 0, a, 2.0 ** E_MIN)
        e = torch.round(torch.log2(a / E4M3_MAX))  # the smallest e with a <= 448 2^e is this one or the next
        e = torch.where(a <= E4M3_MAX * torch.exp2(e), e, e + 1)
        e = torch.where(a <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
        y = x / torch.exp2(e)[..., None]
        # e4m3: three bits after the leading one, down to steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
        codes = torch.zeros(s["k8"].shape, dtype=torch.float64, device=DEVICE)
        scale = torch.full(s["kexp"].shape, 2.0 ** -127, dtype=torch.float64, device=DEVICE)  # of the zero byte
        for i in range(N):
            at = int(start[i])
            codes[i, :, at:at + t] = y[i].clamp(-E4M3_MAX, E4M3_MAX)
            scale[i, :, at:at + t] = torch.exp2(e[i])
        got[name + "8"], got[name + "scale"] = codes, scale
    return dict(got, seq_len=start + t)


def _exact_read(s, c):
    got = {}
    for name in ("k", "v"):
        x = torch.zeros((c["N"], c["H"], c["n"], D), dtype=torch.float64, device=DEVICE)
        for i in range(c["N"]):
            n = max(0, min(c["n"], int(s["seq_len"][i]) - c["t0"]))
            at = slice(c["t0"], c["t0"] + n)
            scale = torch.exp2(s[name + "exp"][i, :, at].double() - 127)
            x[i, :, :n] = s[name + "8"][i, :, at].view(torch.float8_e4m3fn).double() * scale[..., None]
        got[name] = x
    return got


def _exact_attend(s, c):
    N, H, G, P = c["N"], c["H"], c["G"], c["P"]
    own_len, plen = _lengths(c)

    def rows(r, i, h, n):
        if len(r) == 2:
            return r[0][i, h, :n].double(), r[1][i, h, :n].double()
        return tuple(r[j][i, h, :n].double() * torch.exp2(r[j + 1][i, h, :n].double() - 127)[:, None] for j in (0, 2))

    def part(q, k, v):
        """Maximum, sum and weighted values of a set of rows."""
        x = q @ k.T / D ** 0.5
        m = x.amax(-1)
        p = torch.exp(x - m[:, None])
        return m, p.sum(-1), p @ v

    out = torch.zeros((N, H, G, D), dtype=torch.float64, device=DEVICE)
    for h in range(H):
        of_prefix = {}
        for p in range(P):
            mine = [i for i in range(N) if i % P == p]
            if mine:
                m, l, o = part(s["q"][mine, h].double().reshape(-1, D), *rows(s["prows"], p, h, plen[p]))
                for j, i in enumerate(mine):
                    of_prefix[i] = (m[j * G:j * G + G], l[j * G:j * G + G], o[j * G:j * G + G])
        for i in range(N):
            parts = [of_prefix[i]] if i in of_prefix else []
            if own_len[i]:
                parts.append(part(s["q"][i, h].double(), *rows(s["rows"], i, h, own_len[i])))
            if parts:
                top = torch.stack([m for m, _, _ in parts]).amax(0)
                w = [torch.exp(m - top) for m, _, _ in parts]
                total = sum(a * l for a, (_, l, _) in zip(w, parts))
                out[i, h] = sum(a[:, None] * o for a, (_, _, o) in zip(w, parts)) / total[:, None]
    return out
