"""Sequences so long that a CTA is busy with one run of new tokens for longer than
any single wait of the kernel may take."""
import pytest
import torch
from test_gpu_shared import pk  # noqa: F401

pytestmark = pytest.mark.gpu
D = 128


def test_a_run_that_takes_seconds(pk):
    """Behind 204.8 million 8-bit rows of one KV head every CTA has one run of 1.6 million tiles, some 2.8 s, while a
    wait is given up after 4e9 cycles (2 s) without a step: what is waited for until the run's end must not count as
    that.  The first 128 rows, and 128 near the end, share all of the weight (logits 181, the others 0): the mean of
    their values, 1 and 3, is exact."""
    H, G, T, cap = 1, 8, 152 * 32, 1600000 * 128
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("the rows take 53 GB")
    c = pk.Rows8(1, H, G, cap)
    for x in (c.k8, c.v8):
        x.zero_()
    for x in (c.kexp, c.vexp):
        x.fill_(127)
    end = cap - T - 7
    for a, v in ((0, 0x38), (end - 128, 0x44)):  # 1 and 3
        c.k8[0, 0, a:a + 128] = 0x38
        c.kexp[0, 0, a:a + 128] = 127 + 4
        c.v8[0, 0, a:a + 128] = v
    c.seq_len.fill_(cap)
    c.n_max = cap
    q = torch.ones((T, H, G, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    a = pk.prompt_args(q, out, torch.tensor([0, T], device="cuda"), cache=c)
    ws = pk.prompt_workspace(a)
    pk.bpkv_prompt_attend(a, ws, ws.numel())
    assert pk.bpkv_read_status(ws) == 0
    assert (out == 2).all()
    del a, c, x
    torch.cuda.empty_cache()
