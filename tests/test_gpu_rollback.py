"""Drafted tokens taken back from a Cache, round after round."""
import pytest
import torch
from test_gpu_shared import draw_rows, pk  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_rounds_than_the_capacity_has_drafts_for(pk):
    """30 rounds of 40 drafted tokens of which 3 are kept, in 512 rows: the bound is set back with the lengths, and the
    rows, planes and scales are those of a cache that never saw what was taken back."""
    H, n, t, keep, rounds = 2, 100, 40, 3, 30
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = draw_rows(g, 1, H, n + t * rounds)
    c, want = pk.Cache(1, H, 4, 512), pk.Cache(1, H, 4, 512)
    c.append(k[:, :, :n].contiguous(), v[:, :, :n].contiguous())
    kept = [torch.arange(n)]
    for r in range(rounds):
        at = n + t * r
        c.append(k[:, :, at:at + t].contiguous(), v[:, :, at:at + t].contiguous())
        kept.append(torch.arange(at, at + keep))
        end = n + keep * (r + 1)
        c.seq_len.fill_(end)
        c.n_max = end
    with pytest.raises(ValueError):
        c.n_max = 513
    # the last block is coded when the next token comes
    last = [x[:, :, n:n + 1].contiguous() for x in (k, v)]
    c.append(*last)
    rows = torch.cat(kept).to("cuda")
    want.append(k[:, :, rows].contiguous(), v[:, :, rows].contiguous())
    want.append(*last)
    end, nb = n + keep * rounds + 1, (n + keep * rounds + 64) // 64
    assert c.seq_len.tolist() == want.seq_len.tolist() == [end] and c.n_max == want.n_max == end
    for name in ("k_rows", "v_rows"):
        assert torch.equal(getattr(c, name)[:, :, :end], getattr(want, name)[:, :, :end])
    for name in ("planes", "scales"):
        assert torch.equal(getattr(c, name)[..., :nb], getattr(want, name)[..., :nb])
