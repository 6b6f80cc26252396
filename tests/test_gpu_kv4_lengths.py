"""Lengths and row starts of the attention over the MXFP4 cache (kv4_attn.h) that only the device sees:
what a call too large for its ranges leaves."""
import numpy as np
import pytest

import moe_layer_tail_gb300 as mt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def test_a_call_of_too_many_tiles_gives_nan_and_says_so():
    # 32 kv heads x 2^27 tiles; nothing of the cache is read.  The rows of both requests are NaN, the
    # others stay, and a call that is not too large is right again with the same tables
    D, heads, G, page, width = 64, 32, 2, 1024, (1 << 21)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cache = mt.kv4_cache(2, page, heads, D)
    k = torch.randn((20, heads, D), generator=g, device="cuda").to(BF)
    mt.kv4_append(cache, k, k, torch.arange(page, page + 20, device="cuda"))
    table = torch.zeros((2, width), dtype=I32, device="cuda")
    table[1, 0] = 1
    starts = torch.tensor([1, 3, 4], dtype=I32, device="cuda")
    q = torch.randn((5, heads * G, D), generator=g, device="cuda").to(BF)
    for st in (torch.zeros(1, dtype=I32, device="cuda"), None):
        out = torch.full((5, heads * G + 8, D), 5.0, dtype=BF, device="cuda")[:, :heads * G]
        lens = torch.tensor([(1 << 31) - 2000, 20], dtype=I32, device="cuda")
        mt.kv4_attention(q, cache, table, starts, lens, out, max_new=2, status=st)
        assert bool(out[1:4].isnan().all()) and bool((out[0] == 5).all()) and bool((out[4] == 5).all())
        assert bool((out._base[:, heads * G:] == 5).all())
        assert st is None or int(st) == mt.KV4_STATUS_BAD_LENGTH
    lens[0] = 2
    st = torch.zeros(1, dtype=I32, device="cuda")
    both, alone = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    mt.kv4_attention(q, cache, table, starts, lens, both, max_new=2, status=st)
    mt.kv4_attention(q, cache, table[1:], starts[1:], lens[1:], alone, max_new=2, status=st)
    assert int(st) == 0 and torch.equal(both[3], alone[3]) and not bool(both[1:4].isnan().any())
