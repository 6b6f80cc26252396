"""Lengths and row starts of the attention over the MXFP4 cache (kv4_attn.h) that only the device sees:
what a call too large for its ranges leaves, a length past its table row, row starts that descend."""
import numpy as np
import pytest

import kv4_ref as ref
import moe_layer_tail_gb300 as mt
from test_gpu_kv4 import Step

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


@pytest.mark.parametrize("D,G,new", [(64, 8, 1), (128, 4, 3), (256, 16, 2)])
def test_a_length_past_its_table_row_is_cut_to_it(D, G, new):
    # request 1 says 113 tokens and its row of the table holds 7 pages of 16: the values are those of 112
    s = Step(18, [100, 80, 41], new, G, 1, D, 16, garbage=False)
    s.table[1] = [s.table[1, 0], s.table[1, 1], s.table[1, 2], s.table[1, 3], s.table[1, 4], s.table[0, 2], s.table[0, 3]]
    for said in (113, 100000, (1 << 31) - 1):
        s.lens[1] = said
        got = s.run()
        assert s.status == mt.KV4_STATUS_BAD_LENGTH
        s.lens[1] = 112
        s.check(got)
    assert np.array_equal(got, s.run()) and s.status == 0


def test_row_starts_that_descend_or_pass_the_rows_skip_their_requests_alone():
    s = Step(19, [20, 30, 40, 25], 1, 8, 1, 64, 16, pad=3)
    K, V = ref.decode(s.cache)
    for starts, rows in (([0, 2, 1, 99, 99], {0: (0, 0, 2), 1: (0, 0, 2)}),  # 1 descends, 2 ends and 3 lies past the rows
                         ([5, 3, 4, 4, 7], {3: (1, 3, 4), 4: (3, 4, 7), 5: (3, 4, 7), 6: (3, 4, 7)}),
                         ([-1, 2, 3, 4, 8], {2: (1, 2, 3), 3: (2, 3, 4)})):
        s.starts[:] = starts
        got = s.run(max_new=2)
        assert s.status == mt.KV4_STATUS_BAD_LENGTH
        for i in range(len(got)):
            if i not in rows:
                assert (got[i] == 5).all()
                continue
            r, first, end = rows[i]
            want = ref.attention(ref.bf16_to_f64(s.q), K, V, s.table[r:r + 1], np.array([first, end]),
                                 s.lens[r:r + 1], 16, 64 ** -0.5)[i]
            assert (np.abs(got[i] - want[0]) <= ref.attention_tolerance(*want, 64)).all(), (starts, i)
