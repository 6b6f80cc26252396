"""A step with more rows than the caller's tables hold (kv4_attn.h, status ROWS): it becomes the step of
its first max_rows rows, in every table, and the attention sees these rows where positions says."""
import numpy as np
import pytest

import kv4_ref as ref
import moe_layer_tail_gb300 as mt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def kept(new, max_rows):
    """What is left of each request's rows."""
    ends = np.minimum(np.cumsum(new), max_rows)
    return np.diff(np.concatenate([[0], ends]))


def run_tables(cached, new, free, table, page, max_rows):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=I32, device="cuda")
    t = dev(table)
    R = len(cached)
    starts, lens, used, st = (torch.full((n,), -3, dtype=I32, device="cuda") for n in (R + 1, R, 1, 1))
    pos = torch.full((max_rows,), -3, dtype=I32, device="cuda")
    slots = torch.full((max_rows,), -3, dtype=torch.int64, device="cuda")
    st.zero_()
    mt.step_tables(dev(cached), dev(new), dev(free) if len(free) else None, t, page, starts, lens, pos, slots,
                   used, status=st)
    return [x.cpu().numpy() for x in (t, starts, lens, pos, slots, used, st)]


@pytest.mark.parametrize("reqs,rows,max_rows,page,n_free", [
    (1, 40, 1, 16, 9), (4, 55, 30, 16, 9), (4, 55, 14, 16, 9), (4, 55, 54, 16, 2), (33, 200, 100, 32, 64),
    (33, 200, 1, 32, 64), (1000, 5000, 2500, 16, 900), (1024, 1024, 1000, 16, 2048), (1024, 3000, 7, 48, 3)])
def test_a_cut_step_is_the_step_of_its_first_rows(reqs, rows, max_rows, page, n_free):
    rng = np.random.default_rng([reqs, rows, max_rows])
    cached = rng.integers(0, 5 * page, reqs)
    new = np.array([14, 40, 1, 0]) if reqs == 4 else rng.multinomial(rows, np.ones(reqs) / reqs)
    if reqs == 4:
        cached = np.array([20, 0, 16, 5])
    width = -(-int((cached + new).max()) // page)
    table = np.full((reqs, width), -7)
    held = -(-cached // page)
    at = 5000
    for r in range(reqs):
        table[r, :held[r]] = np.arange(at, at + held[r])
        at += held[r]
    free = np.arange(n_free)
    left = kept(new, max_rows)
    assert left.sum() == max_rows < new.sum()
    want = list(ref.step_tables(cached, left, free, table, page, max_rows))
    want[6] |= mt.KV4_STATUS_ROWS
    for got, exp in zip(run_tables(cached, new, free, table, page, max_rows), want):
        assert np.array_equal(got, np.atleast_1d(exp))


def test_a_cut_step_through_cache_and_attention():
    """Tables, cache rows and attention of a step of 55 rows in tables of 30, then of the rest: what
    each row sees is its own request up to its position."""
    D, heads, G, page, width, R = 64, 2, 4, 16, 8, 4
    rng = np.random.default_rng(1)
    cache = mt.kv4_cache(40, page, heads, D)
    cache.fill_(255)  # (slots that nothing writes hold NaN)
    table = torch.full((R, width), -1, dtype=I32, device="cuda")
    free = torch.arange(40, dtype=I32, device="cuda")
    lens = torch.zeros(R, dtype=I32, device="cuda")
    todo, hist, taken = np.array([14, 40, 1, 0]), [[] for _ in range(R)], 0
    st = torch.zeros(1, dtype=I32, device="cuda")
    bits = lambda *s: ref.f32_to_bf16(rng.standard_normal(s).astype(np.float32))
    dev = lambda b: torch.from_numpy(b.view(np.int16)).cuda().view(BF)
    for cut in (30, 30):
        n = torch.tensor(todo, dtype=I32, device="cuda")
        starts, kv = (torch.zeros(k, dtype=I32, device="cuda") for k in (R + 1, R))
        pos, used = (torch.zeros(k, dtype=I32, device="cuda") for k in (cut, 1))
        slots = torch.zeros(cut, dtype=torch.int64, device="cuda")
        mt.step_tables(lens, n, free[taken:], table, page, starts, kv, pos, slots, used, status=st)
        q, k, v = bits(cut, heads * G, D), bits(cut, heads, D), bits(cut, heads, D)
        mt.kv4_append(cache, dev(k), dev(v), slots, status=st)
        out = torch.full((cut, heads * G, D), 5.0, dtype=BF, device="cuda")
        mt.kv4_attention(dev(q), cache, table, starts, kv, out, max_new=40, status=st)
        taken += int(used)
        left = kept(todo, cut)
        at = 0
        for r in range(R):
            for _ in range(left[r]):
                assert int(pos[at]) == len(hist[r])
                hist[r].append((k[at], v[at]))
                at += 1
        assert int(st) == (mt.KV4_STATUS_ROWS if left.sum() < todo.sum() else 0)
        assert kv.cpu().tolist() == [len(h) for h in hist] and taken == sum(-(-len(h) // page) for h in hist)
        L = max(len(h) for h in hist)
        K, V = np.zeros((R, heads, L, D)), np.zeros((R, heads, L, D))
        for r in range(R):
            for dst, x in ((K, 0), (V, 1)):
                if hist[r]:
                    dst[r, :, :len(hist[r])] = ref.values(*ref.quantize(np.stack([h[x] for h in hist[r]], 1)))
        want = ref.attention(ref.bf16_to_f64(q), K, V, np.arange(R)[:, None].repeat(L, 1),
                             starts.cpu().numpy(), kv.cpu().numpy(), L, D ** -0.5)
        got = ref.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
        assert len(want) == left.sum()
        for i, (o, avg, spread, total) in want.items():
            assert (np.abs(got[i] - o) <= ref.attention_tolerance(o, avg, spread, total, D)).all(), i
        assert (got[left.sum():] == 5).all()
        lens, todo = kv, todo - left
        st.zero_()
    assert todo.sum() == 0
