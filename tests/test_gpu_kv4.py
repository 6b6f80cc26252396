"""The decode step's attention block (kv4_attn.h) on the GPU against float64 restatements
(kv4_ref.py): cache rows byte for byte, tables number for number, the norm with rotation and the
attention within tolerances that follow from their roundings; masks, garbage in unwritten slots,
NaN in masked places, bad pages and lengths, strides, streams, graphs, and a run of all of them
into the layer tail."""
import numpy as np
import pytest

import kv4_ref as ref
import moe_layer_tail_gb300 as mt
import oracle
from moe_layer_tail_gb300 import inputs as gen
from parity import bf16_step, check_parity

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(BF)


def to_bits(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def normal_bits(rng, *shape):
    return ref.f32_to_bf16(rng.standard_normal(shape).astype(np.float32))


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------- cache rows ----

@pytest.mark.parametrize("D,heads,page,rows", [(64, 1, 16, 1), (64, 3, 48, 33), (128, 8, 64, 40),
                                               (128, 1, 1024, 17), (256, 2, 32, 50)])
def test_append_and_read(D, heads, page, rows):
    rng = np.random.default_rng([D, heads, page, rows])
    pages = -(-2 * rows // page) + 2
    k, v = normal_bits(rng, rows, heads, D), normal_bits(rng, rows, heads, D)
    # blocks at the format's edges: zeros, -0, one large channel, the smallest and largest values,
    # ties of the rounding, infinities and NaN
    k[0, 0, :32] = 0
    v[0, 0, :32] = 0x8000
    k[-1, -1, 32:64] = ref.f32_to_bf16(np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 4))
    v[-1, -1, :32] = 0x0001
    k[rows // 2, 0, 5] = 0x7F7F
    v[rows // 2, -1, D - 1] = 0xFF80
    k[rows // 3, -1, D - 32] = 0x7FC1
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    expect = rng.integers(0, 256, (pages, heads, page // 16, 17 * D), dtype=np.uint8)
    cache = torch.from_numpy(expect.copy()).cuda()
    for r in range(rows):
        ref.write_row(expect, slots[r], k[r], v[r])
    # rows are slices of a packed projection
    packed = torch.cat([to_dev(k).flatten(1), to_dev(v).flatten(1)], 1)
    kd, vd = packed[:, :heads * D].view(rows, heads, D), packed[:, heads * D:].view(rows, heads, D)
    st = status_word()
    mt.kv4_append(cache, kd, vd, torch.from_numpy(slots).cuda(), status=st)
    assert np.array_equal(cache.cpu().numpy(), expect)
    ko = torch.full((rows, heads, D), 7.0, dtype=BF, device="cuda")
    vo = torch.full_like(ko, 7.0)
    mt.kv4_read(cache, torch.from_numpy(slots).cuda(), ko, vo, status=st)
    K, V = ref.decode(expect)
    for got, full in ((ko, K), (vo, V)):
        want = full[slots // page, :, slots % page]
        assert np.array_equal(ref.bf16_to_f64(to_bits(got)), want, equal_nan=True)
    assert int(st) == 0


@pytest.mark.parametrize("D,heads", [(64, 1), (64, 5), (128, 3), (256, 2)])
def test_rows_side_by_side_in_their_tiles(D, heads):
    # runs of rows as prompts leave them: on and off the tiles' boundaries, over pages, with breaks,
    # gaps and an end inside a tile; what is not theirs stays
    rng = np.random.default_rng([D, heads])
    page, pages = 32, 12
    runs = [(0, 64), (64 + 5, 40), (200, 3), (211, 4), (250, 1), (256, 27), (300, 37)]
    slots = np.concatenate([np.arange(a, a + n) for a, n in runs]).astype(np.int64)
    for skip in ((), (7, 100, 101)):
        at = slots.copy()
        at[list(skip)] = -1
        rows = len(at)
        k, v = normal_bits(rng, rows, heads, D), normal_bits(rng, rows, heads, D)
        expect = rng.integers(0, 256, (pages, heads, page // 16, 17 * D), dtype=np.uint8)
        cache = torch.from_numpy(expect.copy()).cuda()
        for r in range(rows):
            if at[r] >= 0:
                ref.write_row(expect, at[r], k[r], v[r])
        st = status_word()
        mt.kv4_append(cache, to_dev(k), to_dev(v), torch.from_numpy(at).cuda(), status=st)
        assert np.array_equal(cache.cpu().numpy(), expect) and int(st) == 0
    # a run into the end of the cache: its last rows have no slot
    at = np.arange(pages * page - 9, pages * page + 3).astype(np.int64)
    for r in range(9):
        ref.write_row(expect, at[r], k[r], v[r])
    mt.kv4_append(cache, to_dev(k)[:12], to_dev(v)[:12], torch.from_numpy(at).cuda(), status=st)
    assert np.array_equal(cache.cpu().numpy(), expect) and int(st) == mt.KV4_STATUS_BAD_SLOT


@pytest.mark.parametrize("D,heads,rows", [(64, 1, 21000), (128, 5, 17000), (128, 8, 9800), (256, 3, 13001),
                                          (64, 12, 13100)])
def test_rows_that_fill_the_gpu(D, heads, rows):
    # enough rows for the forms that take several heads of a row together; rows without a slot between
    rng = np.random.default_rng([D, heads, rows])
    page = 64
    pages = -(-rows // page) + 1
    slots = rng.permutation(pages)[np.arange(rows) // page] * page + np.arange(rows) % page
    slots[rng.random(rows) < 0.01] = -1
    at = torch.from_numpy(slots.astype(np.int64)).cuda()
    k, v = (torch.from_numpy(normal_bits(rng, rows, heads, D).view(np.int16)).cuda().view(BF) for _ in range(2))
    one, two = mt.kv4_cache(pages, page, heads, D), mt.kv4_cache(pages, page, heads, D)
    st = status_word()
    mt.kv4_append(one, k, v, at, status=st)
    for r in range(0, rows, 200):  # (small calls take another form, checked above)
        mt.kv4_append(two, k[r:r + 200], v[r:r + 200], at[r:r + 200], status=st)
    assert torch.equal(one, two) and int(one.count_nonzero()) > 0
    outs = [[torch.full((rows, heads, D), 7.0, dtype=BF, device="cuda") for _ in range(2)] for _ in range(2)]
    mt.kv4_read(one, at, *outs[0], status=st)
    for r in range(0, rows, 200):
        mt.kv4_read(one, at[r:r + 200], *(o[r:r + 200] for o in outs[1]), status=st)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]) and int(st) == 0


def test_rows_without_a_slot_are_left_alone():
    rng = np.random.default_rng(1)
    before = rng.integers(0, 256, (2, 2, 1, 17 * 64), dtype=np.uint8)
    cache = torch.from_numpy(before.copy()).cuda()
    x = to_dev(normal_bits(rng, 4, 2, 64))
    st = status_word()
    slots = torch.tensor([-1, 32, -5, 1 << 40], device="cuda")
    mt.kv4_append(cache, x, x, slots, status=st)
    assert np.array_equal(cache.cpu().numpy(), before) and int(st) == mt.KV4_STATUS_BAD_SLOT
    out = torch.full((4, 2, 64), 3.0, dtype=BF, device="cuda")
    st.zero_()
    mt.kv4_read(cache, slots, out, out, status=st)
    assert bool((out == 3).all()) and int(st) == mt.KV4_STATUS_BAD_SLOT
    st.zero_()
    mt.kv4_append(cache, x, x, torch.tensor([-1, -1, 31, -1], device="cuda"), status=st)
    ref.write_row(before, 31, to_bits(x)[2], to_bits(x)[2])
    assert np.array_equal(cache.cpu().numpy(), before) and int(st) == 0


# ------------------------------------------------------------------------- step tables ----

@pytest.mark.parametrize("reqs,rows,page,longest", [(1, 1, 16, 0), (1, 5, 64, 63), (7, 40, 16, 33),
                                                    (32, 32, 64, 4000), (33, 64, 48, 100),
                                                    (1000, 5000, 32, 200), (1024, 1024, 16, 50)])
def test_step_tables(reqs, rows, page, longest):
    rng = np.random.default_rng([reqs, rows, page])
    cached = rng.integers(0, longest + 1, reqs)
    cached[rng.integers(reqs)] = 0
    new = rng.multinomial(rows - rows // 10, np.ones(reqs) / reqs)  # some without rows, some padding
    if reqs > 4:
        cached[2], new[2] = page, 1          # a full page, then one more row
        cached[3], new[3] = page - 1, 1      # the last slot of a page
    width = -(-int((cached + new).max()) // page) + 1
    held = -(-cached // page)
    pages = rng.permutation(int(held.sum()) + reqs + rows)
    table = np.full((reqs, width), -7)
    at = 0
    for r in range(reqs):
        table[r, :held[r]] = pages[at:at + held[r]]
        at += held[r]
    free = pages[at:]
    max_rows = max(rows, int(new.sum()))
    want = ref.step_tables(cached, new, free, table, page, max_rows)
    _check_tables(cached, new, free, table, page, max_rows, want)


def _check_tables(cached, new, free, table, page, max_rows, want, stride=3):
    reqs, width = table.shape
    i32 = torch.int32

    def dev(x, t=i32):
        return torch.tensor(np.asarray(x), dtype=t, device="cuda")

    wide = torch.full((reqs, width + stride), -9, dtype=i32, device="cuda")
    wide[:, :width] = dev(table)
    outs = [torch.full((n + 4,), -3, dtype=t, device="cuda") for n, t in
            ((reqs + 1, i32), (reqs, i32), (max_rows, i32), (max_rows, torch.int64), (1, i32))]
    st = status_word()
    mt.step_tables(dev(cached), dev(new), dev(free) if len(free) else None, wide[:, :width], page,
                   *[o[:-4] for o in outs], status=st)
    assert np.array_equal(wide[:, :width].cpu().numpy(), want[0])
    assert bool((wide[:, width:] == -9).all()) and all(bool((o[-4:] == -3).all()) for o in outs)
    for got, exp in zip(outs, want[1:6]):
        assert np.array_equal(got[:-4].cpu().numpy(), np.atleast_1d(exp))
    assert int(st) == want[6]


@pytest.mark.parametrize("case", ["pages", "no_pages", "length", "width", "rows", "empty"])
def test_step_tables_reports(case):
    cached, new = np.array([20, 0, 16, 5]), np.array([14, 40, 1, 0])
    table = np.array([[4, 5, -1, -1], [-1, -1, -1, -1], [6, -1, -1, -1], [7, -1, -1, -1]])
    free, max_rows = np.arange(20, 30), 64
    if case == "pages":
        free = free[:2]
    elif case == "no_pages":
        free = free[:0]
    elif case == "length":
        cached[0], new[2] = -1, -4
    elif case == "width":
        new[1] = 65
    elif case == "rows":
        max_rows = 30
    elif case == "empty":
        new[:] = 0
    want = ref.step_tables(cached, new, free, table, 16, max_rows)
    assert want[6] == {"pages": 32, "no_pages": 32, "length": 16, "width": 16, "rows": 64, "empty": 0}[case]
    _check_tables(cached, new, free, table, 16, max_rows, want)


# --------------------------------------------------------------------- norm and rotation ----

@pytest.mark.parametrize("T,hq,hk,D,rot,inter,far", [
    (1, 1, 1, 16, 16, False, 100), (1, 128, 8, 128, 128, False, 1 << 20),
    (5, 6, 2, 64, 32, True, 4000), (3, 5, 0, 96, 96, False, 1 << 31),
    (33, 16, 3, 192, 64, False, 1 << 31), (32, 64, 4, 256, 256, True, 1 << 31),
    (7, 40, 8, 256, 64, False, 1 << 17), (700, 8, 1, 128, 0, False, 10), (9, 3, 3, 112, 16, True, 50),
    # many heads to a warp: one run of a ring and more
    (3000, 40, 3, 64, 32, True, 1 << 31), (900, 20, 3, 256, 256, False, 1 << 17),
    (8000, 64, 8, 16, 16, False, 1 << 20), (2500, 33, 7, 48, 32, False, 1 << 10)])
def test_qk_norm_rope(T, hq, hk, D, rot, inter, far):
    rng = np.random.default_rng([T, hq, D, rot])
    w = (hq + hk) * D
    packed = ref.f32_to_bf16(rng.standard_normal((T, w + 24)).astype(np.float32)
                             * np.exp2(rng.integers(-20, 20, (T, 1))))
    packed[0, :D] = 0  # a head of zeros
    gq = ref.f32_to_bf16(1 + 0.1 * rng.standard_normal(D).astype(np.float32))
    gk = ref.f32_to_bf16(1 + 0.1 * rng.standard_normal(D).astype(np.float32))
    pos = rng.integers(0, far, T)
    pos[0] = far - 1
    freq = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    dev = to_dev(packed)
    q, k = dev[:, :hq * D].view(T, hq, D), dev[:, hq * D:w].view(T, hk, D)
    eps = 1e-6
    posd = torch.tensor(pos, dtype=torch.int32, device="cuda")
    freqd = torch.from_numpy(freq).cuda() if rot else None

    def check(got, cols, heads, gamma):
        x = ref.bf16_to_f64(packed[:, cols]).reshape(T, heads, D)
        g = None if gamma is None else ref.bf16_to_f64(gamma)
        want, mag = ref.norm_rope(x, g, pos, freq if rot else np.zeros(0, np.float32), eps, inter)
        # one rounding to bf16 (2^-8 of the value at most); the norm's fp32 sum of D squares,
        # reciprocal root and two products, the angle (fp32 after the reduction: 2^-22 of a turn
        # for the fp32 fraction and the sine's own error; 2^-28 for the oracle's far angles) and
        # the rotation's two products: D/8 + 16 steps of 2^-24 of the pair, and 2 pi 2^-24
        tol = 2.0 ** -8 * np.abs(want) + (D / 8 + 32) * 2.0 ** -24 * mag + 1e-40
        err = np.abs(ref.bf16_to_f64(to_bits(got)).reshape(T, heads, D) - want)
        assert (err <= tol).all(), float((err - tol).max())

    qo = torch.full((T, hq, D), 9.0, dtype=BF, device="cuda")
    ko = torch.full((T, hk, D), 9.0, dtype=BF, device="cuda") if hk else None
    mt.qk_norm_rope(q, k if hk else None, to_dev(gq), to_dev(gk) if hk else None, posd, freqd, qo, ko,
                    eps=eps, interleaved=inter)
    check(qo, slice(0, hq * D), hq, gq)
    if hk:
        check(ko, slice(hq * D, w), hk, gk)
    if not rot:  # (positions are not needed then)
        again = torch.empty_like(qo)
        mt.qk_norm_rope(q, None, to_dev(gq), None, None, None, again, None, eps=eps)
        assert torch.equal(again, qo)
    # without a query norm, and in place in the packed tensor
    mt.qk_norm_rope(q, k if hk else None, None, to_dev(gk) if hk else None, posd, freqd, q,
                    k if hk else None, eps=eps, interleaved=inter)
    check(q, slice(0, hq * D), hq, None)
    if hk:
        assert torch.equal(k, ko)
    assert np.array_equal(to_bits(dev)[:, w:], packed[:, w:])


# ----------------------------------------------------------------------------- attention ----

class Step:
    """A cache with random pages, some of them unwritten garbage, and one step's query rows."""

    def __init__(self, seed, lens, new, G, heads, D, page, spread=1.0, garbage=True, pad=2):
        rng = np.random.default_rng([seed, D, G, page])
        self.D, self.page = D, page
        self.lens = np.array(lens)
        n = np.broadcast_to(np.array(new), self.lens.shape)
        self.starts = np.concatenate([[0], np.cumsum(n)])
        held = -(-self.lens // page)
        width = max(1, int(held.max()))
        pages = int(held.sum()) + 2
        perm = rng.permutation(pages)
        self.table = np.full((len(lens), width), -1)
        self.cache = (rng.integers(0, 256, (pages, heads, page // 16, 17 * D), dtype=np.uint8)
                      if garbage else np.zeros((pages, heads, page // 16, 17 * D), np.uint8))
        k, v = normal_bits(rng, pages, heads, page, D), normal_bits(rng, pages, heads, page, D)
        written = np.zeros((pages, page), bool)
        at = 0
        for r, h in enumerate(held):
            self.table[r, :h] = perm[at:at + h]
            for e in range(h):
                written[perm[at + e], :min(page, self.lens[r] - e * page)] = True
            at += h
        clean = np.zeros_like(self.cache)
        ref.fill(clean, k, v)
        kc, vc, ks, vs = ref.offsets(D)
        for p, s in zip(*np.nonzero(written)):
            tile, t = divmod(int(s), 16)
            for o in (kc[t], vc[t], ks[t], vs[t]):
                self.cache[p, :, tile, o] = clean[p, :, tile, o]
        T = int(self.starts[-1]) + pad  # rows behind the last request
        self.q = ref.f32_to_bf16(spread * rng.standard_normal((T, heads * G, D)).astype(np.float32))

    def run(self, window=0, sinks=0, scale=None, max_new=None, stride=8, **kw):
        T, Hq, D = self.q.shape
        dev = torch.zeros((T, Hq * D + stride), dtype=BF, device="cuda")
        dev[:, :Hq * D] = to_dev(self.q).flatten(1)
        q = dev[:, :Hq * D].view(T, Hq, D)
        buf = torch.full((T, Hq * D + stride), 5.0, dtype=BF, device="cuda")
        out = buf[:, :Hq * D].view(T, Hq, D)
        st = status_word()
        i32 = torch.int32
        new = int(np.diff(self.starts).max(initial=1))
        mt.kv4_attention(q, torch.from_numpy(self.cache).cuda(),
                         torch.tensor(self.table, dtype=i32, device="cuda"),
                         torch.tensor(self.starts, dtype=i32, device="cuda"),
                         torch.tensor(self.lens, dtype=i32, device="cuda"), out, scale=scale,
                         window=window, sinks=sinks, max_new=max_new or max(new, 1), status=st, **kw)
        torch.cuda.synchronize()
        assert bool((buf[:, Hq * D:] == 5).all())
        self.status = int(st)
        return ref.bf16_to_f64(to_bits(out))

    def check(self, got, window=0, sinks=0, scale=None):
        K, V = ref.decode(self.cache)
        want = ref.attention(ref.bf16_to_f64(self.q), K, V, self.table, self.starts, self.lens,
                             self.page, scale or self.D ** -0.5, window, sinks)
        for i, (out, avg, spread, total) in want.items():
            tol = ref.attention_tolerance(out, avg, spread, total, self.D)
            bad = ~(np.abs(got[i] - out) <= tol) & ~(np.isnan(got[i]) & np.isnan(out))
            assert not bad.any(), (i, int(bad.sum()), float(np.nanmax(np.abs(got[i] - out) / tol)))
        assert (got[int(self.starts[-1]):] == 5).all()  # no request's rows: left as they were


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,heads", [(1, 3), (8, 1), (5, 2), (16, 2), (12, 1), (40, 1)])
def test_attention_heads(D, G, heads):
    s = Step(1, [1, 17, 300], 1, G, heads, D, 16)
    s.check(s.run())
    assert s.status == 0


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 129, 255, 513, 1000])
def test_attention_lengths(L):
    s = Step(2, [L], 1, 8, 2, 128, 64)
    s.check(s.run())


@pytest.mark.parametrize("page", [16, 32, 48, 112, 1024])
@pytest.mark.parametrize("new", [1, 2, 3, 4])
def test_attention_rows_of_a_request(page, new):
    s = Step(3, [new, 40, 333, 16], new, 6, 2, 64, page)
    s.check(s.run())
    assert s.status == 0


@pytest.mark.parametrize("D,G,new", [(64, 16, 4), (128, 16, 4), (256, 16, 4), (128, 8, 9), (64, 3, 70)])
def test_attention_many_rows(D, G, new):
    s = Step(4, [new, 200, 75], new, G, 1, D, 32)
    s.check(s.run())


@pytest.mark.parametrize("D,G,heads,new,lens", [
    (64, 256, 1, 1, [70, 3]), (128, 1, 256, 1, [40]), (256, 1, 100, 1, [33, 1]), (64, 2, 255, 1, [18]),
    (128, 4, 1, 513, [513]), (64, 1, 2, 400, [400, 1100]), (256, 16, 1, 4, [900, 30, 2500]),
    (256, 40, 2, 1, [300, 1300]), (256, 3, 1, 100, [640])])
def test_attention_at_the_limits_of_heads_and_rows(D, G, heads, new, lens):
    s = Step(40, lens, new, G, heads, D, 16)
    s.check(s.run())
    s.check(s.run(max_new=1))  # an estimate that is off changes the cut, not what is computed


def test_rows_before_the_first_request_and_wide_strides():
    s = Step(41, [50, 20, 35], [2, 0, 1], 8, 2, 64, 16, pad=3)
    s.starts = s.starts + 2  # two rows and the last one belong to nobody
    got = s.run(stride=2048)
    s.check(got)
    assert (got[:2] == 5).all() and (got[5:] == 5).all()


def test_attention_ragged_rows_and_empty_requests():
    s = Step(5, [5, 100, 3, 0, 257, 64], [2, 0, 3, 0, 1, 5], 8, 2, 128, 16)
    s.check(s.run(max_new=1))
    a = s.run(max_new=1)
    s.check(s.run(max_new=64))
    assert np.array_equal(a, s.run(max_new=1))


def test_attention_a_request_shorter_than_its_rows():
    # the first rows stand before the first token: they see nothing and come out as zeros
    s = Step(6, [2, 0, 30], [4, 3, 2], 4, 1, 64, 16)
    got = s.run()
    s.check(got)
    assert (got[:2] == 0).all() and (got[4:7] == 0).all() and s.status == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (33, 0), (64, 5), (200, 17),
                                          (300, 100), (5000, 4), (40, 1 << 30), ((1 << 31) - 1, 3)])
@pytest.mark.parametrize("new", [1, 3])
def test_attention_window(window, sinks, new):
    s = Step(7, [new, 50, 400, 129, 16], new, 8, 1, 64, 16)
    s.check(s.run(window=window, sinks=sinks), window=window, sinks=sinks)


def test_attention_peaked_and_large_queries():
    s = Step(8, [500, 90], 1, 8, 1, 128, 16, spread=40.0)
    s.check(s.run())
    # rows of very different magnitude, a row of zeros, subnormal queries
    s = Step(9, [300, 300, 300, 300], 1, 4, 1, 64, 16)
    s.q[0] = ref.f32_to_bf16(ref.bf16_to_f64(s.q[0]) * 2.0 ** 60)
    s.q[1] = ref.f32_to_bf16(ref.bf16_to_f64(s.q[1]) * 2.0 ** -100)
    s.q[2] = 0
    s.q[3] = 0x0003
    s.check(s.run())
    s.check(s.run(scale=3.0), scale=3.0)


@pytest.mark.parametrize("D,G,new", [(64, 16, 2), (128, 8, 1), (128, 16, 1), (128, 40, 1), (256, 16, 1)])
def test_attention_scores_that_outgrow_the_first_step(D, G, new):
    # keys that grow (and shrink) by octaves every 128 tokens: the running maximum moves far, in
    # the first parts of a request as in its later ones
    _, _, ks, _ = ref.offsets(D)
    for grow in ((0, 5, 6, 3, 7, 0, 8, 9), (8, 0, 4, 2, 9, 1, 0, 10)):
        s = Step(30, [900, 260], new, G, 1, D, 16)
        for r in range(2):
            for e in range(-(-int(s.lens[r]) // 16)):
                at = s.cache[s.table[r, e], 0, 0]
                at[ks] = np.where(at[ks] == 255, 255, np.minimum(at[ks].astype(int) + grow[e // 8], 200))
        s.check(s.run())


def test_attention_rows_that_see_nothing_of_their_first_steps():
    s = Step(31, [5000, 700], [300, 200], 1, 2, 64, 16)
    for window, sinks in ((17, 0), (1, 0), (250, 3)):
        s.check(s.run(window=window, sinks=sinks), window=window, sinks=sinks)


def test_nan_in_one_of_many_parts():
    s = Step(32, [40000], 1, 8, 1, 64, 64, garbage=False)
    _, _, ks, vs = ref.offsets(64)
    page, off = divmod(30001, 64)
    row = s.cache[s.table[0, page], 0, off // 16]
    keep = row[vs[off % 16, 1]]
    row[vs[off % 16, 1]] = 255
    got = s.run()
    s.check(got)
    assert np.isnan(got[0, :, 32:]).all() and not np.isnan(got[0, :, :32]).any()
    row[vs[off % 16, 1]] = keep
    row[ks[off % 16, 0]] = 255
    assert np.isnan(s.run()[0]).all()


def test_attention_value_scales_far_apart():
    # value blocks between 2^-100 and 2^100 in every order, in one tile and from tile to tile
    rng = np.random.default_rng(10)
    s = Step(11, [700, 64], 1, 8, 1, 128, 16)
    _, _, ks, vs = ref.offsets(128)
    for lo, hi in ((27, 227), (120, 150), (110, 128)):
        s.cache[:, :, :, vs] = rng.integers(lo, hi, s.cache[:, :, :, vs].shape)
        s.check(s.run())


def test_attention_key_scales_far_apart():
    rng = np.random.default_rng(12)
    s = Step(13, [300, 64], 1, 8, 1, 64, 16)
    _, _, ks, vs = ref.offsets(64)
    s.cache[:, :, :, ks] = rng.integers(1, 130, s.cache[:, :, :, ks].shape)
    s.check(s.run())


@pytest.mark.parametrize("what", ["keys", "values"])
def test_nan_in_the_cache_stays_with_the_rows_that_see_it(what):
    s = Step(14, [40, 100], 3, 8, 2, 128, 16)
    _, _, ks, vs = ref.offsets(128)
    at = ks if what == "keys" else vs
    page, off = s.table[0, 39 // 16], 39 % 16   # the last token: only the last of three rows
    s.cache[page, 0, 0, at[off, 1]] = 255
    got = s.run()
    s.check(got)
    assert not np.isnan(got[:2]).any() and np.isnan(got[2, :8]).any()
    assert not np.isnan(got[2, 8:]).any() and not np.isnan(got[3:6]).any()
    # behind a window: nobody sees it
    s = Step(15, [40], 1, 8, 1, 128, 16)
    s.cache[s.table[0, 0], 0, 0, at[3, 2]] = 255
    got = s.run(window=20)
    s.check(got, window=20)
    assert not np.isnan(got[:1]).any()


def test_nan_and_infinite_queries_stay_in_their_rows():
    s = Step(16, [70, 70], 2, 4, 1, 64, 16)
    clean = s.run()
    s.q[1, 2, 5] = 0x7FC0
    s.q[2, 0, 9] = 0x7F80
    got = s.run()
    assert np.isnan(got[1, 2]).all() and np.isnan(got[2, 0]).all()
    got[1, 2], got[2, 0] = clean[1, 2], clean[2, 0]
    assert np.array_equal(got, clean)


def test_bad_pages_and_lengths_are_reported():
    s = Step(17, [100, 80], 1, 8, 1, 64, 16)
    s.table[0, 2], s.table[1, 0] = -1, s.cache.shape[0]
    got = s.run()
    s.check(got)
    assert s.status == mt.KV4_STATUS_BAD_PAGE
    s = Step(18, [100, 80], 1, 8, 1, 64, 16)
    s.lens[1] = 113  # the table holds 7 pages of 16: cut to 112
    got = s.run()
    assert s.status & mt.KV4_STATUS_BAD_LENGTH
    s = Step(19, [20, 30, 40], 1, 8, 1, 64, 16, pad=0)
    s.starts[:] = [0, 2, 1, 99]
    got = s.run(max_new=1)
    assert s.status == mt.KV4_STATUS_BAD_LENGTH  # requests 1, 2 are skipped; row 2 is nobody's
    assert (got[2] == 5).all()


@pytest.mark.parametrize("D,G,heads,L", [(128, 8, 1, 70001), (64, 16, 2, 40007), (256, 4, 1, 30011)])
def test_long_context_is_split_and_joined(D, G, heads, L):
    s = Step(20, [L], 1, G, heads, D, 64, garbage=False)
    got = s.run()
    s.check(got)
    assert np.array_equal(got, s.run())  # the same call gives the same bits


def test_many_requests():
    rng = np.random.default_rng(21)
    s = Step(21, rng.integers(0, 90, 1024), 1, 4, 1, 64, 16, garbage=False)
    s.check(s.run())


def test_many_requests_of_many_wide_rows():
    rng = np.random.default_rng(22)
    s = Step(22, rng.integers(5, 60, 270), 5, 5, 1, 256, 16, garbage=False)
    s.check(s.run())


def test_slots_past_32_bits_of_bytes():
    # a cache of 5 GB whose last pages lie past 2^32 bytes
    D, heads, page = 128, 8, 64
    n = 5 * (1 << 30) // (heads * page // 16 * 17 * D)
    cache = mt.kv4_cache(n, page, heads, D)
    rng = np.random.default_rng(22)
    L = 100
    k, v = normal_bits(rng, L, heads, D), normal_bits(rng, L, heads, D)
    table = np.array([[n - 1, n - 2]])
    pos = np.arange(L)
    slots = torch.tensor(table[0, pos // page] * page + pos % page, device="cuda")
    mt.kv4_append(cache, to_dev(k), to_dev(v), slots)
    small = np.zeros((2, heads, page // 16, 17 * D), np.uint8)
    for i in range(L):
        ref.write_row(small, (1 - i // page) * page + i % page, k[i], v[i])
    assert np.array_equal(cache[n - 2:].cpu().numpy(), small)
    assert int(cache[:n - 2].count_nonzero()) == 0
    q = normal_bits(rng, 1, 16, D)
    out = torch.empty((1, 16, D), dtype=BF, device="cuda")
    i32 = torch.int32
    mt.kv4_attention(to_dev(q), cache, torch.tensor(table, dtype=i32, device="cuda"),
                     torch.tensor([0, 1], dtype=i32, device="cuda"),
                     torch.tensor([L], dtype=i32, device="cuda"), out)
    K, V = ref.decode(small)
    o, avg, spread, total = ref.attention(ref.bf16_to_f64(q), K, V, np.array([[1, 0]]), np.array([0, 1]),
                                   np.array([L]), page, D ** -0.5)[0]
    err = np.abs(ref.bf16_to_f64(to_bits(out))[0] - o)
    assert (err <= ref.attention_tolerance(o, avg, spread, total, D)).all()


def test_streams_and_graphs():
    s = Step(23, [900, 333], 2, 8, 2, 128, 16)
    plain = s.run()
    i32 = torch.int32
    q = to_dev(s.q)
    cache = torch.from_numpy(s.cache).cuda()
    table, starts, lens = (torch.tensor(x, dtype=i32, device="cuda") for x in (s.table, s.starts, s.lens))
    T = int(s.starts[-1])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.full_like(q, 5.0) for _ in range(4)]
    torch.cuda.synchronize()
    # an own stream given by argument; the allocator's workspace belongs to it
    mt.kv4_attention(q, cache, table, starts, lens, outs[0], max_new=2, stream=other)
    # two graphs with a workspace each, replayed at the same time in two streams
    n = mt.kv4_attention_workspace(16, 2, 128, 2)
    graphs = []
    for i in (1, 2):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            mt.kv4_attention(q, cache, table, starts, lens, outs[i], max_new=2, workspace=ws)
        graphs.append((g, ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    # back to back in one stream with one workspace
    for _ in range(5):
        mt.kv4_attention(q, cache, table, starts, lens, outs[3], max_new=2, workspace=graphs[0][1])
        torch.cuda.synchronize()
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(ref.bf16_to_f64(to_bits(o))[:T], plain[:T])


def test_a_captured_call_keeps_the_workspace_it_took():
    # without a workspace argument the memory belongs to the graph: calls and tensors that come
    # between capture and replay, in this stream and in others, do not share it
    s = Step(35, [3000, 1333], 1, 8, 2, 128, 16)
    plain = s.run()
    i32 = torch.int32
    q = to_dev(s.q)
    cache = torch.from_numpy(s.cache).cuda()
    table, starts, lens = (torch.tensor(x, dtype=i32, device="cuda") for x in (s.table, s.starts, s.lens))
    outs = [torch.full_like(q, 5.0) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mt.kv4_attention(q, cache, table, starts, lens, outs[0])
    n = mt.kv4_attention_workspace(16, 2, 128)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        graph.replay()
        mt.kv4_attention(q, cache, table, starts, lens, outs[1], stream=other)
        with torch.cuda.stream(other):
            junk = torch.full((n // 4,), float("nan"), device="cuda")
            mt.kv4_attention(q, cache, table, starts, lens, outs[2])
            del junk
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(ref.bf16_to_f64(to_bits(o))[:2], plain[:2])


def test_a_decode_run_into_the_layer_tail():
    """Steps of four requests as a server runs them: tables from the lengths, norm and rotation,
    cache rows, attention, then the layer tail with its output projection."""
    R, hq, heads, D, page = 4, 8, 2, 64, 16
    shape = gen.TailShape(R, 256, 8, 2, 128, 128, Ha=hq * D)
    d = gen.make_weights(shape, 3, keys=gen._LAYER_WEIGHTS + ("w_o",))
    d.update(gen.make_activations(shape, 3))
    rng = np.random.default_rng(24)
    i32 = torch.int32
    lens = torch.zeros(R, dtype=i32, device="cuda")
    width = 8
    table = torch.full((R, width), -1, dtype=i32, device="cuda")
    free = torch.randperm(40).to(i32).cuda()
    taken = 0
    cache = mt.kv4_cache(40, page, heads, D)
    gq, gk = (ref.f32_to_bf16(1 + 0.1 * rng.standard_normal(D).astype(np.float32)) for _ in range(2))
    freq = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
    hist = [([], []) for _ in range(R)]
    plan = [[17, 3, 30, 1], [1, 1, 1, 1], [1, 1, 0, 1], [2, 2, 2, 2], [1, 1, 1, 1]]
    st = status_word()
    for new in plan:
        T = sum(new)
        n = torch.tensor(new, dtype=i32, device="cuda")
        starts, kv = torch.empty(R + 1, dtype=i32, device="cuda"), torch.empty(R, dtype=i32, device="cuda")
        pos, slots = torch.empty(T, dtype=i32, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
        used = torch.empty(1, dtype=i32, device="cuda")
        mt.step_tables(lens, n, free[taken:], table, page, starts, kv, pos, slots, used, status=st)
        qkv = normal_bits(rng, T, (hq + 2 * heads) * D)
        dev = to_dev(qkv)
        q = dev[:, :hq * D].view(T, hq, D)
        k = dev[:, hq * D:(hq + heads) * D].view(T, heads, D)
        v = dev[:, (hq + heads) * D:].view(T, heads, D)
        mt.qk_norm_rope(q, k, to_dev(gq), to_dev(gk), pos, torch.from_numpy(freq).cuda(), q, k)
        mt.kv4_append(cache, k, v, slots, status=st)
        out = torch.empty((T, hq, D), dtype=BF, device="cuda")
        mt.kv4_attention(q, cache, table, starts, kv, out, max_new=max(new), status=st)
        taken += int(used)
        # the same from the history, without pages
        qn, kn, vn = (ref.bf16_to_f64(to_bits(t)) for t in (q, k, v))
        at = 0
        for r in range(R):
            for _ in range(new[r]):
                assert int(pos[at]) == len(hist[r][0])
                hist[r][0].append(to_bits(k)[at])
                hist[r][1].append(to_bits(v)[at])
                at += 1
        starts_h = np.concatenate([[0], np.cumsum(new)])
        kv_h = np.array([len(h[0]) for h in hist])
        assert np.array_equal(starts.cpu().numpy(), starts_h) and np.array_equal(kv.cpu().numpy(), kv_h)
        Lm = int(kv_h.max())
        K, V = np.zeros((R, heads, Lm, D)), np.zeros((R, heads, Lm, D))
        for r in range(R):
            for x, dst in ((hist[r][0], K), (hist[r][1], V)):
                dst[r, :, :len(x)] = ref.values(*ref.quantize(np.stack(x, 1)))
        want = ref.attention(qn, K, V, np.arange(R)[:, None].repeat(Lm, 1), starts_h, kv_h, Lm, D ** -0.5)
        got = ref.bf16_to_f64(to_bits(out))
        for i, (o, avg, spread, total) in want.items():
            assert (np.abs(got[i] - o) <= ref.attention_tolerance(o, avg, spread, total, D)).all()
        lens.copy_(kv)
    assert int(st) == 0
    # the last step's rows through the layer tail
    weights = {k: v for k, v in d.items() if k not in ("x", "residual")}
    tail = mt.MoeTail(shape, mt.weights_to_device(weights), max_rows=R)
    res = mt.acts_to_device(d["residual"])
    y = torch.empty((R, 256), dtype=BF, device="cuda")
    tail.run_attn(out.view(R, hq * D), res, y)
    torch.cuda.synchronize()
    d["attn"] = to_bits(out.view(R, hq * D))
    orc = oracle.moe_tail(d, shape.k, shape.eps)
    x_orc = oracle.out_proj(d["attn"], d["w_o"])
    ids, _, _ = tail.routing(R)
    check_parity(to_bits(y), to_bits(res), ids, orc, shape.k,
                 residual_tol=bf16_step(x_orc) + bf16_step(orc["residual"]))
    assert tail.status() == 0
    tail.close()


def test_a_captured_decode_step_follows_the_lengths():
    """One graph of a whole step, replayed while the lengths in device memory grow, with requests that
    pause (their rows go to the end of the step, a padded batch): the same bits as the calls one by
    one on a second cache, and the padded rows stay."""
    R, hq, heads, D, page, width = 3, 16, 2, 128, 16, 20
    shape = gen.TailShape(R, 256, 8, 2, 128, 128, Ha=hq * D)
    d = gen.make_weights(shape, 4, keys=gen._LAYER_WEIGHTS + ("w_o",))
    tail = mt.MoeTail(shape, mt.weights_to_device(d), max_rows=R)
    rng = np.random.default_rng(33)
    i32 = torch.int32
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).cuda()
    gain = to_dev(ref.f32_to_bf16(1 + 0.1 * rng.standard_normal(D).astype(np.float32)))
    new = torch.ones(R, dtype=i32, device="cuda")
    ws = torch.empty(mt.kv4_attention_workspace(hq, heads, D), dtype=torch.uint8, device="cuda")
    first = torch.tensor([250, 15, 0], dtype=i32, device="cuda")

    class Side:
        def __init__(self):
            self.cache = mt.kv4_cache(64, page, heads, D)
            self.table = torch.full((R, width), -1, dtype=i32, device="cuda")
            self.free = torch.arange(64, dtype=i32, device="cuda")
            self.lens = first.clone()
            self.qkv = torch.zeros((R, (hq + 2 * heads) * D), dtype=BF, device="cuda")
            self.res = torch.zeros((R, 256), dtype=BF, device="cuda")
            self.starts, self.kv = (torch.zeros(n, dtype=i32, device="cuda") for n in (R + 1, R))
            self.pos, self.used = (torch.zeros(n, dtype=i32, device="cuda") for n in (R, 1))
            self.slots = torch.zeros(R, dtype=torch.int64, device="cuda")
            self.out = torch.zeros((R, hq, D), dtype=BF, device="cuda")
            self.y = torch.zeros((R, 256), dtype=BF, device="cuda")
            self.st = status_word()

        def step(self):
            q = self.qkv[:, :hq * D].view(R, hq, D)
            k = self.qkv[:, hq * D:(hq + heads) * D].view(R, heads, D)
            v = self.qkv[:, (hq + heads) * D:].view(R, heads, D)
            mt.step_tables(self.lens, new, self.free, self.table, page, self.starts, self.kv, self.pos,
                           self.slots, self.used, status=self.st)
            mt.qk_norm_rope(q, k, gain, gain, self.pos, freq, q, k)
            mt.kv4_append(self.cache, k, v, self.slots, status=self.st)
            mt.kv4_attention(q, self.cache, self.table, self.starts, self.kv, self.out, workspace=ws,
                             status=self.st)
            tail.run_attn(self.out.view(R, hq * D), self.res, self.y)
            self.lens.copy_(self.kv)

    def prompts(side):  # the tokens that are there already
        n = first.clone()
        zero = torch.zeros_like(n)
        T = int(n.sum())
        pos, slots = torch.empty(T, dtype=i32, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
        mt.step_tables(zero, n, side.free, side.table, page, side.starts, side.kv, pos, slots, side.used)
        x = to_dev(normal_bits(np.random.default_rng(34), T, heads, D))
        mt.kv4_append(side.cache, x, x, slots)
        side.free = side.free[int(side.used):].clone()

    one, two = Side(), Side()
    prompts(one)
    prompts(two)
    one.step()  # (warm: what the calls set up once)
    torch.cuda.synchronize()
    fresh = Side()
    prompts(fresh)
    for name in ("cache", "table", "lens", "res", "free", "out", "qkv", "y"):
        getattr(one, name).copy_(getattr(fresh, name))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step()
    torch.cuda.synchronize()
    free = one.free.clone()
    count = first.clone()
    for step, active in enumerate(((1, 1, 1), (1, 0, 1), (0, 0, 0), (0, 1, 0), (1, 1, 1), (1, 1, 0), (1, 1, 1))):
        new.copy_(torch.tensor(active, dtype=i32, device="cuda"))
        count += new
        before = one.out.clone()
        x = to_dev(normal_bits(rng, R, (hq + 2 * heads) * D))
        for side in (one, two):
            side.qkv.copy_(x)
            side.free[:len(free)].copy_(free)
        graph.replay()
        two.step()
        torch.cuda.synchronize()
        for name in ("starts", "kv", "pos", "slots", "used", "table", "cache", "out", "res", "y", "lens"):
            assert torch.equal(getattr(one, name), getattr(two, name)), (step, name)
        assert int(one.st) == 0 and int(two.st) == 0
        assert torch.equal(one.lens, count) and torch.equal(one.out[sum(active):], before[sum(active):])
        free = torch.cat([free[int(one.used):], torch.full((int(one.used),), -1, dtype=i32, device="cuda")])
    assert tail.status() == 0
    tail.close()
