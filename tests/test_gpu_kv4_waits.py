"""The waits between the warps of the attention over the MXFP4 cache (kv4_attn.h) when a hand-over
never comes: moe_tail_debug_kv4_stall lets one barrier of the first CTA expect an arrival more than
is sent, so that its waits run out on the device.  The call ends, says so, and the next one is right."""
import numpy as np
import pytest

import moe_layer_tail_gb300 as mt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


class Batch:
    """Requests of these lengths with `new` rows each, their cache filled by kv4_append."""

    def __init__(self, D, G, heads, lens, new, window=0, sinks=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(sum(lens) + D)
        page, total = 32, sum(-(-n // 32) for n in lens)
        self.cache = mt.kv4_cache(total, page, heads, D)
        order = torch.randperm(total, generator=g, device="cuda").to(I32)
        self.table = torch.full((len(lens), -(-max(lens) // page)), -1, dtype=I32, device="cuda")
        at = 0
        for r, n in enumerate(lens):
            self.table[r, :-(-n // page)] = order[at:at + -(-n // page)]
            at += -(-n // page)
        x = [torch.randn((total * page, heads, D), generator=g, device="cuda").to(BF) for _ in range(2)]
        mt.kv4_append(self.cache, *x, torch.arange(total * page, device="cuda"))
        T = new * len(lens)
        self.q = torch.randn((T, heads * G, D), generator=g, device="cuda").to(BF)
        self.starts = torch.arange(0, T + 1, new, dtype=I32, device="cuda")
        self.lens = torch.tensor(lens, dtype=I32, device="cuda")
        self.new, self.window, self.sinks = new, window, sinks

    def run(self, stall=-1, report=True):
        """(output as integers, status) of a call whose hand-over number `stall` stays away."""
        out, st = torch.full_like(self.q, 5.0), torch.zeros(1, dtype=I32, device="cuda")
        assert mt.load_library().moe_tail_debug_kv4_stall(stall) == mt.OK
        mt.kv4_attention(self.q, self.cache, self.table, self.starts, self.lens, out, max_new=self.new,
                         window=self.window, sinks=self.sinks, status=st if report else None)
        torch.cuda.synchronize()
        return out.view(torch.int16).cpu().numpy(), int(st)


def batches(D, G):
    heads = 8
    # the first CTA has 13 steps of one request; ten and more requests of one step; rows that see
    # nothing of their first steps, where a softmax warp's next turn depends on the others'
    yield Batch(D, G, heads, [40000], 1)
    yield Batch(D, G, heads, [40 + r % 60 for r in range(300)], 1)
    yield Batch(D, G, heads, [3000, 2500], 200, window=17, sinks=3)


def barriers(D):
    """(barriers of a CTA, those that these batches wait for): rings of raw tiles, operands, notes,
    queries; then the keys' two, scores, numerators, values, free values, outputs, four checks, two
    meetings.  With D <= 128 nothing waits for free keys and values (3); D 256 has one place for
    queries (2 fewer).  (With 32 rows an item it has one for values too, but 300 requests go through
    items of 16 rows, which have two.)"""
    raw, ops = {64: (6, 3), 128: (4, 3), 256: (2, 2)}[D]
    n = 2 * raw + 2 * ops + 8 + 4 + 12 + 4 + 2
    return n, n - (3 if D <= 128 else 2)


@pytest.mark.parametrize("D,G", [(64, 8), (128, 16), (256, 4), (256, 32)])
def test_a_hand_over_that_never_comes_ends_the_call(D, G):
    n, used = barriers(D)
    seen = set()
    for i, b in enumerate(batches(D, G)):
        clean, st = b.run()
        assert st == 0
        for stall in range(n + 1):
            if i and stall in seen and stall < n - 18:  # (a call that gives up takes 0.1 s)
                continue
            out, st = b.run(stall)
            assert st in (0, mt.STATUS_TIMEOUT)
            if st:
                seen.add(stall)
            else:
                assert np.array_equal(out, clean)
            again, st = b.run()
            assert st == 0 and np.array_equal(again, clean)
    assert len(seen) == used and n not in seen


@pytest.mark.parametrize("D,G", [(64, 8), (128, 16), (256, 4), (256, 32)])
def test_rows_that_were_given_up_are_nan(D, G):
    # without a status word: each head of a row is what it always is, or NaN throughout
    n, _ = barriers(D)
    for b in batches(D, G):
        clean, _ = b.run()
        nan = np.zeros(clean.shape[:2], bool)
        for stall in (0, n // 2, n - 10, n - 1):
            out, _ = b.run(stall, report=False)
            gone = (out & 0x7FFF) > 0x7F80
            assert np.array_equal(gone.all(-1), gone.any(-1))
            assert np.array_equal(out[~gone], clean[~gone])
            nan |= gone.any(-1)
        assert 0 < nan.sum() < nan.size


def test_the_order_holds_for_one_call_and_can_be_taken_back():
    b = next(batches(64, 8))
    clean, _ = b.run()
    lib = mt.load_library()
    lib.moe_tail_debug_kv4_stall(0)
    with pytest.raises(mt.MoeTailError):  # (a refused call is none)
        mt.kv4_attention(b.q, b.cache, b.table, b.starts, b.lens, b.q)
    out, st = b.run()  # (takes it back)
    assert st == 0 and np.array_equal(out, clean)
