"""kv4_attn.h without a GPU: the entry points are exported, constants match the header, bad
arguments are refused before any launch, the binding refuses wrong tensors, and the format's
restatement (kv4_ref.py) holds its own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv4_ref as ref
import moe_layer_tail_gb300 as mt
from moe_layer_tail_gb300 import build as mt_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "kv4_attn.h")).read()
INV, UNS = mt.ERR_INVALID_ARG, mt.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    mt_build.build()
    return mt.load_library()


def test_declared_symbols_are_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src))
    assert names == {"moe_step_tables", "moe_qk_norm_rope", "moe_kv4_append", "moe_kv4_read",
                     "moe_kv4_attention", "moe_kv4_attention_workspace"}
    for n in names:
        assert hasattr(lib, n), "missing export " + n


def test_status_bits_match_header():
    bits = dict(re.findall(r"#define MOE_KV4_STATUS_(\w+) (\d+)", HEADER))
    assert set(bits) == {"BAD_LENGTH", "NO_PAGES", "ROWS", "BAD_SLOT", "BAD_PAGE"}
    for name, v in bits.items():
        assert getattr(mt, "KV4_STATUS_" + name) == int(v)


def _call(fn, defaults, kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return fn(*args.values())


A = 0x10000  # an aligned address that nothing dereferences: refusal comes first
TABLES = dict(reqs=2, max_rows=4, page_size=16, n_free=3, table_width=5, table_stride=5,
              cached_lens=A, new_lens=A + 16, free_pages=A, block_table=A, row_starts=A, kv_lens=A + 32,
              positions=A, slots=A, pages_used=A, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(reqs=0), INV), (dict(reqs=1025), UNS), (dict(max_rows=0), INV),
    (dict(max_rows=(1 << 24) + 1), UNS), (dict(page_size=0), UNS), (dict(page_size=24), UNS),
    (dict(page_size=1040), UNS), (dict(n_free=-1), INV), (dict(table_width=0), INV),
    (dict(table_stride=4), INV), (dict(cached_lens=None), INV), (dict(new_lens=None), INV),
    (dict(free_pages=None), INV), (dict(block_table=None), INV), (dict(row_starts=None), INV),
    (dict(kv_lens=None), INV), (dict(positions=None), INV), (dict(slots=None), INV),
    (dict(pages_used=None), INV), (dict(kv_lens=A), INV), (dict(kv_lens=A + 16), INV)])
def test_step_tables_refuses(lib, kw, code):
    assert _call(lib.moe_step_tables, TABLES, kw) == code


ROPE = dict(rows=2, q_heads=4, k_heads=2, head_dim=64, rot_dim=32, interleaved=0, eps=1e-6, q=A,
            ld_q=256, k=A, ld_k=128, q_gamma=A, k_gamma=A, positions=A, inv_freq=A, q_out=A + 4096,
            ld_qo=256, k_out=A + 4096, ld_ko=128, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=(1 << 24) + 1), INV), (dict(eps=0.0), INV),
    (dict(eps=float("nan")), INV), (dict(q_heads=0), UNS), (dict(q_heads=1025), UNS),
    (dict(k_heads=-1), UNS), (dict(head_dim=0), UNS), (dict(head_dim=72), UNS),
    (dict(head_dim=272), UNS), (dict(rot_dim=80), UNS), (dict(rot_dim=24), UNS),
    (dict(rot_dim=-16), UNS), (dict(q=None), INV), (dict(q=A + 8), INV), (dict(k=None), INV),
    (dict(k_out=None), INV), (dict(q_out=A + 2), INV), (dict(q_gamma=A + 4), INV),
    (dict(k_gamma=A + 4), INV), (dict(positions=None), INV), (dict(inv_freq=None), INV),
    (dict(ld_q=248), INV), (dict(ld_q=260), INV), (dict(ld_k=120), INV), (dict(ld_qo=0), INV),
    (dict(ld_ko=-128), INV), (dict(q_out=A, ld_qo=512), INV), (dict(k_out=A, ld_ko=512), INV)])
def test_qk_norm_rope_refuses(lib, kw, code):
    assert _call(lib.moe_qk_norm_rope, ROPE, kw) == code


ROWS = dict(rows=2, kv_heads=2, head_dim=128, page_size=32, n_pages=4, cache=A, k=A, ld_k=256, v=A,
            ld_v=256, slots=A, status=None, stream=None)


@pytest.mark.parametrize("fn", ["moe_kv4_append", "moe_kv4_read"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=(1 << 24) + 1), INV), (dict(n_pages=0), INV),
    (dict(n_pages=1 << 31), INV), (dict(kv_heads=0), UNS), (dict(kv_heads=257), UNS),
    (dict(head_dim=96), UNS), (dict(page_size=8), UNS), (dict(page_size=2048), UNS),
    (dict(cache=None), INV), (dict(cache=A + 8), INV), (dict(k=None), INV), (dict(v=A + 2), INV),
    (dict(slots=None), INV), (dict(ld_k=248), INV), (dict(ld_v=257), INV)])
def test_cache_rows_refuse(lib, fn, kw, code):
    assert _call(getattr(lib, fn), ROWS, kw) == code


ATTN = dict(rows=4, reqs=2, q_heads=16, kv_heads=2, head_dim=128, page_size=32, n_pages=4, q=A,
            ld_q=2048, cache=A, block_table=A, table_width=3, table_stride=3, row_starts=A, kv_lens=A,
            scale=0.1, window=0, sinks=0, max_new=1, out=A + 4096, ld_o=2048, workspace=A,
            workspace_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=(1 << 20) + 1), UNS), (dict(reqs=0), INV), (dict(reqs=1025), UNS),
    (dict(n_pages=0), INV), (dict(n_pages=1 << 31), INV), (dict(table_width=0), INV),
    (dict(table_stride=2), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(window=-1), INV),
    (dict(sinks=-1), INV), (dict(max_new=0), INV), (dict(q_heads=15), UNS), (dict(q_heads=0), UNS),
    (dict(q_heads=2 * 257), UNS), (dict(kv_heads=0), UNS), (dict(head_dim=192), UNS),
    (dict(page_size=20), UNS), (dict(q=None), INV), (dict(q=A + 4), INV), (dict(cache=A + 8), INV),
    (dict(out=None), INV), (dict(workspace=None), INV), (dict(workspace=A + 8), INV),
    (dict(block_table=None), INV), (dict(row_starts=None), INV), (dict(kv_lens=None), INV),
    (dict(ld_q=2040), INV), (dict(ld_o=2052), INV), (dict(out=A), INV)])
def test_attention_refuses(lib, kw, code):
    assert _call(lib.moe_kv4_attention, ATTN, kw) == code


@pytest.mark.parametrize("args,code", [((16, 2, 128, 0), INV), ((16, 3, 128, 1), UNS),
                                       ((16, 2, 100, 1), UNS), ((0, 2, 128, 1), UNS)])
def test_workspace_refuses(lib, args, code):
    assert lib.moe_kv4_attention_workspace(*args) == code


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    cache = mt.kv4_cache(2, 16, 2, 64, device="cpu")
    assert cache.shape == (2, 2, 1, 17 * 64)
    for f in (lambda: mt.kv4_append(cache, x, x, torch.zeros(1, dtype=torch.int64)),
              lambda: mt.qk_norm_rope(x, None, None, None, i, None, x, None),
              lambda: mt.step_tables(i, i, i, i.view(1, 1), 16, i, i, i, i, i),
              lambda: mt.kv4_attention(x, cache, i.view(1, 1), i, i, x)):
        with pytest.raises(mt.MoeTailError) as e:
            f()
        assert e.value.code == INV
    with pytest.raises(mt.MoeTailError):
        mt.kv4_cache(1, 20, 1, 64, device="cpu")


# -------------------------------------------------- the restatement's own pins ----

@pytest.mark.parametrize("D", [64, 128, 256])
def test_format_places_every_byte_once(D):
    kc, vc, ks, vs = ref.offsets(D)
    used = np.concatenate([kc[:, ::2].ravel(), vc[:, ::2].ravel(), ks.ravel(), vs.ravel()])
    assert np.array_equal(kc[:, ::2], kc[:, 1::2]) and np.array_equal(vc[:, ::2], vc[:, 1::2])
    assert np.array_equal(np.sort(used), np.arange(17 * D))


def test_format_round_trip_and_nearest_value():
    rng = np.random.default_rng(5)
    x = ref.f32_to_bf16((rng.standard_normal((40, 64)) * np.exp2(rng.integers(-140, 120, (40, 1))))
                        .astype(np.float32))
    codes, scales = ref.quantize(x)
    got, want = ref.values(codes, scales), ref.bf16_to_f64(x)
    f = np.repeat(np.exp2(scales.astype(float) - 127), 32, -1)
    # nearest of all sixteen codes at the block's scale, and no smaller scale holds the block
    every = np.concatenate([ref.GRID, -ref.GRID])
    best = np.abs(every[:, None, None] * f - want).min(0)
    assert np.array_equal(np.abs(got - want), best)
    amax = np.abs(want).reshape(40, 2, 32).max(-1)
    s = np.exp2(scales.astype(float) - 127)
    assert (amax <= 6 * s).all() and ((amax > 3 * s) | (scales == 1)).all()


def test_attention_restatement_against_uniform_weights():
    # zero queries: the mean of the visible values
    rng = np.random.default_rng(6)
    K, V = rng.standard_normal((2, 3, 2, 16, 64))
    out, _, _, _ = ref.attention(np.zeros((1, 4, 64)), K, V, np.array([[2, 0]]), np.array([0, 1]),
                                 np.array([20]), 16, 1.0, window=3, sinks=2)[0]
    seen = np.stack([V[2, :, 0], V[2, :, 1], V[0, :, 1], V[0, :, 2], V[0, :, 3]])
    assert np.allclose(out[:2], seen[:, 0].mean(0)) and np.allclose(out[2:], seen[:, 1].mean(0))


def test_rotation_restatement_turns_by_the_angle():
    x = np.zeros((1, 1, 32))
    x[0, 0, 3] = 2.0
    y, _ = ref.norm_rope(x, None, np.array([5]), np.full(16, 0.25, np.float32), 1e-6, False)
    assert np.isclose(y[0, 0, 3], 2 * np.cos(1.25)) and np.isclose(y[0, 0, 19], 2 * np.sin(1.25))
