"""The operators of one decode step's attention block, in front of the layer tail: what is timed.

Four operators, used in this order by a step (request lengths -> rows -> cache -> attention
output, which moe_tail_run_attn's projection then takes):

  tables  block tables, row starts, positions and cache slots of a step from request lengths
  rope    RMSNorm of every query and key head and the position rotation, in one pass
  rows    keys and values written to a paged MXFP4 cache (E2M1 codes, one E8M0 scale per 32
          channels) and the same slots read back as bf16
  attn    attention of the step's query rows over that cache, with an optional sliding
          window and a few first tokens that stay visible

The plain forms below (own = False) are elementary torch operations in 32 bits (64 for the
angles); own = True makes the library's calls on the same inputs.
"""
import math
import random

import torch

own = False

# The cache: uint8 [pages, kv heads, page_size / 16, 17 * D].  A tile of 16 tokens is
# K codes (8 D bytes), V codes (8 D), K scales (D / 2), V scales (D / 2); within the codes the
# bytes stand in the order that the matrix instructions' lanes read them (see _tile_values).


# ------------------------------------------------------------------------------- cases ----

def listed():
    return [
        # one decode step of a full batch of rows: one new token for each of 32 requests
        dict(name="tables_decode_r32", op="tables", reqs=32, rows=32, page=64, longest=32768),
        # admission of a large batch: prompts of 1024 requests enter the cache together
        dict(name="tables_prompts_r1024", op="tables", reqs=1024, rows=262144, page=16,
             longest=4096),
        # a single decode row, the smallest call: latency
        dict(name="rope_r1_d128", op="rope", rows=1, hq=128, hkv=8, dim=128, rot=128,
             interleaved=False, far=32768),
        # a full decode batch, wide heads with a quarter of the channels rotated, far positions
        dict(name="rope_r32_d256", op="rope", rows=32, hq=64, hkv=4, dim=256, rot=64,
             interleaved=True, far=1 << 20),
        # a prompt chunk
        dict(name="rope_r8192_d128", op="rope", rows=8192, hq=64, hkv=8, dim=128, rot=128,
             interleaved=False, far=131072),
        # the cache rows of a full decode batch
        dict(name="rows_r32_d128", op="rows", rows=32, hkv=8, dim=128, page=64, pages=4096),
        # the cache rows of long prompts
        dict(name="rows_r65537_d128", op="rows", rows=65537, hkv=8, dim=128, page=64,
             pages=2048),
        # one request, a short context: latency
        dict(name="attn_r1_l1000", op="attn", reqs=1, new=1, hq=128, hkv=8, dim=128, page=64,
             longest=1000, ragged=False, window=0, sinks=0, mix=1),
        # a full decode batch with ragged contexts
        dict(name="attn_r32_l32768", op="attn", reqs=32, new=1, hq=128, hkv=8, dim=128, page=64,
             longest=32768, ragged=True, window=0, sinks=0, mix=2),
        # one request, a very long context
        dict(name="attn_r1_l524287", op="attn", reqs=1, new=1, hq=128, hkv=8, dim=128, page=128,
             longest=524287, ragged=False, window=0, sinks=0, mix=3),
        # sliding window with the first four tokens kept, small heads, small pages
        dict(name="attn_r16_l65521_window", op="attn", reqs=16, new=1, hq=64, hkv=8, dim=64,
             page=16, longest=65521, ragged=True, window=4096, sinks=4, mix=4),
        # four rows per request (a verification step of drafted tokens), wide heads
        dict(name="attn_r8_new4_d256", op="attn", reqs=8, new=4, hq=64, hkv=4, dim=256, page=64,
             longest=16384, ragged=True, window=0, sinks=0, mix=5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rows", "attn", "attn", "attn"])
    if op == "tables":
        reqs = _log_int(rng, 1, 1024)
        return dict(op=op, reqs=reqs, rows=max(reqs, _log_int(rng, 1, 262144)),
                    page=rng.choice([16, 32, 48, 64, 128]), longest=_log_int(rng, 16, 32768))
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192, 256])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 5, 8, 16])
        return dict(op=op, rows=_log_int(rng, 1, 4096), hq=hq, hkv=hkv, dim=dim,
                    rot=rng.choice([r for r in (16, 32, 64, 96, 128, dim) if r <= dim]),
                    interleaved=rng.random() < 0.5, far=_log_int(rng, 4096, 1 << 20))
    if op == "rows":
        page = rng.choice([16, 32, 48, 64, 128])
        rows = _log_int(rng, 1, 32768)
        return dict(op=op, rows=rows, hkv=rng.choice([1, 2, 3, 4, 8]),
                    dim=rng.choice([64, 128, 256]), page=page,
                    pages=2 + (2 * rows + page - 1) // page)
    reqs = _log_int(rng, 1, 32)
    hkv = rng.choice([1, 2, 3, 4, 8])
    new = rng.choice([1, 1, 1, 2, 3, 4])
    dim = rng.choice([64, 128, 256])
    window = rng.choice([0, 0, _log_int(rng, 64, 8192)])
    budget = (1 << 30) // (hkv * dim * reqs * new)  # values of the padded keys, for each row
    return dict(op=op, reqs=reqs, new=new, hq=hkv * rng.choice([1, 2, 4, 6, 8, 12, 16]), hkv=hkv,
                dim=dim, page=rng.choice([16, 32, 48, 64, 128]),
                longest=_log_int(rng, 64, max(64, min(131072, budget))),
                ragged=rng.random() < 0.7, window=window,
                sinks=rng.choice([0, 1, 4, 17]) if window else 0, mix=rng.randrange(1 << 30))


def _kv_lens(case):
    """The context length of each request after the step (from the case alone)."""
    r = random.Random(case["mix"])
    top = max(case["longest"], case["new"])
    if not case["ragged"]:
        return [top] * case["reqs"]
    lens = [r.randint(max(case["new"], top // 64), top) for _ in range(case["reqs"])]
    lens[r.randrange(len(lens))] = top
    return lens


def _visible(case, length):
    """Cache positions that some row of a request of this length sees."""
    if not case["window"]:
        return length
    first = max(0, length - case["new"] - case["window"] + 1)
    return length - max(0, first - case["sinks"])


# ------------------------------------------------------------------------------ inputs ----

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if case["op"] == "tables":
        R, N, P = case["reqs"], case["rows"], case["page"]
        # N new rows spread over the requests, one at least each, some with many more than others
        share = [1 + i * 37 % 11 for i in range(R)]
        total, spread = sum(share), []
        for i in range(R):
            spread.append(1 + (N - R) * sum(share[:i + 1]) // total
                          - (N - R) * sum(share[:i]) // total)
        order = torch.randperm(R, generator=g, device=dev)
        new = torch.tensor(spread, device=dev)[order]
        cached = torch.randint(0, case["longest"] + 1, (R,), generator=g, device=dev)
        M = (case["longest"] + max(spread) + P - 1) // P
        F = R + (N + P - 1) // P
        old = (cached + P - 1) // P
        pages = torch.randperm(int(old.sum()) + F, generator=g, device=dev).to(torch.int32)
        table = torch.full((R, M), -1, dtype=torch.int32, device=dev)
        held = torch.arange(M, device=dev)[None, :] < old[:, None]
        table[held] = pages[F:]
        s.update(cached=cached.to(torch.int32), new=new.to(torch.int32), free=pages[:F].clone(),
                 table=table, row_starts=torch.empty(R + 1, dtype=torch.int32, device=dev),
                 kv_lens=torch.empty(R, dtype=torch.int32, device=dev),
                 positions=torch.empty(N, dtype=torch.int32, device=dev),
                 slots=torch.empty(N, dtype=torch.int64, device=dev),
                 used=torch.empty(1, dtype=torch.int32, device=dev))
        return s
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["rows"], case["hq"], case["hkv"], case["dim"]
        # the packed output of a projection: queries, keys, values of a row side by side
        qkv = (normal(T, (Hq + 2 * Hkv) * D) * 1.7).bfloat16()
        s.update(q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
                 q_gamma=(1 + 0.1 * normal(D)).bfloat16(), k_gamma=(1 + 0.1 * normal(D)).bfloat16(),
                 positions=torch.randint(0, case["far"], (T,), generator=g, device=dev,
                                         dtype=torch.int32),
                 inv_freq=(10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64,
                                                     device=dev) / case["rot"])).float(),
                 q_out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev),
                 k_out=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev))
        return s
    if case["op"] == "rows":
        T, Hkv, D, P, n = case["rows"], case["hkv"], case["dim"], case["page"], case["pages"]
        gain = torch.exp2(2 * normal(1, Hkv, D)).clamp(0.25, 8)  # a few channels stand out
        s.update(k=(normal(T, Hkv, D) * gain).bfloat16(), v=normal(T, Hkv, D).bfloat16(),
                 cache=torch.zeros((n, Hkv, P // 16, 17 * D), dtype=torch.uint8, device=dev),
                 k_out=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev),
                 v_out=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev))
        # runs of consecutive slots in pages anywhere in the cache, as a step's table gives them
        page = torch.randperm(n, generator=g, device=dev)
        at = torch.arange(T, device=dev) + P // 2
        s["slots"] = page[at // P] * P + at % P
        return s
    R, new, Hq, Hkv, D, P = (case[x] for x in ("reqs", "new", "hq", "hkv", "dim", "page"))
    lens = _kv_lens(case)
    held = [(n + P - 1) // P for n in lens]
    n_pages, M = sum(held) + 3, max(held)
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((R, M), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = table.to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    cache = torch.empty((n_pages, Hkv, P // 16, 17 * D), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 25) // (Hkv * P * D))
    gain = torch.exp2(normal(1, Hkv, 1, D).clamp(-2, 2))
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        k = (normal(b - a, Hkv, P, D) * gain).bfloat16().view(b - a, Hkv, P // 16, 16, D)
        v = normal(b - a, Hkv, P, D).bfloat16().view(b - a, Hkv, P // 16, 16, D)
        cache[a:b] = _tile_bytes(k, v)
    s.update(q=(1.5 * normal(R * new, Hq, D)).bfloat16(), cache=cache, table=table,
             row_starts=(torch.arange(R + 1, device=dev) * new).to(torch.int32),
             kv_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             out=torch.empty((R * new, Hq, D), dtype=torch.bfloat16, device=dev),
             scale=D ** -0.5)
    return s


# ------------------------------------------------------------------- the cache's format ----

def _quantize(x):
    """bf16 [..., D] -> E2M1 codes [..., D] and E8M0 scale bytes [..., D / 32] (both uint8):
    the scale is the smallest power of two with |x| <= 6 times it, from 2^-126 to 2^125."""
    b = x.float().unflatten(-1, (x.shape[-1] // 32, 32))
    m, e = torch.frexp(b.abs().amax(-1))  # amax = m 2^e, m in [0.5, 1)
    e = (e - 3 + (m > 0.75).int()).clamp(-126, 125)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    y = torch.ldexp(b, -e[..., None])
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5).int() + 8 * torch.signbit(y).int())
    return code.flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The inverse: fp32 [..., D]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       device=codes.device)
    x = lut[codes.int()].unflatten(-1, (scales.shape[-1], 32))
    return (x * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _k_order(x, D):
    """Byte pairs [..., 16 t, D/2] of a tile's keys -> the order they are stored in, [..., 8 D].
    t = 8 hh + g, channel pair p = 16 b + 4 c + j; stored [16-byte vector][g][c][16]."""
    x = x.unflatten(-1, (D // 32, 4, 4)).unflatten(-4, (2, 8))        # hh g b c j
    x = x.movedim((-4, -2), (-5, -4))                                 # g c hh b j
    x = x.flatten(-3).unflatten(-1, (D // 64, 16))                    # g c v 16
    return x.movedim(-2, -4).flatten(-4)


def _v_order(x, D):
    """The same for values: t = 8 h + 2 c + o, channel pair p = 16 b + 2 g + j."""
    x = x.unflatten(-1, (D // 32, 8, 2)).unflatten(-4, (2, 4, 2))     # h c o b g j
    x = x.movedim((-2, -5), (-6, -5))                                 # g c h o b j
    x = x.flatten(-4).unflatten(-1, (D // 64, 16))
    return x.movedim(-2, -4).flatten(-4)


def _ks_order(x):
    """Scale bytes [..., 16 t, D/32] of a tile's keys -> stored [g][hh][D/32]."""
    return x.unflatten(-2, (2, 8)).movedim(-3, -2).flatten(-3)


def _vs_order(x):
    """Scale bytes [..., 16 t, D/32] of a tile's values -> stored [c][D/32][h][o]."""
    return x.unflatten(-2, (2, 4, 2)).movedim((-3, -1), (-4, -3)).flatten(-4)


def _tile_bytes(k, v):
    """bf16 [..., 16, D] keys and values -> the tile's bytes [..., 17 D]."""
    D = k.shape[-1]
    (kc, ks), (vc, vs) = _quantize(k), _quantize(v)
    kc = kc[..., 0::2] | (kc[..., 1::2] << 4)  # channel 2p in the low four bits
    vc = vc[..., 0::2] | (vc[..., 1::2] << 4)
    return torch.cat([_k_order(kc, D), _v_order(vc, D), _ks_order(ks), _vs_order(vs)], -1)


def _tile_values(tile):
    """The tile's bytes [..., 17 D] -> fp32 keys and values [..., 16, D]."""
    D = tile.shape[-1] // 17

    def pairs(x):
        return torch.stack([x & 15, x >> 4], -1).flatten(-2)

    k = tile[..., :8 * D].unflatten(-1, (D // 64, 8, 4, 16)).movedim(-4, -2).flatten(-2)
    k = k.unflatten(-1, (2, D // 32, 4)).movedim((-5, -4), (-4, -2))  # g c hh b j -> hh g b c j
    k = pairs(k.flatten(-3).flatten(-3, -2))
    v = tile[..., 8 * D:16 * D].unflatten(-1, (D // 64, 8, 4, 16)).movedim(-4, -2).flatten(-2)
    v = v.unflatten(-1, (2, 2, D // 32, 2)).movedim((-6, -5), (-2, -5))  # -> h c o b g j
    v = pairs(v.flatten(-3).flatten(-4, -2))
    ks = tile[..., 16 * D:16 * D + D // 2].unflatten(-1, (8, 2, D // 32)).movedim(-2, -3)
    vs = tile[..., 16 * D + D // 2:].unflatten(-1, (4, D // 32, 2, 2))  # c b h o
    vs = vs.movedim((-2, -4), (-4, -3)).movedim(-2, -1)                # -> h c o b
    return _values(k, ks.flatten(-3, -2)), _values(v, vs.flatten(-4, -2))


# ------------------------------------------------------------------------- plain forms ----

def _plain_tables(s):
    P, N = s["page"], s["slots"].shape[0]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"].long()
    R, M = table.shape
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, want = (cached + P - 1) // P, (cached + new + P - 1) // P
    off = (want - have).cumsum(0) - (want - have)
    j = torch.arange(M, device=table.device)[None, :]
    fresh = (j >= have[:, None]) & (j < want[:, None])
    at = (off[:, None] + j - have[:, None]).clamp(0, free.shape[0] - 1)
    table = torch.where(fresh, free[at], table.long())
    row = torch.arange(N, device=table.device)
    req = torch.searchsorted(starts[1:], row, right=True)
    pos = cached[req] + row - starts[req]
    slots = table[req, pos // P] * P + pos % P
    return (table.int(), starts.int(), (cached + new).int(), pos.int(), slots,
            (want - have).sum().reshape(1).int())


def _plain_rope_half(x, gamma, cos, sin, rot, interleaved):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * gamma.float()
    a, b = ((y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved
            else (y[..., :rot // 2], y[..., rot // 2:rot]))
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, y[..., rot:]], -1).bfloat16()


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return (_plain_rope_half(s["q"], s["q_gamma"], cos, sin, s["rot"], s["interleaved"]),
            _plain_rope_half(s["k"], s["k_gamma"], cos, sin, s["rot"], s["interleaved"]))


def _plain_rows(s):
    k, v, cache, slots, P = s["k"], s["v"], s["cache"], s["slots"], s["page"]
    T, Hkv, D = k.shape
    flat = cache.view(-1)
    # where byte p of token t's codes, and its scale bytes, stand in a tile
    at = torch.arange(8 * D, device=k.device)
    inv = torch.empty_like(at)
    inv[_k_order(at.view(16, D // 2), D)] = at
    k_at = inv.view(16, D // 2)
    inv = torch.empty_like(at)
    inv[_v_order(at.view(16, D // 2), D)] = at
    v_at = inv.view(16, D // 2) + 8 * D
    at = torch.arange(D // 2, device=k.device)
    inv = torch.empty_like(at)
    inv[_ks_order(at.view(16, D // 32))] = at
    ks_at = inv.view(16, D // 32) + 16 * D
    inv = torch.empty_like(at)
    inv[_vs_order(at.view(16, D // 32))] = at
    vs_at = inv.view(16, D // 32) + 16 * D + D // 2
    t = slots % 16
    tile = (((slots // P)[:, None] * Hkv + torch.arange(Hkv, device=k.device)) * (P // 16)
            + ((slots % P) // 16)[:, None]) * (17 * D)
    out = []
    for x, c_at, s_at in ((k, k_at, ks_at), (v, v_at, vs_at)):  # keys, then values
        codes, scales = _quantize(x)
        flat[tile[..., None] + c_at[t][:, None]] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        flat[tile[..., None] + s_at[t][:, None]] = scales
    for c_at, s_at in ((k_at, ks_at), (v_at, vs_at)):
        c = flat[tile[..., None] + c_at[t][:, None]]
        codes = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        out.append(_values(codes, flat[tile[..., None] + s_at[t][:, None]]).bfloat16())
    return tuple(out)


def _plain_attn(s):
    q, cache, kv_lens, row_starts = s["q"], s["cache"], s["kv_lens"].long(), s["row_starts"].long()
    R, Q, P, dev = s["reqs"], s["new"], s["page"], q.device
    T, Hq, D = q.shape
    Hkv = cache.shape[1]
    k, v = _tile_values(cache[s["table"].clamp(min=0).long()])     # [R, M, Hkv, P/16, 16, D]
    k = k.movedim(2, 1).flatten(2, 4)                              # [R, Hkv, M P, D]
    v = v.movedim(2, 1).flatten(2, 4)
    L = k.shape[2]
    tok = torch.arange(Q, device=dev)
    row = (row_starts[:-1, None] + tok).clamp(max=T - 1)           # [R, Q]
    qr = q.float()[row].unflatten(2, (Hkv, Hq // Hkv)).movedim(2, 1)   # [R, Hkv, Q, G, D]
    sc = torch.matmul(qr.flatten(2, 3), k.mT) * s["scale"]         # [R, Hkv, Q G, L]
    pos = kv_lens[:, None] - (row_starts[1:] - row_starts[:-1])[:, None] + tok  # [R, Q]
    j = torch.arange(L, device=dev)
    seen = j <= pos[..., None]
    if s["window"]:
        seen &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    seen = seen[:, None, :, None, :].expand(-1, -1, -1, Hq // Hkv, -1).flatten(2, 3)
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    o = torch.where(top == -math.inf, torch.zeros_like(o), o)
    o = o.unflatten(2, (Q, Hq // Hkv)).movedim(1, 2).flatten(2, 3)  # [R, Q, Hq, D]
    at = torch.arange(T, device=dev)
    req = torch.searchsorted(row_starts[1:], at, right=True).clamp(max=R - 1)
    return o[req, at - row_starts[req]].bfloat16()


def run(s):
    if own:
        import moe_layer_tail_gb300 as mt
        if s["op"] == "tables":
            mt.step_tables(s["cached"], s["new"], s["free"], s["table"], s["page"],
                           s["row_starts"], s["kv_lens"], s["positions"], s["slots"], s["used"])
            return (s["table"], s["row_starts"], s["kv_lens"], s["positions"], s["slots"],
                    s["used"])
        if s["op"] == "rope":
            mt.qk_norm_rope(s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["positions"],
                            s["inv_freq"], s["q_out"], s["k_out"], eps=1e-6,
                            interleaved=s["interleaved"])
            return s["q_out"], s["k_out"]
        if s["op"] == "rows":
            mt.kv4_append(s["cache"], s["k"], s["v"], s["slots"])
            mt.kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
            return s["k_out"], s["v_out"]
        mt.kv4_attention(s["q"], s["cache"], s["table"], s["row_starts"], s["kv_lens"], s["out"],
                         scale=s["scale"], window=s["window"], sinks=s["sinks"],
                         max_new=s["new"])
        return s["out"]
    return {"tables": _plain_tables, "rope": _plain_rope, "rows": _plain_rows,
            "attn": _plain_attn}[s["op"]](s)


# ---------------------------------------------------------------------- work of one pass ----

def work(case):
    if case["op"] == "tables":
        R, N, P = case["reqs"], case["rows"], case["page"]
        # lengths in, starts and lengths out, each row's position and slot, the new pages
        return {"bytes": 16 * R + 12 * N + 8 * (N // P), "flops": 8 * N}
    if case["op"] == "rope":
        n = case["rows"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["rows"] + 4 * case["dim"] + 2 * case["rot"],
                "flops": 6 * n + 3 * n * case["rot"] // case["dim"]}
    if case["op"] == "rows":
        n = 2 * case["rows"] * case["hkv"] * case["dim"]
        # values in, codes and scales out; codes and scales in, values out
        return {"bytes": 4 * n + 2 * n * 17 // 32 + 16 * case["rows"], "flops": 4 * n}
    seen = sum(_visible(case, n) for n in _kv_lens(case))
    rows = case["reqs"] * case["new"] * case["hq"] * case["dim"]
    return {"bytes": seen * case["hkv"] * 17 * case["dim"] // 16 + 4 * rows
            + 4 * (seen // case["page"]),
            "flops": 4 * seen * case["new"] * case["hq"] * case["dim"]}


# ------------------------------------------------------------- the definition in 64 bits ----

def _exact_code_values(codes, scales):
    """Sign, exponent and mantissa bits of each code, and the scale's power of two."""
    c = codes.long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    return torch.where(c >= 8, -mag, mag) * torch.exp2(scales.double() - 127)


def _exact_tiles(tiles):
    """Tile bytes [n, 17 D] -> float64 keys and values [n, 16, D], byte by byte from the
    format's formulas."""
    D = tiles.shape[-1] // 17
    t = torch.arange(16, device=tiles.device)[:, None]
    d = torch.arange(D, device=tiles.device)[None, :]
    lane = (t % 8) * 4 + (d % 32) // 8
    k_in = (t // 8) * (D // 8) + 4 * (d // 32) + (d % 8) // 2
    k_byte = (k_in // 16) * 512 + lane * 16 + k_in % 16
    lane = ((d % 32) // 4) * 4 + (t % 8) // 2
    v_in = (2 * (t // 8) + t % 2) * (D // 16) + 2 * (d // 32) + (d % 4) // 2
    v_byte = 8 * D + (v_in // 16) * 512 + lane * 16 + v_in % 16
    ks = 16 * D + t % 8 * (D // 16) + t // 8 * (D // 32) + d // 32
    vs = 16 * D + D // 2 + (t % 8) // 2 * (D // 8) + d // 32 * 4 + t // 8 * 2 + t % 2
    up = 4 * (d % 2)
    return (_exact_code_values((tiles[:, k_byte] >> up) & 15, tiles[:, ks]),
            _exact_code_values((tiles[:, v_byte] >> up) & 15, tiles[:, vs]))


def _exact_rows(x):
    """The values that the cache holds for x, by nearest-value search in each block."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    b = x.double().unflatten(-1, (x.shape[-1] // 32, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((amax / 6).clamp(min=2.0 ** -126)))
    e = torch.where(6 * torch.exp2(e - 1) >= amax, e - 1, e)  # log2 near a whole number
    e = torch.where(6 * torch.exp2(e) < amax, e + 1, e).clamp(-126, 125)
    y = b / torch.exp2(e)
    hi = torch.searchsorted(grid, y.abs().contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, dn = grid[hi] - y.abs(), y.abs() - grid[lo]
    pick = torch.where((up < dn) | ((up == dn) & (hi % 2 == 0)), hi, lo)
    return (torch.copysign(grid[pick], y) * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    if case["op"] == "rope":
        rot, out = s["rot"], []
        turn = s["positions"].double()[:, None, None] * s["inv_freq"].double()
        for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
            x = x.double()
            n = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
            n = n * gamma.double()
            if s["interleaved"]:
                z = torch.complex(n[..., 0:rot:2].contiguous(), n[..., 1:rot:2].contiguous())
            else:
                z = torch.complex(n[..., :rot // 2].contiguous(),
                                  n[..., rot // 2:rot].contiguous())
            z = z * torch.polar(torch.ones_like(turn), turn)
            y = n.clone()
            if s["interleaved"]:
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            else:
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            out.append(y)
        return tuple(out)
    if case["op"] == "rows":
        return _exact_rows(s["k"]), _exact_rows(s["v"])
    q, P, Hkv = s["q"].double(), s["page"], s["hkv"]
    T, Hq, D = q.shape
    G, new = Hq // Hkv, s["new"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    for r, n in enumerate(_kv_lens(case)):
        pages = s["table"][r, :(n + P - 1) // P].long()
        for h in range(Hkv):
            k, v = _exact_tiles(s["cache"][pages, h].flatten(0, 1))
            k, v = k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]
            for i in range(new):
                at = n - new + i
                if s["window"]:
                    first = max(0, at - s["window"] + 1)
                    see = torch.cat([torch.arange(min(s["sinks"], first)),
                                     torch.arange(first, at + 1)]).to(q.device)
                    kk, vv = k[see], v[see]
                else:
                    kk, vv = k[:at + 1], v[:at + 1]
                rows = q[r * new + i, h * G:(h + 1) * G]
                out[r * new + i, h * G:(h + 1) * G] = torch.softmax(
                    rows @ kk.T * s["scale"], -1) @ vv
    return out
