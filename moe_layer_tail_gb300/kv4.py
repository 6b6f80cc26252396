"""The decode step's attention block (kv4_attn.h): step tables, query/key norm with rotation,
the paged MXFP4 cache and attention over it.  Thin bindings: shapes, types and devices are
checked here, everything runs in the library's CUDA kernels on the tensors' device and, unless
`stream` is given, its current stream.

    cache = kv4_cache(n_pages, page_size, kv_heads, head_dim)
    step_tables(cached_lens, new_lens, free_pages, block_table, page_size,
                row_starts, kv_lens, positions, slots, pages_used)
    qk_norm_rope(q, k, q_gamma, k_gamma, positions, inv_freq, q, k)
    kv4_append(cache, k, v, slots)
    kv4_attention(q, cache, block_table, row_starts, kv_lens, out)
    tail.run_attn(out.view(rows, -1), residual, y)

`status` (optional everywhere): an int32 CUDA tensor of one element into which the kernels OR
KV4_STATUS_* bits; the caller zeroes it.
"""
import ctypes

KV4_STATUS_BAD_LENGTH = 16
KV4_STATUS_NO_PAGES = 32
KV4_STATUS_ROWS = 64
KV4_STATUS_BAD_SLOT = 128
KV4_STATUS_BAD_PAGE = 256


def declare(lib):
    """The argument types of kv4_attn.h's entry points (called by load_library)."""
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.moe_step_tables.argtypes = [i32] * 5 + [i64] + [P] * 11
    lib.moe_qk_norm_rope.argtypes = [i32] * 6 + [f32, P, i64, P, i64, P, P, P, P, P, i64, P, i64, P]
    lib.moe_kv4_append.argtypes = [i32] * 4 + [i64, P, P, i64, P, i64, P, P, P]
    lib.moe_kv4_read.argtypes = [i32] * 4 + [i64, P, P, i64, P, i64, P, P, P]
    lib.moe_kv4_attention.argtypes = ([i32] * 6 + [i64, P, i64, P, P, i32, i64, P, P, f32, i32, i32,
                                                   i32, P, i64, P, ctypes.c_size_t, P, P])
    lib.moe_kv4_attention_workspace.argtypes = [i32] * 4
    for name in ("moe_step_tables", "moe_qk_norm_rope", "moe_kv4_append", "moe_kv4_read",
                 "moe_kv4_attention"):
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_kv4_attention_workspace.restype = i64


def _lib():
    from . import load_library
    return load_library()


def _refuse(what, why):
    from . import ERR_INVALID_ARG, MoeTailError
    raise MoeTailError(ERR_INVALID_ARG, "%s: %s" % (what, why))


def _done(rc, what):
    if rc:
        from . import MoeTailError
        raise MoeTailError(rc, what)


class _Call:
    """The tensors of one call: each checked for type, shape and device as it is added."""

    def __init__(self, what, anchor):
        self.what = what
        if not getattr(anchor, "is_cuda", False):
            _refuse(what, "needs CUDA tensors")
        self.device = anchor.device

    def _check(self, name, t, dtype):
        if not getattr(t, "is_cuda", False) or t.device != self.device:
            _refuse(self.what, "%s must be a CUDA tensor on %s" % (name, self.device))
        if t.dtype != dtype:
            _refuse(self.what, "%s must be %s, is %s" % (name, dtype, t.dtype))

    def flat(self, name, t, dtype, n, at_least=False):
        """A contiguous 1-D tensor of n elements (or more)."""
        if t is None:
            return None
        self._check(name, t, dtype)
        if t.dim() != 1 or not t.is_contiguous() or (t.numel() < n if at_least else t.numel() != n):
            _refuse(self.what, "%s must be contiguous with %s%d elements, has shape %s"
                    % (name, "at least " if at_least else "", n, tuple(t.shape)))
        return t.data_ptr()

    def rows(self, name, t, dtype, heads=None, dim=None, rows=None):
        """[rows, heads, dim] whose rows are contiguous: (pointer, row stride)."""
        self._check(name, t, dtype)
        if (t.dim() != 3 or (heads is not None and t.shape[1] != heads)
                or (dim is not None and t.shape[2] != dim)
                or (rows is not None and t.shape[0] < rows)):
            _refuse(self.what, "%s has shape %s, expected [%s, %s, %s]"
                    % (name, tuple(t.shape), "rows" if rows is None else ">= %d" % rows,
                       "heads" if heads is None else heads, "head_dim" if dim is None else dim))
        if (t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            _refuse(self.what, "%s: a row's heads must be contiguous" % name)
        ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])
        return t.data_ptr(), ld

    def table(self, name, t, reqs):
        import torch
        self._check(name, t, torch.int32)
        if t.dim() != 2 or t.shape[0] < reqs or t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
            _refuse(self.what, "%s must be [>= %d, width] with contiguous rows, has shape %s"
                    % (name, reqs, tuple(t.shape)))
        ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])
        if ld < t.shape[1]:
            _refuse(self.what, "%s: rows overlap" % name)
        return t.data_ptr(), t.shape[1], ld

    def cache(self, t):
        """(pointer, pages, kv heads, page size, head dim) of a cache tensor."""
        import torch
        self._check("cache", t, torch.uint8)
        if t.dim() != 4 or not t.is_contiguous() or t.shape[3] % 17 or 0 in t.shape:
            _refuse(self.what, "cache must be contiguous uint8 [pages, kv_heads, page_size / 16, "
                    "17 * head_dim], has shape %s" % (tuple(t.shape),))
        return t.data_ptr(), t.shape[0], t.shape[1], t.shape[2] * 16, t.shape[3] // 17

    def status(self, t):
        import torch
        return None if t is None else self.flat("status", t, torch.int32, 1)

    def stream(self, stream):
        import torch
        if stream is None:
            return torch.cuda.current_stream(self.device).cuda_stream
        if stream.device != self.device:
            _refuse(self.what, "stream is on %s, the tensors on %s" % (stream.device, self.device))
        return stream.cuda_stream

    def guard(self):
        import torch
        return torch.cuda.device(self.device)


def kv4_cache(n_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
    """A zeroed cache: uint8 [n_pages, kv_heads, page_size / 16, 17 * head_dim]."""
    import torch
    if (n_pages < 1 or kv_heads < 1 or head_dim not in (64, 128, 256) or page_size < 16
            or page_size > 1024 or page_size % 16):
        _refuse("kv4_cache", "n_pages >= 1, page_size a multiple of 16 up to 1024, kv_heads >= 1, "
                "head_dim 64, 128 or 256")
    return torch.zeros((n_pages, kv_heads, page_size // 16, 17 * head_dim), dtype=torch.uint8,
                       device=device)


def step_tables(cached_lens, new_lens, free_pages, block_table, page_size: int, row_starts,
                kv_lens, positions, slots, pages_used, status=None, stream=None) -> None:
    """Block tables, row starts, positions and slots of one step from the requests' lengths
    (moe_step_tables).  cached_lens, new_lens int32 [reqs]; free_pages int32 [n]; block_table
    int32 [reqs, width], filled in place; row_starts int32 [reqs + 1], kv_lens int32 [reqs],
    positions int32 and slots int64 [max_rows], pages_used int32 [1]: written."""
    import torch
    c = _Call("step_tables", cached_lens)
    i32 = torch.int32
    reqs, n = cached_lens.numel(), positions.numel()
    pt, width, ld = c.table("block_table", block_table, reqs)
    args = [c.flat("cached_lens", cached_lens, i32, reqs), c.flat("new_lens", new_lens, i32, reqs),
            c.flat("free_pages", free_pages, i32, 0, True), pt,
            c.flat("row_starts", row_starts, i32, reqs + 1), c.flat("kv_lens", kv_lens, i32, reqs),
            c.flat("positions", positions, i32, n), c.flat("slots", slots, torch.int64, n),
            c.flat("pages_used", pages_used, i32, 1), c.status(status)]
    n_free = 0 if free_pages is None else free_pages.numel()
    with c.guard():
        _done(_lib().moe_step_tables(reqs, n, int(page_size), n_free, width, ld, *args,
                                     c.stream(stream)), "moe_step_tables")


def qk_norm_rope(q, k, q_gamma, k_gamma, positions, inv_freq, q_out, k_out, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """RMSNorm of every query and key head and the position rotation (moe_qk_norm_rope): q
    [rows, q_heads, D] and k [rows, k_heads, D] bf16 (or k, k_out None) with any row stride,
    gammas bf16 [D] or None (no norm on that side), positions int32 [rows], inv_freq float32
    [rot_dim / 2]; q_out may be q and k_out k."""
    import torch
    c = _Call("qk_norm_rope", q)
    bf = torch.bfloat16
    pq, ldq = c.rows("q", q, bf)
    T, hq, D = q.shape
    pqo, ldqo = c.rows("q_out", q_out, bf, hq, D, T)
    hk, pk, ldk, pko, ldko = 0, None, 0, None, 0
    if k is not None:
        pk, ldk = c.rows("k", k, bf, None, D, T)
        hk = k.shape[1]
        if k_out is None:
            _refuse("qk_norm_rope", "k without k_out")
        pko, ldko = c.rows("k_out", k_out, bf, hk, D, T)
    gq = c.flat("q_gamma", q_gamma, bf, D)
    gk = c.flat("k_gamma", k_gamma, bf, D)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    pos = c.flat("positions", positions, torch.int32, T, True)
    fr = c.flat("inv_freq", inv_freq, torch.float32, rot // 2)
    with c.guard():
        _done(_lib().moe_qk_norm_rope(T, hq, hk, D, rot, int(bool(interleaved)), float(eps), pq, ldq,
                                      pk, ldk, gq, gk, pos, fr, pqo, ldqo, pko, ldko,
                                      c.stream(stream)), "moe_qk_norm_rope")


def _cache_rows(what, fn, cache, k, v, slots, status, stream):
    import torch
    c = _Call(what, cache)
    pc, n_pages, heads, page, D = c.cache(cache)
    T = slots.numel()
    ps = c.flat("slots", slots, torch.int64, T)
    pk, ldk = c.rows("k", k, torch.bfloat16, heads, D, T)
    pv, ldv = c.rows("v", v, torch.bfloat16, heads, D, T)
    with c.guard():
        _done(fn(T, heads, D, page, n_pages, pc, pk, ldk, pv, ldv, ps, c.status(status),
                 c.stream(stream)), "moe_" + what)


def kv4_append(cache, k, v, slots, status=None, stream=None) -> None:
    """Quantise k, v bf16 [rows, kv_heads, D] (any row stride) into slots int64 [rows] of the
    cache (moe_kv4_append); negative slots are skipped."""
    _cache_rows("kv4_append", _lib().moe_kv4_append, cache, k, v, slots, status, stream)


def kv4_read(cache, slots, k, v, status=None, stream=None) -> None:
    """The cache's values in slots int64 [rows] into k, v bf16 [rows, kv_heads, D] (exact)."""
    _cache_rows("kv4_read", _lib().moe_kv4_read, cache, k, v, slots, status, stream)


def kv4_attention_workspace(q_heads: int, kv_heads: int, head_dim: int, max_new: int = 1,
                            device=None) -> int:
    """Bytes of workspace that kv4_attention needs on `device` (default: the current one)."""
    import torch
    with torch.cuda.device(device):
        n = _lib().moe_kv4_attention_workspace(int(q_heads), int(kv_heads), int(head_dim),
                                               int(max_new))
    if n < 0:
        _done(int(n), "moe_kv4_attention_workspace")
    return int(n)


def kv4_attention(q, cache, block_table, row_starts, kv_lens, out, scale: float = None,
                  window: int = 0, sinks: int = 0, max_new: int = 1, workspace=None, status=None,
                  stream=None) -> None:
    """Attention of the step's rows over the cache (moe_kv4_attention): q, out bf16 [rows,
    q_heads, D]; block_table int32 [reqs, width], row_starts int32 [reqs + 1], kv_lens int32
    [reqs].  scale defaults to D ** -0.5; window 0 sees everything up to the row's position,
    otherwise the last `window` tokens and the first `sinks`.  workspace: uint8, at least
    kv4_attention_workspace bytes, not shared with a call that may run at the same time (two
    captured graphs replayed in different streams need two); None takes one from PyTorch's
    allocator for this call."""
    import torch
    c = _Call("kv4_attention", q)
    pc, n_pages, heads, page, D = c.cache(cache)
    pq, ldq = c.rows("q", q, torch.bfloat16, None, D)
    T, hq = q.shape[0], q.shape[1]
    po, ldo = c.rows("out", out, torch.bfloat16, hq, D, T)
    reqs = kv_lens.numel()
    pt, width, ld = c.table("block_table", block_table, reqs)
    prs = c.flat("row_starts", row_starts, torch.int32, reqs + 1)
    pkl = c.flat("kv_lens", kv_lens, torch.int32, reqs)
    with c.guard():
        lib = _lib()
        if workspace is None:
            n = kv4_attention_workspace(hq, heads, D, max_new, c.device)
            # memory of the launching stream: the allocator reuses it only behind this call
            with torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=c.device)
        pw = c.flat("workspace", workspace, torch.uint8, 0, True)
        _done(lib.moe_kv4_attention(T, reqs, hq, heads, D, page, n_pages, pq, ldq, pc, pt, width, ld,
                                    prs, pkl, float(D ** -0.5 if scale is None else scale),
                                    int(window), int(sinks), int(max_new), po, ldo, pw,
                                    workspace.numel(), c.status(status), c.stream(stream)),
              "moe_kv4_attention")
