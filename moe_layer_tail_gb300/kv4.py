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
`stream` (optional everywhere): the torch.cuda.Stream to launch in, in place of the current one.
PyTorch's allocator does not learn of it: the caller keeps the tensors alive until the work there
has passed them (or calls record_stream on them).
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
    lib.moe_tail_debug_kv4_stall.argtypes = [i32]
    for name in ("moe_step_tables", "moe_qk_norm_rope", "moe_kv4_append", "moe_kv4_read",
                 "moe_kv4_attention"):
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_kv4_attention_workspace.restype = i64


def _refuse(what, why):
    from . import ERR_INVALID_ARG, MoeTailError
    raise MoeTailError(ERR_INVALID_ARG, "%s: %s" % (what, why))


def _failed(rc, what):
    from . import MoeTailError
    raise MoeTailError(rc, what)


# The checks below run on every call of a decode step, so they stay close to the bare attribute
# reads: a step of small kernels is otherwise bound by its host side.

_torch = None
_library = None


def _begin(what, anchor):
    """(torch, the library, the CUDA device index of `anchor`)."""
    global _torch, _library
    if _library is None:
        import torch
        from . import load_library
        _torch, _library = torch, load_library()
    dev = anchor.get_device()
    if dev < 0:
        _refuse(what, "needs CUDA tensors")
    return _torch, _library, dev


def _wrong(what, name, t, dtype, dev):
    if not getattr(t, "is_cuda", False) or t.get_device() != dev:
        _refuse(what, "%s must be a CUDA tensor on cuda:%d" % (name, dev))
    _refuse(what, "%s must be %s, is %s" % (name, dtype, t.dtype))


def _flat(what, name, t, dtype, dev, n, more=False):
    """The address of a contiguous 1-D tensor of n elements (or more)."""
    if t.dtype is not dtype or t.get_device() != dev:
        _wrong(what, name, t, dtype, dev)
    have = t.numel()
    if t.dim() != 1 or not t.is_contiguous() or (have < n if more else have != n):
        _refuse(what, "%s must be contiguous with %s%d elements, has shape %s"
                % (name, "at least " if more else "", n, tuple(t.shape)))
    return t.data_ptr()


def _rows(what, name, t, dtype, dev, heads, dim, rows):
    """The address and row stride of [>= rows, heads, dim] whose rows are contiguous."""
    if t.dtype is not dtype or t.get_device() != dev:
        _wrong(what, name, t, dtype, dev)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or shape[0] < rows:
        _refuse(what, "%s has shape %s, expected [>= %d, %d, %d]"
                % (name, tuple(shape), rows, heads, dim))
    ld, sh, sd = t.stride()
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim):
        _refuse(what, "%s: a row's heads must be contiguous" % name)
    if shape[0] == 1 and ld < heads * dim:
        ld = heads * dim  # (one row: its stride says nothing)
    return t.data_ptr(), ld


def _table(what, t, dev, reqs, i32):
    """The address, width and row stride of a block table [>= reqs, width]."""
    if t.dtype is not i32 or t.get_device() != dev:
        _wrong(what, "block_table", t, i32, dev)
    shape = t.shape
    if len(shape) != 2 or shape[0] < reqs or shape[1] < 1 or (shape[1] > 1 and t.stride(1) != 1):
        _refuse(what, "block_table must be [>= %d, width] with contiguous rows, has shape %s"
                % (reqs, tuple(shape)))
    ld = t.stride(0)
    if ld < shape[1]:
        if shape[0] > 1:
            _refuse(what, "block_table: rows overlap")
        ld = shape[1]
    return t.data_ptr(), shape[1], ld


def _cache(what, t, dev, u8):
    """The address, pages, kv heads, page size and head dim of a cache tensor."""
    if t.dtype is not u8 or t.get_device() != dev:
        _wrong(what, "cache", t, u8, dev)
    shape = t.shape
    if len(shape) != 4 or shape[3] % 17 or 0 in shape or not t.is_contiguous():
        _refuse(what, "cache must be contiguous uint8 [pages, kv_heads, page_size / 16, "
                "17 * head_dim], has shape %s" % (tuple(shape),))
    return t.data_ptr(), shape[0], shape[1], shape[2] * 16, shape[3] // 17


def _launch(what, torch, dev, stream, call):
    """Run call(raw stream) with `dev` current, on its current stream or the given one."""
    if stream is not None and stream.device.index != dev:
        _refuse(what, "stream is on %s, the tensors on cuda:%d" % (stream.device, dev))
    if torch._C._cuda_getDevice() == dev:
        rc = call(torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = call(torch._C._cuda_getCurrentRawStream(dev) if stream is None
                      else stream.cuda_stream)
    if rc:
        _failed(rc, "moe_" + what)


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
    (moe_step_tables).  cached_lens, new_lens int32 [reqs]; free_pages int32 [n] or None;
    block_table int32 [reqs, width], filled in place; row_starts int32 [reqs + 1], kv_lens int32
    [reqs], positions int32 and slots int64 [max_rows], pages_used int32 [1]: written.  A step of
    more than max_rows rows is cut to its first ones (KV4_STATUS_ROWS): kv_lens and pages_used
    count the rows that are left."""
    w = "step_tables"
    torch, lib, dev = _begin(w, cached_lens)
    i32 = torch.int32
    reqs, n = cached_lens.numel(), positions.numel()
    n_free = 0 if free_pages is None else free_pages.numel()
    pt, width, ld = _table(w, block_table, dev, reqs, i32)
    args = (reqs, n, page_size, n_free, width, ld,
            _flat(w, "cached_lens", cached_lens, i32, dev, reqs),
            _flat(w, "new_lens", new_lens, i32, dev, reqs),
            _flat(w, "free_pages", free_pages, i32, dev, n_free) if n_free else None, pt,
            _flat(w, "row_starts", row_starts, i32, dev, reqs + 1),
            _flat(w, "kv_lens", kv_lens, i32, dev, reqs),
            _flat(w, "positions", positions, i32, dev, n),
            _flat(w, "slots", slots, torch.int64, dev, n),
            _flat(w, "pages_used", pages_used, i32, dev, 1),
            None if status is None else _flat(w, "status", status, i32, dev, 1))
    _launch(w, torch, dev, stream, lambda st: lib.moe_step_tables(*args, st))


def qk_norm_rope(q, k, q_gamma, k_gamma, positions, inv_freq, q_out, k_out, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """RMSNorm of every query and key head and the position rotation (moe_qk_norm_rope): q
    [rows, q_heads, D] and k [rows, k_heads, D] bf16 (or k, k_out None) with any row stride,
    gammas bf16 [D] or None (no norm on that side), positions int32 [rows], inv_freq float32
    [rot_dim / 2] (None: no rotation); q_out may be q and k_out k."""
    w = "qk_norm_rope"
    torch, lib, dev = _begin(w, q)
    bf = torch.bfloat16
    if q.dim() != 3:
        _refuse(w, "q must be [rows, heads, head_dim], has shape %s" % (tuple(q.shape),))
    T, hq, D = q.shape
    pq, ldq = _rows(w, "q", q, bf, dev, hq, D, T)
    pqo, ldqo = _rows(w, "q_out", q_out, bf, dev, hq, D, T)
    hk, pk, ldk, pko, ldko = 0, None, 0, None, 0
    if k is not None:
        if k_out is None or k.dim() != 3:
            _refuse(w, "k must be [rows, heads, head_dim] and come with k_out")
        hk = k.size(1)
        pk, ldk = _rows(w, "k", k, bf, dev, hk, D, T)
        pko, ldko = _rows(w, "k_out", k_out, bf, dev, hk, D, T)
    half = 0 if inv_freq is None else inv_freq.numel()
    args = (T, hq, hk, D, 2 * half, 1 if interleaved else 0, eps, pq, ldq, pk, ldk,
            None if q_gamma is None else _flat(w, "q_gamma", q_gamma, bf, dev, D),
            None if k_gamma is None else _flat(w, "k_gamma", k_gamma, bf, dev, D),
            None if positions is None else _flat(w, "positions", positions, torch.int32, dev, T, True),
            None if not half else _flat(w, "inv_freq", inv_freq, torch.float32, dev, half),
            pqo, ldqo, pko, ldko)
    _launch(w, torch, dev, stream, lambda st: lib.moe_qk_norm_rope(*args, st))


def _cache_rows(w, torch, lib, dev, fn, cache, k, v, slots, status, stream):
    bf = torch.bfloat16
    pc, n_pages, heads, page, D = _cache(w, cache, dev, torch.uint8)
    T = slots.numel()
    ps = _flat(w, "slots", slots, torch.int64, dev, T)
    pk, ldk = _rows(w, "k", k, bf, dev, heads, D, T)
    pv, ldv = _rows(w, "v", v, bf, dev, heads, D, T)
    st = None if status is None else _flat(w, "status", status, torch.int32, dev, 1)
    _launch(w, torch, dev, stream,
            lambda s: fn(T, heads, D, page, n_pages, pc, pk, ldk, pv, ldv, ps, st, s))


def kv4_append(cache, k, v, slots, status=None, stream=None) -> None:
    """Quantise k, v bf16 [rows, kv_heads, D] (any row stride) into slots int64 [rows] of the
    cache (moe_kv4_append); negative slots are skipped."""
    torch, lib, dev = _begin("kv4_append", cache)
    _cache_rows("kv4_append", torch, lib, dev, lib.moe_kv4_append, cache, k, v, slots, status, stream)


def kv4_read(cache, slots, k, v, status=None, stream=None) -> None:
    """The cache's values in slots int64 [rows] into k, v bf16 [rows, kv_heads, D] (exact)."""
    torch, lib, dev = _begin("kv4_read", cache)
    _cache_rows("kv4_read", torch, lib, dev, lib.moe_kv4_read, cache, k, v, slots, status, stream)


_workspace_bytes = {}  # (device, q heads, kv heads, head dim, max_new) -> bytes


def kv4_attention_workspace(q_heads: int, kv_heads: int, head_dim: int, max_new: int = 1,
                            device=None) -> int:
    """Bytes of workspace that kv4_attention needs on `device` (default: the current one)."""
    import torch
    from . import load_library
    with torch.cuda.device(device):
        n = load_library().moe_kv4_attention_workspace(int(q_heads), int(kv_heads), int(head_dim),
                                                       int(max_new))
    if n < 0:
        _failed(int(n), "moe_kv4_attention_workspace")
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
    allocator for this call, which a graph captured by torch.cuda.graph keeps; a capture begun in
    any other way must be given one, since nothing would keep that memory for its replays.  A call of more than 2^31 - 1 tiles of 16 tokens (counted for each kv
    head and 32 rows: some 90000 rows of a prompt with 16 query heads to each of 8 kv heads) gives
    NaN and KV4_STATUS_BAD_LENGTH: cut the prompt into several calls."""
    w = "kv4_attention"
    torch, lib, dev = _begin(w, q)
    i32, bf = torch.int32, torch.bfloat16
    pc, n_pages, heads, page, D = _cache(w, cache, dev, torch.uint8)
    if q.dim() != 3:
        _refuse(w, "q must be [rows, heads, head_dim], has shape %s" % (tuple(q.shape),))
    T, hq, _ = q.shape
    pq, ldq = _rows(w, "q", q, bf, dev, hq, D, T)
    po, ldo = _rows(w, "out", out, bf, dev, hq, D, T)
    reqs = kv_lens.numel()
    pt, width, ld = _table(w, block_table, dev, reqs, i32)
    prs = _flat(w, "row_starts", row_starts, i32, dev, reqs + 1)
    pkl = _flat(w, "kv_lens", kv_lens, i32, dev, reqs)
    st = None if status is None else _flat(w, "status", status, i32, dev, 1)
    sc = D ** -0.5 if scale is None else scale
    if workspace is not None:
        n = workspace.numel()
        pw = _flat(w, "workspace", workspace, torch.uint8, dev, n)
        _launch(w, torch, dev, stream, lambda s: lib.moe_kv4_attention(
            T, reqs, hq, heads, D, page, n_pages, pq, ldq, pc, pt, width, ld, prs, pkl, sc, window,
            sinks, max_new, po, ldo, pw, n, st, s))
        return
    key = (dev, hq, heads, D, max_new)
    n = _workspace_bytes.get(key)
    if n is None:
        n = _workspace_bytes[key] = kv4_attention_workspace(hq, heads, D, max_new, dev)

    def call(s):
        # memory of the launching stream: the allocator reuses it only behind this call (a tensor
        # would do, for 5 us more on the host)
        p = torch._C._cuda_cudaCachingAllocator_raw_alloc(n, s)
        try:
            return lib.moe_kv4_attention(
                T, reqs, hq, heads, D, page, n_pages, pq, ldq, pc, pt, width, ld, prs, pkl, sc, window,
                sinks, max_new, po, ldo, p, n, st, s)
        finally:
            torch._C._cuda_cudaCachingAllocator_raw_delete(p)

    _launch(w, torch, dev, stream, call)
