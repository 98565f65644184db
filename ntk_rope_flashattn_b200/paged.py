"""The paged key/value cache: ``PagedCache`` and the calls that work on it
(``pages_extend``, ``pages_fork``, ``pages_free``, ``pages_compact``,
``pages_copy``, ``paged_append``, ``paged_decode``; see ``include/lcx.h``).

    cache = lcx.PagedCache(num_pages=4096, page_size=16, kv_heads=8, head_dim=128,
                           max_seqs=64, max_pages_per_seq=512, num_layers=32)
    start = lcx.pages_extend(cache, seq_ids, n_new)       # room for the new tokens
    for layer in range(32):
        lcx.paged_append(cache, k, v, seq_ids, start, rope, layer=layer, cu_new=cu)
        o = lcx.paged_decode(cache, q, seq_ids, rope, layer=layer)

All bookkeeping lives on the device and no call synchronises, so a decode step
(extend, append, decode) can be captured into a CUDA graph and replayed.  Index
arguments are int32 CUDA tensors; a negative sequence number marks a padded entry
that every call leaves out.  What the device finds wrong (a bad number, no free
page) skips the entry and is reported through the optional ``status`` tensor
(one int32; written, never cleared).
"""
import ctypes
import functools
import struct

from . import RopeParams, _check, _dtype_code, _RopeParams, load

LCX_ERR_NO_PAGES = 5
LCX_PAGES_MAX_ENTRIES = 1024
LCX_DECODE_PREROTATED = 1

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Cache(ctypes.Structure):
    _fields_ = [("k_pages", _P), ("v_pages", _P), ("block_table", _P), ("seq_lens", _P),
                ("ref_counts", _P), ("free_pages", _P), ("n_free", _P), ("scratch", _P),
                ("dtype", _I32), ("page_size", _I32), ("num_layers", _I64), ("num_pages", _I64),
                ("Hkv", _I64), ("D", _I64), ("max_seqs", _I64), ("max_pages", _I64),
                ("k_strides", _I64 * 5), ("v_strides", _I64 * 5)]


class _AppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("q", _P), ("q_out", _P), ("k_out", _P), ("seq_ids", _P),
                ("start", _P), ("cu_new", _P), ("dev_status", _P), ("n", _I64), ("T", _I64),
                ("Hq", _I64), ("layer", _I64), ("k_strides", _I64 * 3), ("v_strides", _I64 * 3),
                ("q_strides", _I64 * 3), ("q_out_strides", _I64 * 3),
                ("k_out_strides", _I64 * 3), ("rope", _RopeParams)]


class _DecodeArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("o", _P), ("lse", _P), ("seq_ids", _P), ("dev_status", _P),
                ("n", _I64), ("Hq", _I64), ("layer", _I64), ("q_strides", _I64 * 3),
                ("o_strides", _I64 * 3), ("rope", _RopeParams), ("window", _I64),
                ("sinks", _I64), ("softmax_scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


_CODES = {_P: "P", _I64: "q", _I32: "i", ctypes.c_uint32: "I", ctypes.c_float: "f"}


def _packer(cls):
    """pack(*values) -> the bytes of a cls (three times as fast as filling one): arrays
    spread, a NULL as 0, structs inside as bytes."""
    fmt = ""
    for _, t in cls._fields_:
        if issubclass(t, ctypes.Array):
            fmt += "%d%s" % (t._length_, _CODES[t._type_])
        elif issubclass(t, ctypes.Structure):
            fmt += "%ds" % ctypes.sizeof(t)
        else:
            fmt += _CODES[t]
    s = struct.Struct("@" + fmt + "0q")
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_append, _pack_decode = _packer(_AppendArgs), _packer(_DecodeArgs)


@functools.lru_cache(maxsize=None)
def _raw(name, pointers, sizes=0):
    """The entry point under argument types that take packed structs: `pointers`
    addresses (or bytes), `sizes` int64 values, the stream."""
    fn = load()[name]
    fn.argtypes = [_P] * pointers + [_I64] * sizes + [_P]
    fn.restype = ctypes.c_int
    return fn


def _declare(lib):
    c = ctypes.POINTER(_Cache)
    lib.lcx_paged_scratch_ints.argtypes = [_I64]
    lib.lcx_paged_scratch_ints.restype = _I64
    lib.lcx_pages_extend.argtypes = [c, _P, _P, _I64, _P, _P, _P]
    lib.lcx_pages_fork.argtypes = [c, _P, _P, _I64, _P, _P]
    lib.lcx_pages_free.argtypes = [c, _P, _I64, _P, _P]
    lib.lcx_pages_compact.argtypes = [c, _P, _P]
    lib.lcx_pages_copy.argtypes = [c, _P, _P, _I64, _P, _P]
    lib.lcx_paged_append.argtypes = [c, ctypes.POINTER(_AppendArgs), _P]
    lib.lcx_paged_decode.argtypes = [c, ctypes.POINTER(_DecodeArgs), _P, _I64, _P]
    lib.lcx_paged_decode_workspace_bytes.argtypes = [_I64] * 4
    lib.lcx_paged_decode_workspace_bytes.restype = _I64
    for f in ("extend", "fork", "free", "compact", "copy"):
        getattr(lib, "lcx_pages_" + f).restype = ctypes.c_int
    lib.lcx_paged_append.restype = lib.lcx_paged_decode.restype = ctypes.c_int


_FIXED = frozenset(("k_pages", "v_pages", "meta", "block_table", "seq_lens", "ref_counts",
                    "free_pages", "n_free", "scratch", "num_pages", "page_size", "kv_heads",
                    "head_dim", "max_seqs", "max_pages_per_seq", "num_layers", "dtype", "device",
                    "_struct", "_dev"))


class PagedCache:
    """A key/value cache in pages (mirrors ``lcx_paged_cache``).

    ``k_pages`` / ``v_pages`` are [num_layers, num_pages, page_size, kv_heads,
    head_dim], allocated with each head's slots of a page together (or passed in,
    strided as they are).  ``meta`` is the whole bookkeeping in one int32 tensor
    (copy it to save or restore the state); ``block_table``, ``seq_lens``,
    ``ref_counts``, ``free_pages`` and ``n_free`` are views of it.  Calls on one
    cache must be ordered: one stream, or events between streams."""

    def __init__(self, num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages_per_seq,
                 num_layers=1, dtype=None, device="cuda", k_pages=None, v_pages=None):
        import torch
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("a PagedCache lives on a CUDA device (got %s)" % device)
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        dtype = torch.bfloat16 if dtype is None else dtype
        sizes = dict(num_pages=num_pages, page_size=page_size, kv_heads=kv_heads,
                     head_dim=head_dim, max_seqs=max_seqs, max_pages_per_seq=max_pages_per_seq,
                     num_layers=num_layers)
        for name, x in sizes.items():
            if int(x) <= 0:
                raise ValueError("%s must be positive (got %s)" % (name, x))
            setattr(self, name, int(x))
        shape = (self.num_layers, self.num_pages, self.page_size, self.kv_heads, self.head_dim)
        self.device, self.dtype, self._dev = device, dtype, device.index
        pools = []
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t is None:
                t = torch.zeros((shape[0], shape[1], shape[3], shape[2], shape[4]), dtype=dtype,
                                device=device).transpose(2, 3)
            if tuple(t.shape) != shape or t.dtype != dtype or t.device != device:
                raise ValueError("%s must be %s of %s on %s" % (name, shape, dtype, device))
            pools.append(t)
        self.k_pages, self.v_pages = pools
        n_scratch = int(load().lcx_paged_scratch_ints(self.num_pages))
        if n_scratch < 0:
            raise ValueError("num_pages %d is out of range" % self.num_pages)
        a, b, p = self.max_seqs * self.max_pages_per_seq, self.max_seqs, self.num_pages
        self.meta = torch.empty(a + b + 2 * p + 1, dtype=torch.int32, device=device)
        self.block_table = self.meta[:a].view(self.max_seqs, self.max_pages_per_seq)
        self.seq_lens = self.meta[a:a + b]
        self.ref_counts = self.meta[a + b:a + b + p]
        self.free_pages = self.meta[a + b + p:a + b + 2 * p]
        self.n_free = self.meta[a + b + 2 * p:]
        self.scratch = torch.zeros(n_scratch, dtype=torch.int32, device=device)
        self._struct = ctypes.byref(self._c())
        self._workspace_bytes = {}
        self.reset()

    def __setattr__(self, name, value):
        # the C struct holds the buffers' addresses
        if ("_struct" in self.__dict__ and name in _FIXED and
                value is not self.__dict__[name]):
            raise AttributeError("%s of a PagedCache does not change (copy into it)" % name)
        object.__setattr__(self, name, value)

    def reset(self):
        """Empty the cache: every page free, every sequence without tokens."""
        import torch
        self.block_table.fill_(-1)
        self.seq_lens.zero_()
        self.ref_counts.zero_()
        self.free_pages.copy_(torch.arange(self.num_pages - 1, -1, -1, dtype=torch.int32,
                                           device=self.device))
        self.n_free.fill_(self.num_pages)
        self.scratch.zero_()

    def _c(self):
        c = _Cache()
        for f in ("k_pages", "v_pages", "block_table", "seq_lens", "ref_counts", "free_pages",
                  "n_free", "scratch"):
            setattr(c, f, getattr(self, f).data_ptr())
        c.dtype = _dtype_code(self.k_pages)
        c.page_size, c.num_layers, c.num_pages = self.page_size, self.num_layers, self.num_pages
        c.Hkv, c.D = self.kv_heads, self.head_dim
        c.max_seqs, c.max_pages = self.max_seqs, self.max_pages_per_seq
        c.k_strides = (_I64 * 5)(*self.k_pages.stride())
        c.v_strides = (_I64 * 5)(*self.v_pages.stride())
        return c


def _index(cache, **tensors):
    """Index arguments: contiguous int32 vectors on the cache's device."""
    import torch
    out, dev, int32 = [], cache._dev, torch.int32
    for name, t in tensors.items():
        if t is None:
            out.append(0)
            continue
        if not isinstance(t, torch.Tensor) or t.dtype is not int32 or t.dim() != 1:
            raise ValueError("%s must be a 1-D int32 tensor" % name)
        if t.get_device() != dev:
            raise ValueError("%s must be a CUDA tensor on %s (got %s)" % (name, cache.device,
                                                                         t.device))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        out.append(t.data_ptr())
    return out


def _on_device(dev, **tensors):
    """Every tensor given (None skipped) must lie on CUDA device `dev`."""
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError("%s must be a CUDA tensor on cuda:%d (got %s)" % (name, dev, t.device))


def _current_stream(dev):
    """The handle of device `dev`'s current stream (without a Stream object, where torch
    gives it so: 0.2 instead of 1.3 us)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw else torch.cuda.current_stream(dev).cuda_stream


def _call_on(dev, call, *args):
    """call(*args, stream) with device `dev` current, on its current stream."""
    import torch
    if torch.cuda.current_device() == dev:
        _check(call(*args, _current_stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(call(*args, _current_stream(dev)))


def _launch(cache, call, *args):
    _call_on(cache._dev, call, *args)


def pages_extend(cache, seq_ids, n_new=None, start=None, status=None):
    """Sequence seq_ids[i] grows by n_new[i] tokens (one each without n_new).
    Returns ``start``: the position of each entry's first new token, -1 where the
    entry was skipped (padded, refused, or out of pages; see lcx_pages_extend)."""
    import torch
    if n_new is not None and n_new.shape != seq_ids.shape:
        raise ValueError("n_new must have one value per entry")
    if start is None:
        start = torch.empty_like(seq_ids)
    elif start.shape != seq_ids.shape:
        raise ValueError("start must have one value per entry")
    ids, nn, st, word = _index(cache, seq_ids=seq_ids, n_new=n_new, start=start, status=status)
    _launch(cache, load().lcx_pages_extend, cache._struct, ids, nn, seq_ids.numel(), st, word)
    return start


def pages_fork(cache, src, dst, status=None):
    """Sequence dst[i] (empty) becomes a copy of src[i]: full pages shared, a partial
    last page copied (lcx_pages_fork)."""
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    a, b, word = _index(cache, src=src, dst=dst, status=status)
    _launch(cache, load().lcx_pages_fork, cache._struct, a, b, src.numel(), word)


def pages_free(cache, seq_ids, status=None):
    """The sequences end; pages nobody holds return to the free stack."""
    ids, word = _index(cache, seq_ids=seq_ids, status=status)
    _launch(cache, load().lcx_pages_free, cache._struct, ids, seq_ids.numel(), word)


def pages_compact(cache, status=None):
    """Move the used pages to the lowest numbers (lcx_pages_compact)."""
    word, = _index(cache, status=status)
    _launch(cache, load().lcx_pages_compact, cache._struct, word)


def pages_copy(cache, src_pages, dst_pages, status=None):
    """Copy page src_pages[i] to dst_pages[i] in every layer (lcx_pages_copy)."""
    if src_pages.shape != dst_pages.shape:
        raise ValueError("src_pages and dst_pages must have the same length")
    a, b, word = _index(cache, src_pages=src_pages, dst_pages=dst_pages, status=status)
    _launch(cache, load().lcx_pages_copy, cache._struct, a, b, src_pages.numel(), word)


def _tokens(t, name, heads, D, dtype):
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != D:
        raise ValueError("%s must be [tokens, %s, %d], got %s" % (name, heads or "heads", D,
                                                                  tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))


@functools.lru_cache(maxsize=64)
def _rope_struct(*fields):
    c = RopeParams(*fields)._c()
    return c, bytes(c)


def _rope_c(rope):
    """The rope's C struct and its bytes, one per set of field values (factor tables may
    change in place: built anew; the struct keeps the arrays that the bytes point to)."""
    if rope.factors is not None or rope.factors_short is not None:
        c = rope._c()
        return c, bytes(c)
    return _rope_struct(rope.mode, int(rope.head_dim), float(rope.base), float(rope.scale),
                        int(rope.original_max_pos), float(rope.alpha), float(rope.beta),
                        rope.pairing, int(rope.seq_len))


def paged_append(cache, k, v, seq_ids, start, rope: RopeParams, layer: int = 0, cu_new=None,
                 q=None, q_out=None, k_out=None, status=None):
    """Rotate new keys k [T, Hkv, D] and write them and v into their pages of one
    layer; entry i's tokens are rows cu_new[i] .. cu_new[i + 1] - 1 (row i without
    cu_new) at positions from start[i] on (``pages_extend`` gives it).  With q
    [T, Hq, D] the queries are rotated along, into q_out (allocated when not
    given; q itself rotates in place).  k_out receives the rotated keys packed
    like k.  Rows of skipped entries are not written: those of a q_out that the call
    allocates hold nothing.  Returns q_out (None without q)."""
    import torch
    _on_device(cache._dev, k=k, v=v, q=q, q_out=q_out, k_out=k_out)
    H, D = cache.kv_heads, cache.head_dim
    _tokens(k, "k", H, D, cache.dtype)
    _tokens(v, "v", H, D, cache.dtype)
    T = k.shape[0]
    if v.shape != k.shape:
        raise ValueError("shape mismatch: k %s v %s" % (tuple(k.shape), tuple(v.shape)))
    if start.shape != seq_ids.shape:
        raise ValueError("start must have one value per entry")
    if cu_new is not None and cu_new.shape != (seq_ids.shape[0] + 1,):
        raise ValueError("cu_new must have one value more than seq_ids")
    if cu_new is None and T != seq_ids.shape[0]:
        raise ValueError("without cu_new k must have one row per entry")
    ids, st, cu, word = _index(cache, seq_ids=seq_ids, start=start, cu_new=cu_new, status=status)
    Hq = 0
    if q is not None:
        _tokens(q, "q", None, D, cache.dtype)
        if q.shape[0] != T:
            raise ValueError("q must have k's %d rows" % T)
        if q_out is None:
            q_out = torch.empty_like(q)
        Hq = q.shape[1]
        _tokens(q_out, "q_out", Hq, D, cache.dtype)
        if q_out.shape != q.shape:
            raise ValueError("q_out must be shaped like q")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is not None:
        _tokens(k_out, "k_out", H, D, cache.dtype)
        if k_out.shape != k.shape:
            raise ValueError("k_out must be shaped like k")
    none = (0, 0, 0)
    owner, rope_c = _rope_c(rope)      # (alive during the call: it owns factor tables)
    a = _pack_append(
        k.data_ptr(), v.data_ptr(), 0 if q is None else q.data_ptr(),
        0 if q is None else q_out.data_ptr(), 0 if k_out is None else k_out.data_ptr(), ids, st,
        cu, word, seq_ids.shape[0], T, Hq, int(layer), *k.stride(), *v.stride(),
        *(none if q is None else q.stride()), *(none if q is None else q_out.stride()),
        *(none if k_out is None else k_out.stride()), rope_c)
    _launch(cache, _raw("lcx_paged_append", 2), cache._struct, a)
    return q_out


def paged_decode_workspace_bytes(cache, n, q_heads) -> int:
    """Workspace bytes of ``paged_decode`` for n entries (lcx_paged_decode_workspace_bytes)."""
    need = cache._workspace_bytes.get((n, q_heads))
    if need is None:
        import torch
        with torch.cuda.device(cache.device):
            need = int(load().lcx_paged_decode_workspace_bytes(int(n), int(q_heads),
                                                               cache.kv_heads, cache.head_dim))
        if need < 0:
            raise ValueError("paged_decode: sizes out of range (%d entries, %d heads)" %
                             (n, q_heads))
        cache._workspace_bytes[(n, q_heads)] = need
    return need


def paged_decode(cache, q, seq_ids, rope: RopeParams, layer: int = 0, window: int = 0,
                 sinks: int = 0, softmax_scale: float = 0.0, prerotated: bool = False,
                 return_lse: bool = False, out=None, lse=None, workspace=None, status=None):
    """Attention of one new token per entry, q [n, Hq, D], over its sequence's
    cached keys (its own among them).  Returns o [n, Hq, D] (and lse [n, Hq] fp32
    if asked).  ``prerotated``: q is already rotated (``paged_append``'s q_out);
    else it is rotated at the sequence's last position.  ``workspace`` (uint8 CUDA
    tensor, 256-byte aligned) is allocated when not given; calls in flight at the
    same time, replayed graphs among them, must not share one."""
    import torch
    _on_device(cache._dev, q=q, out=out, lse=lse, workspace=workspace)
    _tokens(q, "q", None, cache.head_dim, cache.dtype)
    n, Hq = q.shape[0], q.shape[1]
    if seq_ids.shape != (n,):
        raise ValueError("seq_ids must have one value per row of q")
    ids, word = _index(cache, seq_ids=seq_ids, status=status)
    o = out if out is not None else torch.empty_like(q, memory_format=torch.contiguous_format)
    _tokens(o, "out", Hq, cache.head_dim, cache.dtype)
    if o.shape != q.shape:
        raise ValueError("out must be shaped like q")
    if return_lse and lse is None:
        lse = q.new_empty((n, Hq), dtype=torch.float32)
    if lse is not None and (lse.shape != (n, Hq) or lse.dtype != torch.float32 or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [%d, %d]" % (n, Hq))
    if workspace is None and Hq % cache.kv_heads == 0:
        need = paged_decode_workspace_bytes(cache, n, Hq)
        workspace = q.new_empty(max(need, 1), dtype=torch.uint8)
    owner, rope_c = _rope_c(rope)      # (alive during the call: it owns factor tables)
    a = _pack_decode(q.data_ptr(), o.data_ptr(), 0 if lse is None else lse.data_ptr(), ids, word,
                     n, Hq, int(layer), *q.stride(), *o.stride(), rope_c, int(window), int(sinks),
                     float(softmax_scale), LCX_DECODE_PREROTATED if prerotated else 0)
    ws, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _launch(cache, _raw("lcx_paged_decode", 3, 1), cache._struct, a, ws, size)
    return (o, lse) if return_lse else o
