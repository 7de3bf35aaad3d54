"""A paged KV cache held in 4 bits on AMD MI355X, and the operators on it.

Where a received KV (see ``transfer``) is kept for decoding: ``append`` quantizes keys and values
into pages, ``attend`` reads them back as matrix operands on the fly, ``weigh`` adds up how much
attention each token gets, ``evict`` cuts sequences down to the tokens that got most of it.  Every
step runs in the HIP kernels of ``libsplitzip.so`` (include/splitzip_kv4.h); this module marshals
arguments.  No call waits for the GPU, so all may be captured into a graph.

A value costs 4.25 bits: E2M1 codes with a power-of-two scale for each 32 channels of a token.

A call's sequences are given by ``table`` (int32 [seqs, pages], the page numbers of each sequence),
``lens`` (int32 [seqs], tokens with the new ones) and ``cu`` (int32 [seqs + 1], the rows of each
sequence in q, k, v; None: one row a sequence).  A sequence's n rows stand at its last n tokens.
They live on the GPU; values out of range are caught there and reported by ``check``.

Nothing here is differentiable: results carry no gradient, also where inputs require one.

    cache = kv4.KV4Cache(num_pages=4096, page_size=64, kv_heads=8, head_dim=128)
    cache.append(k, v, table, lens, cu)
    out, lse = cache.attend(q, table, lens, cu, max_q=longest, window=4096, sinks=4)
    cache.weigh(q, lse, table, lens, cu, max_q=longest, window=4096, sinks=4)
    lens, kept = cache.evict(table, lens, new_table, budget=2048, sinks=4, recent=256)
"""
from __future__ import annotations

import ctypes

from . import E_DEVICE, SplitZipError, _check, lib

BAD_PAGE, BAD_LENGTH, BAD_OFFSETS = 1, 2, 4     # bits of the status word
_BIG = (1 << 31) - 1
BLOCK = 32                                      # channels that share a scale


class splitzip_kv4_cache(ctypes.Structure):
    """Mirror of ``splitzip_kv4_cache`` in include/splitzip_kv4.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "status")] + [
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("device", ctypes.c_int32)]


class splitzip_kv4_batch(ctypes.Structure):
    """Mirror of ``splitzip_kv4_batch``."""
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("total", ctypes.c_int64), ("table_width", ctypes.c_int32),
                ("n_seqs", ctypes.c_int32), ("max_q", ctypes.c_int32), ("max_len", ctypes.c_int32)]


class splitzip_kv4_queries(ctypes.Structure):
    """Mirror of ``splitzip_kv4_queries``."""
    _fields_ = [("q", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("q_heads", ctypes.c_int32), ("dtype", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


_kv4_lib = None


def _lib():
    global _kv4_lib
    if _kv4_lib is None:
        L = lib()
        vp, i64, i32, P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER
        c, b, q = P(splitzip_kv4_cache), P(splitzip_kv4_batch), P(splitzip_kv4_queries)
        L.splitzip_kv4_append.argtypes = [c, b, vp, i64, i64, vp, i64, i64, i32, vp]
        L.splitzip_kv4_read.argtypes = [c, b, vp, vp, i32, vp]
        L.splitzip_kv4_attend_workspace.argtypes = [c, b, q, P(ctypes.c_uint64)]
        L.splitzip_kv4_attend.argtypes = [c, b, q, vp, vp, vp, ctypes.c_uint64, vp]
        L.splitzip_kv4_weigh.argtypes = [c, b, q, vp, vp]
        L.splitzip_kv4_evict.argtypes = [c, b, vp, i64, i32, i32, i32, i32, vp, vp, vp]
        for f in ("append", "read", "attend_workspace", "attend", "weigh", "evict"):
            getattr(L, "splitzip_kv4_" + f).restype = i32
        _kv4_lib = L
    return _kv4_lib


def _dtypes():
    import torch
    return {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _shapes(num_pages: int, page_size: int, kv_heads: int, head_dim: int) -> dict:
    p, h, s, d = num_pages, kv_heads, page_size, head_dim
    return {"k_codes": (p, h, s, d // 2), "k_scales": (p, h, s, d // 32), "v_codes": (p, h, s // 4, 16, 4, d // 32),
            "v_scales": (p, h, d // 32, s), "weights": (p, h, s)}


class KV4Cache:
    """Pages of keys and values in 4 bits, on one GPU.

    ``page_size`` is a power of two in [16, 1024], ``head_dim`` 64, 128 or 256.  The buffers
    (``k_codes``, ``k_scales``, ``v_codes``, ``v_scales``, ``weights``) are torch tensors laid out as
    include/splitzip_kv4.h says; ``page_bytes`` is what one page takes."""

    def __init__(self, num_pages: int, page_size: int = 64, kv_heads: int = 8, head_dim: int = 128, device="cuda"):
        import torch
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if not (16 <= page_size <= 1024 and page_size & (page_size - 1) == 0):
            raise ValueError("page_size must be a power of two in [16, 1024]")
        if num_pages < 1 or kv_heads < 1:
            raise ValueError("num_pages and kv_heads must be at least 1")
        if not torch.cuda.is_available():
            raise SplitZipError(E_DEVICE, "no GPU: the 4-bit cache lives only on the GPU")
        shapes = _shapes(num_pages, page_size, kv_heads, head_dim)
        self._bind(**{n: torch.zeros(s, dtype=torch.float32 if n == "weights" else torch.uint8, device=device)
                      for n, s in shapes.items()})

    @classmethod
    def from_tensors(cls, k_codes, k_scales, v_codes, v_scales, weights) -> "KV4Cache":
        """A cache over buffers that the caller owns, in the layout of include/splitzip_kv4.h."""
        c = cls.__new__(cls)
        c._bind(k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, weights=weights)
        return c

    def _bind(self, **buffers):
        import torch
        k = buffers["k_codes"]
        if k.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, page, half = k.shape
        if half not in (32, 64, 128):
            raise ValueError("head_dim must be 64, 128 or 256")
        if not (16 <= page <= 1024 and page & (page - 1) == 0):
            raise ValueError("page_size must be a power of two in [16, 1024]")
        if not k.is_cuda:
            raise ValueError("the cache's buffers must be on the GPU")
        for n, shape in _shapes(pages, page, heads, 2 * half).items():
            t = buffers[n]
            if tuple(t.shape) != shape or not t.is_contiguous() or t.device != k.device or \
                    t.dtype != (torch.float32 if n == "weights" else torch.uint8):
                raise ValueError(f"{n} must be a contiguous {shape} tensor on {k.device}, of "
                                 f"{'float32' if n == 'weights' else 'uint8'}")
            setattr(self, n, t)
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.device = k.device
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._c = splitzip_kv4_cache(*[getattr(self, n).data_ptr() for n in
                                       ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "status")],
                                     pages, page, heads, 2 * half, k.device.index or 0)
        self._ref = ctypes.byref(self._c)
        self._L = _lib()
        self._dtypes = _dtypes()
        self._index = k.device.index or 0
        self._stream = torch._C._cuda_getCurrentRawStream       # calls of a few microseconds: no lookups in them
        self._i32, self._f32 = torch.int32, torch.float32
        self._empty, self._empty_like = torch.empty, torch.empty_like

    @property
    def page_bytes(self) -> int:
        """Bytes of one page over all heads, weights with it."""
        return self.kv_heads * self.page_size * (self.head_dim + self.head_dim // 16 + 4)

    # -- arguments --------------------------------------------------------------------------
    def _int32(self, t, name: str, shape=None):
        if t.dtype is not self._i32 or t.device != self.device:
            raise ValueError(f"{name} must be int32 on {self.device}, got {t.dtype} on {t.device}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name} must be contiguous along its last dimension")
        return t.data_ptr()

    def _batch(self, table, lens, cu, total: int, max_q, max_len) -> splitzip_kv4_batch:
        if table.dim() != 2:
            raise ValueError("table must be [seqs, pages]")
        n, width = table.shape
        if max_len is None:
            max_len = width * self.page_size
        b = splitzip_kv4_batch(self._int32(table, "table"), self._int32(lens, "lens", (n,)), None,
                               table.stride(0), total, width, n, 1, max_len if max_len < _BIG else _BIG)
        if cu is not None:
            b.cu_seqlens = self._int32(cu, "cu", (n + 1,))
            b.max_q = 0 if max_q is None else max_q if max_q < _BIG else _BIG
        elif total != n:
            raise ValueError(f"without cu there is one row a sequence: {total} rows, {n} sequences")
        return b

    def _rows(self, t, name: str, heads=None, types=3):
        """Type number of a [rows, heads, head_dim] tensor whose channels are adjacent."""
        code = self._dtypes.get(t.dtype, types)
        if code >= types:
            raise TypeError(f"{name} must be {', '.join(str(d) for d, c in self._dtypes.items() if c < types)}, got {t.dtype}")
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.head_dim or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be [rows, {heads or 'heads'}, {self.head_dim}], got {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache is on {self.device}")
        if t.stride(2) != 1:
            raise ValueError(f"{name}'s channels must be adjacent")
        return code

    def _queries(self, q, scale, window, sinks) -> splitzip_kv4_queries:
        code = self._rows(q, "q", types=2)
        if window is not None and window < 1:
            raise ValueError("window must be at least 1 (None: no window)")
        if sinks < 0:
            raise ValueError("sinks must not be negative")
        stride = q.stride()
        return splitzip_kv4_queries(q.data_ptr(), stride[0], stride[1], q.shape[1], code, min(window or 0, _BIG),
                                    sinks if sinks < _BIG else _BIG, self.head_dim ** -0.5 if scale is None else scale)

    def _contiguous_like(self, t):
        """An uninitialized contiguous tensor of t's shape and type."""
        return self._empty_like(t) if t.is_contiguous() else self._empty(*t.shape, dtype=t.dtype, device=self.device)

    # -- operators --------------------------------------------------------------------------
    def append(self, k, v, table, lens, cu=None):
        """Quantizes k and v [rows, kv_heads, head_dim] (bf16, fp16 or fp32, any strides over rows and
        heads) into the sequences' last tokens; those tokens' weights become 0."""
        code = self._rows(k, "k", self.kv_heads)
        if self._rows(v, "v", self.kv_heads) != code or v.shape != k.shape:
            raise ValueError("k and v must have the same shape and type")
        b = self._batch(table, lens, cu, k.shape[0], None, None)
        sk, sv = k.stride(), v.stride()
        _check(self._L.splitzip_kv4_append(self._ref, ctypes.byref(b), k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0],
                                           sv[1], code, self._stream(self._index)))

    def read(self, table, lens, cu=None, total=None, dtype=None):
        """k and v [total, kv_heads, head_dim] as the cache holds them at the sequences' last tokens.
        ``total``: rows, cu[-1] (without cu: one a sequence).  Rows at no token read as NaN."""
        if dtype is None:
            import torch
            dtype = torch.bfloat16
        if dtype not in self._dtypes:
            raise TypeError(f"dtype must be bf16, fp16 or fp32, got {dtype}")
        if total is None:
            if cu is not None:
                raise ValueError("total (the rows, cu[-1]) must be given with cu")
            total = table.shape[0]
        b = self._batch(table, lens, cu, total, None, None)
        k = self._empty(total, self.kv_heads, self.head_dim, dtype=dtype, device=self.device)
        v = self._empty_like(k)
        _check(self._L.splitzip_kv4_read(self._ref, ctypes.byref(b), k.data_ptr(), v.data_ptr(), self._dtypes[dtype],
                                         self._stream(self._index)))
        return k, v

    def attend(self, q, table, lens, cu=None, max_q=None, max_len=None, scale=None, window=None, sinks=0):
        """Attention of q [rows, q_heads, head_dim] (bf16 or fp16) over the cache -> (out, lse): out as q,
        lse fp32 [rows, q_heads].  Query i of a sequence stands at token p = len - n + i and sees
        tokens j <= p with j > p - window (None: all) or j < sinks.  A query that sees nothing gets
        out = 0, lse = -inf.  ``scale``: default head_dim ** -0.5.  ``max_q`` and ``max_len`` (most
        queries and tokens of a sequence, from the host) only choose the launch and its workspace."""
        qs = self._queries(q, scale, window, sinks)
        rows, heads, _ = q.shape
        b = self._batch(table, lens, cu, rows, max_q, max_len)
        b_ref, q_ref, need = ctypes.byref(b), ctypes.byref(qs), ctypes.c_uint64()
        _check(self._L.splitzip_kv4_attend_workspace(self._ref, b_ref, q_ref, ctypes.byref(need)))
        out = self._contiguous_like(q)
        lse = self._empty(rows, heads, dtype=self._f32, device=self.device)
        size = need.value
        work = self._empty(size // 4, dtype=self._f32, device=self.device) if size else None
        _check(self._L.splitzip_kv4_attend(self._ref, b_ref, q_ref, out.data_ptr(), lse.data_ptr(),
                                           work.data_ptr() if size else None, size, self._stream(self._index)))
        return out, lse

    def weigh(self, q, lse, table, lens, cu=None, max_q=None, max_len=None, scale=None, window=None, sinks=0):
        """Adds to ``weights`` the attention that every token and KV head got from q: exp(scale q.k - lse)
        over the queries that see it and the heads of its group.  ``lse`` is what ``attend`` gave
        for these queries and masks.  Pages that sequences share get the sum over all of them."""
        qs = self._queries(q, scale, window, sinks)
        if lse.dtype is not self._f32 or tuple(lse.shape) != tuple(q.shape[:2]) or not lse.is_contiguous() or \
                lse.device != self.device:
            raise ValueError(f"lse must be a contiguous float32 {tuple(q.shape[:2])} tensor on {self.device}")
        b = self._batch(table, lens, cu, q.shape[0], max_q, max_len)
        _check(self._L.splitzip_kv4_weigh(self._ref, ctypes.byref(b), ctypes.byref(qs), lse.data_ptr(), self._stream(self._index)))

    def evict(self, table, lens, out_table, budget: int, sinks: int = 0, recent: int = 0, max_len=None):
        """Cuts every sequence to ``budget`` tokens a KV head: its first ``sinks``, its last ``recent`` and
        the tokens of the largest weights between (the lowest first among equals).  They move, in
        token order, to the pages of ``out_table`` (none of which may be in ``table``)
        -> (out_lens int32 [seqs], kept int32 [seqs, kv_heads, budget], -1 behind the last).  ``max_len``
        (most tokens of a sequence, from the host) only chooses the launch."""
        if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
            raise ValueError("budget must be at least 1 and hold sinks and recent")
        if budget > _BIG - 65536:
            raise ValueError("budget must be below 2^31 - 65536")
        b = self._batch(table, lens, None, table.shape[0], None, max_len)
        if out_table.dim() != 2 or out_table.shape[0] != table.shape[0]:
            raise ValueError("out_table must be [seqs, pages]")
        out_lens = self._empty(table.shape[0], dtype=self._i32, device=self.device)
        kept = self._empty(table.shape[0], self.kv_heads, budget, dtype=self._i32, device=self.device)
        _check(self._L.splitzip_kv4_evict(self._ref, ctypes.byref(b), self._int32(out_table, "out_table"),
                                          out_table.stride(0), out_table.shape[1], budget, sinks, recent,
                                          out_lens.data_ptr(), kept.data_ptr(), self._stream(self._index)))
        return out_lens, kept

    def check(self) -> None:
        """Waits for the GPU, all its streams, and raises if a call since the last check met a page number, a
        length or row offsets out of range."""
        import torch
        torch.cuda.synchronize(self.device)
        bits = int(self.status.item())
        if bits:
            self.status.bitwise_and_(~bits)                     # a bit set meanwhile stays for the next check
            what = [t for b, t in ((BAD_PAGE, "a page number outside the cache"),
                                   (BAD_LENGTH, "a length outside its table"),
                                   (BAD_OFFSETS, "row offsets that decrease or leave the rows")) if bits & b]
            raise ValueError("4-bit cache: " + ", ".join(what))
