"""ctypes binding of the paged key-value cache of libhcr.so (C ABI in include/hcr_paged.h).

A decode window's path behind the attn_q projection (``hcr.matvec_bf16``): ``PagedCache.append`` normalises and
rotates the heads of the new tokens and writes their keys and values into pages, ``attend`` attends over the pages,
and at long contexts ``block_scores``, ``block_topk`` and ``attend_blocks`` attend over the pages of the highest
scores alone.  Argument marshalling only, as in ``hcr.py``: every step runs in the library's kernels, on torch's
current stream of the cache's device or on ``stream`` (a raw hipStream_t).  There is no fallback.

Outputs and scratch made here are made on the stream of the call; with another ``stream`` than torch's current one,
outputs are noted on that one too (``Tensor.record_stream``), so that the caller takes them there, once it has waited
for ``stream``, as any tensor of its own.  The inputs' memory is the caller's: a tensor that may be freed before the
kernels have run is recorded on ``stream``, as for any call of torch's.

A decode step (``y``: the projections' output, [tokens][heads + 2 kv_heads][head_dim])::

    from bf16_hyper_connection_amd.paged import Batch, PagedCache
    cache = PagedCache.allocate(n_pages=4096, kv_heads=8, head_dim=128, page=64)
    batch = Batch(q_start, ctx_len, block_table, max_tokens=4, max_ctx=32768)   # int32 device tensors, host bounds
    q = cache.append(batch, y[:, :32], y[:, 32:40], y[:, 40:], q_norm=wq, k_norm=wk, rope=angles)
    out = cache.attend(batch, q)                                                # or, over the best 32 pages a token:
    out = cache.attend_blocks(batch, q, cache.block_topk(batch, cache.block_scores(batch, q), 32))
"""

import ctypes

import torch

from bf16_hyper_connection_amd import hcr
from bf16_hyper_connection_amd.hcr import HCR_OK, HCRError

HCR_F32, HCR_BF16 = 0, 1
HCR_ROPE_HALVES, HCR_ROPE_PAIRS = 0, 1
_TYPES = {torch.float32: HCR_F32, torch.bfloat16: HCR_BF16}

_vp, _ip, _sz, _ll, _fl, _db = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float,
                                     ctypes.c_double)


class hcr_batch(ctypes.Structure):
    _fields_ = [("n_seqs", _ip), ("n_tokens", _ip), ("max_tokens", _ip), ("max_ctx", _ip), ("table_stride", _ip),
                ("q_start", _vp), ("ctx_len", _vp), ("block_table", _vp)]


class hcr_rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _ll), ("head_stride", _ll)]


_lib = None


def lib():
    """The loaded libhcr.so with the paged cache's entry points (raises if it has not been built)."""
    global _lib
    if _lib is None:
        L = hcr.lib()
        pb, pr = ctypes.POINTER(hcr_batch), ctypes.POINTER(hcr_rows)
        L.hcr_cache_create.restype = _ip
        L.hcr_cache_create.argtypes = [_vp, _vp, _vp, _ip, _ip, _ip, _ip, ctypes.POINTER(_vp)]
        L.hcr_cache_destroy.restype = None
        L.hcr_cache_destroy.argtypes = [_vp]
        L.hcr_cache_pages_bytes.restype = _sz
        L.hcr_cache_pages_bytes.argtypes = [_ip, _ip, _ip, _ip]
        L.hcr_cache_append.restype = _ip
        L.hcr_cache_append.argtypes = [_vp, pb, _ip, _ip, pr, pr, pr, _vp, _vp, _fl, _vp, _ip, _ip, _ip, _vp, _vp]
        L.hcr_attn_scratch_bytes.restype = _sz
        L.hcr_attn_scratch_bytes.argtypes = [_vp, pb, _ip, _ip]
        L.hcr_attn.restype = _ip
        L.hcr_attn.argtypes = [_vp, pb, _ip, _db, _vp, _ip, _vp, _vp, _sz, _vp]
        L.hcr_attn_blocks.restype = _ip
        L.hcr_attn_blocks.argtypes = [_vp, pb, _ip, _db, _vp, _vp, _ip, _ip, _vp, _vp, _sz, _vp]
        L.hcr_block_scores.restype = _ip
        L.hcr_block_scores.argtypes = [_vp, pb, _ip, _vp, _vp, _ip, _vp]
        L.hcr_block_topk.restype = _ip
        L.hcr_block_topk.argtypes = [_vp, pb, _vp, _ip, _ip, _ip, _ip, _vp, _vp]
        _lib = L
    return _lib


def _check(rc, what):
    if rc != HCR_OK:
        raise HCRError(rc, what)


class Batch:
    """The sequences of one call.

    ``q_start`` [n_seqs + 1], ``ctx_len`` [n_seqs] and ``block_table`` [n_seqs][entries] are contiguous int32
    device tensors that the kernels read when they run (a captured graph reads what they hold at its replay);
    ``max_tokens`` and ``max_ctx`` are host bounds of the new tokens and of the length of any sequence.  Rows
    of q, k, v and outputs are numbered by ``q_start``; sequence b's last new token sits at ctx_len[b] - 1.
    Tensors and bounds are fixed (their contents are not): for others make another batch.
    """

    def __init__(self, q_start, ctx_len, block_table, max_tokens, max_ctx):
        for name, t, dim in (("q_start", q_start, 1), ("ctx_len", ctx_len, 1), ("block_table", block_table, 2)):
            if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name}: a contiguous {dim}-D int32 device tensor")
        n = ctx_len.shape[0]
        if q_start.shape[0] != n + 1 or block_table.shape[0] != n:
            raise ValueError(f"q_start [{n + 1}] and block_table [{n}][entries] for ctx_len [{n}]")
        if q_start.device != ctx_len.device or block_table.device != ctx_len.device:
            raise ValueError("q_start, ctx_len and block_table on one device")
        if not 0 <= max_tokens < 1 << 31 or not 0 <= max_ctx < 1 << 31:  # ctypes would cut them to 32 bits
            raise ValueError("max_tokens and max_ctx: not negative, under 2^31")
        self.q_start, self.ctx_len, self.block_table = q_start, ctx_len, block_table
        self.device, self.n_seqs = ctx_len.device, n
        self.max_tokens, self.max_ctx = int(max_tokens), int(max_ctx)
        self._by_rows = {}

    def __setattr__(self, name, value):
        if "_by_rows" in self.__dict__:
            raise AttributeError(f"{name}: a batch's tensors and bounds are fixed")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{name}: a batch's tensors and bounds are fixed")

    def __reduce__(self):  # a copy keeps structs of its own tensors
        return type(self), (self.q_start, self.ctx_len, self.block_table, self.max_tokens, self.max_ctx)

    def _of(self, n_tokens):
        """The C struct for calls of n_tokens rows (kept: a decode loop calls with the same number again)."""
        s = self._by_rows.get(n_tokens)
        if s is None:
            s = hcr_batch(self.n_seqs, n_tokens, self.max_tokens, self.max_ctx, self.block_table.shape[1],
                          self.q_start.data_ptr(), self.ctx_len.data_ptr(), self.block_table.data_ptr())
            self._by_rows[n_tokens] = s
        return s


class PagedCache:
    """One layer's cache: pages that the caller owns, bound to a handle.

    ``k_pages`` BF16 [n_pages][kv_heads][head_dim / 8][page][8], ``v_pages`` BF16
    [n_pages][kv_heads][page / 8][head_dim][8], ``k_means`` BF16 [n_pages][kv_heads][head_dim] or None (no block
    scores).  head_dim is 64, 128 or 256, page 32, 64, 128 or 256.  The pages are fixed (their contents are not): for
    others make another cache.
    """

    def __init__(self, k_pages, v_pages, k_means=None):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("k_means", k_means)):
            if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda):
                raise ValueError(f"{name}: a contiguous bfloat16 device tensor")
        if k_pages.dim() != 5 or k_pages.shape[4] != 8:
            raise ValueError("k_pages: [n_pages][kv_heads][head_dim / 8][page][8]")
        n, heads, chunks, page, _ = k_pages.shape
        if tuple(v_pages.shape) != (n, heads, page // 8, chunks * 8, 8):
            raise ValueError(f"v_pages: expected {(n, heads, page // 8, chunks * 8, 8)}")
        if k_means is not None and tuple(k_means.shape) != (n, heads, chunks * 8):
            raise ValueError(f"k_means: expected {(n, heads, chunks * 8)}")
        if v_pages.device != k_pages.device or (k_means is not None and k_means.device != k_pages.device):
            raise ValueError("pages and means on one device")
        self.k_pages, self.v_pages, self.k_means = k_pages, v_pages, k_means
        self.n_pages, self.kv_heads, self.page, self.head_dim = n, heads, page, chunks * 8
        self.device = k_pages.device
        self._L, self.handle = lib(), None
        h = _vp()
        _check(self._L.hcr_cache_create(k_pages.data_ptr(), v_pages.data_ptr(),
                                        None if k_means is None else k_means.data_ptr(), n, heads, self.head_dim,
                                        page, ctypes.byref(h)), "hcr_cache_create")
        self.handle = h.value
        self._vp, self._destroy_fn = _vp, self._L.hcr_cache_destroy

    @classmethod
    def allocate(cls, n_pages, kv_heads, head_dim, page=64, device="cuda", means=True):
        """A cache of newly allocated (uninitialised) pages."""
        def make(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=device)
        return cls(make(n_pages, kv_heads, head_dim // 8, page, 8), make(n_pages, kv_heads, page // 8, head_dim, 8),
                   make(n_pages, kv_heads, head_dim) if means else None)

    def __del__(self):
        # references bound at creation: at interpreter exit this module's globals may already be gone
        h, fn, vp = getattr(self, "handle", None), getattr(self, "_destroy_fn", None), getattr(self, "_vp", None)
        if h and fn is not None and vp is not None:
            self.__dict__["handle"] = None
            fn(vp(h))

    # what the handle was made of, and what it is destroyed with
    _FIXED = frozenset(("k_pages", "v_pages", "k_means", "n_pages", "kv_heads", "page", "head_dim", "device", "handle",
                        "_L", "_vp", "_destroy_fn"))

    def __setattr__(self, name, value):
        if name in self._FIXED and "_destroy_fn" in self.__dict__:
            raise AttributeError(f"{name}: a cache's pages and geometry are fixed")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError(f"{name}: a cache's pages and geometry are fixed")
        super().__delattr__(name)

    def __reduce__(self):  # a copy makes a handle of its own
        return type(self), (self.k_pages, self.v_pages, self.k_means)

    def _call(self, fn, batch, stream, *args):
        """The entry point on the cache's device, its stream last."""
        if batch.device != self.device:
            raise ValueError(f"batch: on {self.device}")
        index = self.device.index
        st = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream
        if torch._C._cuda_getDevice() == index:
            rc = fn(self.handle, *args, st)
        else:
            with torch.cuda.device(self.device):
                rc = fn(self.handle, *args, st)
        if rc != HCR_OK:
            raise HCRError(rc, fn.__name__)

    def _new(self, stream, shape, dtype, fill=None, returned=True):
        """A new tensor of a call, filled, on the stream that the call runs on: behind that stream's earlier steps and
        ahead of the call's kernels.  Torch's current stream, on which the caller takes what is returned, is noted, so
        that the memory is not used again before that stream is done with it."""
        own = None
        if stream is not None:
            raw = getattr(stream, "value", stream) or 0  # as a number, or as ctypes holds it
            if raw != torch._C._cuda_getCurrentRawStream(self.device.index):
                own = torch.cuda.ExternalStream(raw, device=self.device) if raw else \
                    torch.cuda.default_stream(self.device)
        if own is None:
            t = torch.empty(shape, dtype=dtype, device=self.device)
            return t if fill is None else t.fill_(fill)
        with torch.cuda.stream(own):
            t = torch.empty(shape, dtype=dtype, device=self.device)
            if fill is not None:
                t.fill_(fill)
        if returned:
            t.record_stream(torch.cuda.current_stream(self.device))
        return t

    # The checks below run at every call, ahead of kernels of a few microseconds: each reads a property once.

    def _heads_of(self, q):
        """(rows, heads) of q, BF16 [n_tokens][heads][head_dim]."""
        shape = q.shape
        if q.dtype is not torch.bfloat16 or len(shape) != 3 or shape[2] != self.head_dim or \
                not q.is_contiguous() or q.device != self.device:
            raise ValueError(f"q: contiguous bfloat16 [n_tokens][heads][{self.head_dim}] on {self.device}")
        return shape[0], shape[1]

    def _given(self, name, t, shape, dtype):
        if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {self.device}")

    def _rows(self, name, x, shape, dtype):
        if x.shape != shape or x.dtype is not dtype or x.device != self.device:
            raise ValueError(f"{name}: expected {dtype} {shape} on {self.device}")
        by_token, by_head, by_value = x.stride()
        if by_value != 1:
            raise ValueError(f"{name}: the values of a head side by side")
        return hcr_rows(x.data_ptr(), by_token if shape[0] > 1 else 0, by_head if shape[1] > 1 else 0)

    def append(self, batch, q, k, v, q_norm=None, k_norm=None, eps=1e-6, rope=None, interleaved=False, q_out=None,
               stream=None):
        """Norm and rotate the heads of the new tokens, write k and v into their pages; returns q in BF16.

        ``q`` [n_tokens][heads][head_dim], ``k`` and ``v`` [n_tokens][kv_heads][head_dim]: float32 or bfloat16,
        all of one type, views of one projection's output as well (strides of whole 16 bytes).  ``q_norm`` and
        ``k_norm`` float32 [head_dim] (None: no norm); ``rope`` float32 [positions][rope_dim], cos then sin of
        rope_dim / 2 angles (None: no rotation); ``interleaved`` rotates pairs (2j, 2j + 1) instead of
        (j, j + rope_dim / 2).  Pages that the window completes get their mean key.
        """
        dtype, D = q.dtype, self.head_dim
        if dtype not in _TYPES or q.dim() != 3:
            raise ValueError("q: float32 or bfloat16 [n_tokens][heads][head_dim]")
        n, heads, _ = q.shape
        rq = self._rows("q", q, (n, heads, D), dtype)
        rk = self._rows("k", k, (n, self.kv_heads, D), dtype)
        rv = self._rows("v", v, (n, self.kv_heads, D), dtype)
        if q_norm is not None:
            self._given("q_norm", q_norm, (D,), torch.float32)
        if k_norm is not None:
            self._given("k_norm", k_norm, (D,), torch.float32)
        rope_rows = rope_dim = 0
        if rope is not None:
            if rope.dim() != 2:
                raise ValueError("rope: float32 [positions][rope_dim]")
            rope_rows, rope_dim = rope.shape
            self._given("rope", rope, (rope_rows, rope_dim), torch.float32)
        if q_out is None:
            q_out = self._new(stream, (n, heads, D), torch.bfloat16)
        else:
            self._given("q_out", q_out, (n, heads, D), torch.bfloat16)
        self._call(self._L.hcr_cache_append, batch, stream, batch._of(n), heads, _TYPES[dtype], rq, rk, rv,
                   None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(), eps,
                   rope.data_ptr() if rope_dim else None, rope_rows, rope_dim,
                   HCR_ROPE_PAIRS if interleaved else HCR_ROPE_HALVES, q_out.data_ptr())
        return q_out

    def _attend(self, fn, batch, q, sel, scale, out, out_dtype, scratch, stream):
        n, heads = self._heads_of(q)
        if out is None:
            out = self._new(stream, (n, heads, self.head_dim), out_dtype)
        else:
            self._given("out", out, (n, heads, self.head_dim), out.dtype)
        if out.dtype not in _TYPES:
            raise ValueError("out: float32 or bfloat16")
        n_sel = 0 if sel is None else sel.shape[2]
        c_batch = batch._of(n)
        need = self._L.hcr_attn_scratch_bytes(self.handle, c_batch, heads, n_sel)
        if scratch is None:
            scratch = self._new(stream, need, torch.uint8, returned=False) if need else None
        elif not scratch.is_cuda or scratch.device != self.device or not scratch.is_contiguous():
            raise ValueError(f"scratch: a contiguous tensor on {self.device}")
        room = 0 if scratch is None else scratch.numel() * scratch.element_size()
        listed = () if sel is None else (sel.data_ptr(), n_sel)
        self._call(fn, batch, stream, c_batch, heads, self.head_dim ** -0.5 if scale is None else scale,
                   q.data_ptr(), *listed, _TYPES[out.dtype], out.data_ptr(),
                   None if scratch is None else scratch.data_ptr(), room)
        return out

    def attend(self, batch, q, scale=None, out=None, out_dtype=torch.float32, scratch=None, stream=None):
        """Attention of the window over its sequences' pages (the window's own keys are in them already).

        ``q`` BF16 [n_tokens][heads][head_dim] as ``append`` returns it, ``scale`` head_dim ** -0.5 by default;
        returns float32 (``out_dtype``, or ``out``'s) [n_tokens][heads][head_dim].  ``scratch``: at least
        ``scratch_bytes`` of device memory; calls that share one are ordered on one stream.
        """
        return self._attend(self._L.hcr_attn, batch, q, None, scale, out, out_dtype, scratch, stream)

    def attend_blocks(self, batch, q, sel, scale=None, out=None, out_dtype=torch.float32, scratch=None, stream=None):
        """``attend`` over the pages listed in ``sel``, int32 [n_tokens][kv_heads][n_sel] (-1: none)."""
        n = q.shape[0]
        if sel.dim() != 3:
            raise ValueError(f"sel: int32 [{n}][{self.kv_heads}][n_sel]")
        self._given("sel", sel, (n, self.kv_heads, sel.shape[2]), torch.int32)
        return self._attend(self._L.hcr_attn_blocks, batch, q, sel, scale, out, out_dtype, scratch, stream)

    def scratch_bytes(self, batch, n_tokens, heads, n_sel=0):
        """Bytes that ``attend`` (n_sel 0) or ``attend_blocks`` needs for this batch."""
        return int(self._L.hcr_attn_scratch_bytes(self.handle, batch._of(n_tokens), heads, n_sel))

    def block_scores(self, batch, q, scores=None, stream=None):
        """Scores of the complete pages before each token's own: float32 [n_tokens][kv_heads][pages].

        Entries from the token's own page on are left as they were (in a new tensor: -inf).  ``scores`` begins at a
        whole 16 bytes.
        """
        n, heads = self._heads_of(q)
        if scores is None:
            scores = self._new(stream, (n, self.kv_heads, max(-(-batch.max_ctx // self.page), 1)), torch.float32,
                               float("-inf"))
        else:
            if scores.dim() != 3:
                raise ValueError(f"scores: float32 [{n}][{self.kv_heads}][pages]")
            self._given("scores", scores, (n, self.kv_heads, scores.shape[2]), torch.float32)
        self._call(self._L.hcr_block_scores, batch, stream, batch._of(n), heads, q.data_ptr(),
                   scores.data_ptr(), scores.shape[2])
        return scores

    def block_topk(self, batch, scores, n_sel, n_first=1, n_last=2, sel=None, stream=None):
        """The pages each token attends to, int32 [n_tokens][kv_heads][n_sel]: ascending, -1 behind.

        The first ``n_first``, the last ``n_last`` (the token's own among them) and the highest scores between;
        level scores: the lowest index.
        """
        if scores.dim() != 3:
            raise ValueError(f"scores: float32 [n_tokens][{self.kv_heads}][pages]")
        if not -1 << 31 <= min(n_sel, n_first, n_last) <= max(n_sel, n_first, n_last) < 1 << 31:  # as a batch's bounds
            raise ValueError("n_sel, n_first and n_last: whole numbers of 32 bits")
        n = scores.shape[0]
        self._given("scores", scores, (n, self.kv_heads, scores.shape[2]), torch.float32)
        if sel is None:
            sel = self._new(stream, (n, self.kv_heads, max(n_sel, 0)), torch.int32)
        else:
            self._given("sel", sel, (n, self.kv_heads, n_sel), torch.int32)
        self._call(self._L.hcr_block_topk, batch, stream, batch._of(n), scores.data_ptr(), scores.shape[2],
                   n_sel, n_first, n_last, sel.data_ptr())
        return sel
