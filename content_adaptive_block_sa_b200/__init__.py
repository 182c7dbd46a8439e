"""Content-adaptive block-sparse attention on B200 (sm_100a).

A thin binding over the C ABI of ``libsa.so`` (include/sa.h). The functions
named ``sa_*`` have the C entry points' names and only marshal arguments
(tensor pointers, strides and the current CUDA stream); every step of the
computation runs in the library's CUDA kernels. The helpers below them
(``BlockLists``, ``forward``, ``backward``, ``gist_decode``, ``PagedCache``,
``paged_append``, ``paged_decode``, ``cache_evict``) allocate outputs
and workspaces with PyTorch, which this package uses for device memory and
streams only.
"""
from __future__ import annotations

import ctypes as C
import zlib

import numpy as np
import torch

from . import _abi
from ._abi import *  # noqa: F401,F403  (enums and structs)

_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        _lib = _abi.load()
    return _lib


class SAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().sa_status_string(status).decode()}")


def _check(status: int, where: str) -> None:
    if status != _abi.SA_OK:
        raise SAError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def version() -> str:
    return lib().sa_version().decode()


# ------------------------------------------------------------------ a1 flags
def block_compressed_sizes(x: bytes, b: int) -> np.ndarray:
    """Level-1 zlib size of every b-byte block (host input preparation)."""
    if len(x) % b:
        raise ValueError("byte length must be a multiple of the block size")
    return np.array([len(zlib.compress(x[i:i + b], 1)) for i in range(0, len(x), b)],
                    dtype=np.uint32)


def sa_literal_flags_from_sizes(sizes: np.ndarray) -> np.ndarray:
    sizes = np.ascontiguousarray(sizes, dtype=np.uint32)
    flags = np.zeros(len(sizes), np.uint8)
    _check(lib().sa_literal_flags_from_sizes(
        sizes.ctypes.data_as(C.POINTER(C.c_uint32)), len(sizes),
        flags.ctypes.data_as(C.POINTER(C.c_uint8))), "sa_literal_flags_from_sizes")
    return flags


def literal_flags(x: bytes, b: int) -> np.ndarray:
    return sa_literal_flags_from_sizes(block_compressed_sizes(x, b))


def literal_flags_device(x: torch.Tensor, b: int, stream=None, sizes=None, flags=None):
    """Flags from device bytes x (uint8 [batch, n_bytes]) by the library's
    DEFLATE size estimate (greedy fast-table parse, the smallest of the fixed,
    dynamic and stored block): (sizes uint32 as int32 [batch, B], flags uint8
    [batch, B]), written into `sizes`/`flags` when given."""
    if x.dtype != torch.uint8 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous uint8 [batch, n_bytes] tensor")
    batch, n = x.shape
    B = n // b
    if sizes is None:
        sizes = torch.empty(batch, B, dtype=torch.int32, device=x.device)
    if flags is None:
        flags = torch.empty(batch, B, dtype=torch.uint8, device=x.device)
    for t, dt in ((sizes, torch.int32), (flags, torch.uint8)):
        if t.dtype != dt or t.shape != (batch, B) or not t.is_contiguous() or t.device != x.device:
            raise ValueError("sizes/flags must be contiguous [batch, n_bytes // b] int32/uint8 "
                             "tensors on x's device")
    _check(lib().sa_literal_flags_device(_ptr(x), batch, n, b, _ptr(sizes), _ptr(flags),
                                         _stream(stream)), "sa_literal_flags_device")
    return sizes, flags


# ---------------------------------------------------------------- mask desc
def mask_desc(kind: int, seq_len: int, num_heads: int, batch: int = 1, block_size: int = 0,
              window: int = 0, sinks: int = 0, gist_ratio: int = 0, gist_tail: int = 0,
              head_class=None) -> _abi.sa_mask_desc:
    d = _abi.sa_mask_desc(kind=kind, batch=batch, seq_len=seq_len, block_size=block_size,
                          window=window, num_heads=num_heads, sinks=sinks,
                          gist_ratio=gist_ratio, gist_tail=gist_tail, head_class=None)
    if head_class is not None:
        buf = (C.c_int8 * num_heads)(*[int(c) for c in head_class])
        d._head_class_buf = buf  # keep alive
        d.head_class = C.cast(buf, C.c_void_p)
    return d


def gzip_mask(batch, seq_len, block_size, window, num_heads, head_class=None):
    return mask_desc(_abi.SA_MASK_GZIP, seq_len, num_heads, batch=batch, block_size=block_size,
                     window=window, head_class=head_class)


def gist_mask(seq_len, num_heads, sinks, gist_ratio, window, gist_tail=32, segment=0):
    """Gist layout. segment = 0: interleaved gists and a local window of
    `window` positions; segment = L > 0: the coarse layout, L raw tokens then
    L / gist_ratio gists per segment, full attention inside a segment (window
    ignored)."""
    return mask_desc(_abi.SA_MASK_GIST, seq_len, num_heads, sinks=sinks, gist_ratio=gist_ratio,
                     window=window, gist_tail=gist_tail, block_size=segment)


class BlockLists:
    """Device buffers of sa_block_lists, sized by sa_block_lists_capacity."""

    def __init__(self, desc: _abi.sa_mask_desc, device="cuda"):
        caps = _abi.sa_block_lists_sizes()
        _check(lib().sa_block_lists_capacity(C.byref(desc), C.byref(caps)),
               "sa_block_lists_capacity")
        self.desc = desc
        self.caps = caps
        mk = lambda n, dt: torch.zeros(max(int(n), 1), dtype=dt, device=device) if n else None
        self.row_ptr = mk(caps.row_ptr, torch.int32)
        self.col_idx = mk(caps.nnz, torch.int32)
        self.col_ptr = mk(caps.row_ptr, torch.int32)
        self.row_idx = mk(caps.nnz, torch.int32)
        self.bits = mk(caps.bits, torch.int32)
        self.tile_row_ptr = mk(caps.tile_row_ptr, torch.int32)
        self.tile_col = mk(caps.tile_nnz, torch.int32)
        self.tile_kind = mk(caps.tile_nnz, torch.int8)
        self.tile_col_ptr = mk(caps.tile_row_ptr, torch.int32)
        self.tile_row = mk(caps.tile_nnz, torch.int32)
        self.tile_kind_t = mk(caps.tile_nnz, torch.int8)
        self.perm = mk(caps.perm, torch.int32)
        self.gist_bits = mk(caps.gist_bits, torch.int32)
        self.far_idx = mk(caps.far_idx, torch.int32)
        self.far_ptr = mk(caps.far_ptr, torch.int32)
        self.struct = _abi.sa_block_lists(
            *[_ptr(getattr(self, n)) for n in ("row_ptr", "col_idx", "col_ptr", "row_idx", "bits",
                                                "tile_row_ptr", "tile_col", "tile_kind",
                                                "tile_col_ptr", "tile_row", "tile_kind_t",
                                                "perm", "gist_bits", "far_idx", "far_ptr")],
            int(caps.nnz), int(caps.tile_nnz))


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def sa_build_block_mask(desc, flags, lists: BlockLists, ws: torch.Tensor, stream=None) -> None:
    _check(lib().sa_build_block_mask(C.byref(desc), _ptr(flags), C.byref(lists.struct),
                                     _ptr(ws), ws.numel(), _stream(stream)),
           "sa_build_block_mask")


def build_block_mask(desc, flags=None, device="cuda", stream=None) -> BlockLists:
    """Allocates lists + workspace and runs sa_build_block_mask.

    flags: gzip - uint8 [batch, B] literal flags (host numpy or device tensor);
    gist - None (regular pattern) or uint8 [N] gist flags per logical position."""
    lists = BlockLists(desc, device)
    if flags is not None and not torch.is_tensor(flags):
        flags = torch.from_numpy(np.ascontiguousarray(flags, dtype=np.uint8)).to(device)
    n = C.c_size_t()
    _check(lib().sa_build_block_mask_workspace_size(C.byref(desc), C.byref(n)),
           "sa_build_block_mask_workspace_size")
    ws = _workspace(n.value, device)
    sa_build_block_mask(desc, flags, lists, ws, stream)
    lists._flags = flags
    lists._ws = ws
    return lists


# ---------------------------------------------------------------- attention
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _abi.SA_DTYPE_BF16
    if t.dtype == torch.float32:
        return _abi.SA_DTYPE_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def attn_desc(q, k, v, o, softmax_scale: float = 0.0, impl: int = 0) -> _abi.sa_attn_desc:
    """Descriptor from [Bt, N, H, d] tensors (any strides, last dim contiguous)."""
    Bt, N, Hq, d = q.shape
    st = lambda t: (i64 * 3)(t.stride(0), t.stride(1), t.stride(2))
    for t in (q, k, v, o):
        if t.stride(3) != 1:
            raise ValueError("head_dim must be contiguous")
    return _abi.sa_attn_desc(dtype=_dtype_code(q), batch=Bt, seq_len=N, num_q_heads=Hq,
                             num_kv_heads=k.shape[2], head_dim=d, softmax_scale=softmax_scale,
                             q_strides=st(q), k_strides=st(k), v_strides=st(v), o_strides=st(o),
                             impl=impl)


i64 = C.c_int64


def sa_forward(adesc, mdesc, q, k, v, lists: BlockLists, o, lse, ws, stream=None) -> None:
    _check(lib().sa_forward(C.byref(adesc), C.byref(mdesc), _ptr(q), _ptr(k), _ptr(v),
                            C.byref(lists.struct), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                            _stream(stream)), "sa_forward")


def forward_workspace(adesc, mdesc, device="cuda") -> torch.Tensor:
    n = C.c_size_t()
    _check(lib().sa_forward_workspace_size(C.byref(adesc), C.byref(mdesc), C.byref(n)),
           "sa_forward_workspace_size")
    return _workspace(n.value, device)


def forward(q, k, v, mdesc, lists: BlockLists, softmax_scale: float = 0.0, stream=None,
            impl: int = 0):
    """O [Bt, N, Hq, d] (dtype of q) and LSE fp32 [Bt, Hq, N]."""
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[0], q.shape[2], q.shape[1], dtype=torch.float32, device=q.device)
    ad = attn_desc(q, k, v, o, softmax_scale, impl)
    ws = forward_workspace(ad, mdesc, q.device)
    sa_forward(ad, mdesc, q, k, v, lists, o, lse, ws, stream)
    return o, lse


def sa_backward(adesc, mdesc, q, k, v, o, lse, dout, lists, dq, dk, dv, ws, stream=None) -> None:
    _check(lib().sa_backward(C.byref(adesc), C.byref(mdesc), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                             _ptr(lse), _ptr(dout), C.byref(lists.struct), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)), "sa_backward")


def backward_workspace(adesc, mdesc, device="cuda") -> torch.Tensor:
    n = C.c_size_t()
    _check(lib().sa_backward_workspace_size(C.byref(adesc), C.byref(mdesc), C.byref(n)),
           "sa_backward_workspace_size")
    return _workspace(n.value, device)


def backward(q, k, v, o, lse, dout, mdesc, lists, softmax_scale: float = 0.0, stream=None,
             impl: int = 0):
    """fp32 dQ [Bt, N, Hq, d], dK and dV [Bt, N, Hkv, d]. dout has o's strides."""
    if dout.stride() != o.stride():
        raise ValueError("dout must have the same strides as o")
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    dk = torch.empty(k.shape, dtype=torch.float32, device=q.device)
    dv = torch.empty(v.shape, dtype=torch.float32, device=q.device)
    ad = attn_desc(q, k, v, o, softmax_scale, impl)
    ws = backward_workspace(ad, mdesc, q.device)
    sa_backward(ad, mdesc, q, k, v, o, lse, dout, lists, dq, dk, dv, ws, stream)
    return dq, dk, dv


# ------------------------------------------------------------------- decode
def decode_desc(q, gist_k, k_cache, o, chunk: int, top_k: int, window: int,
                softmax_scale: float = 0.0, select_rule: int = 0,
                top_p: float = 1.0) -> _abi.sa_decode_desc:
    n_seq, Hq, d = q.shape
    _, Hkv, G, _ = gist_k.shape
    L = k_cache.shape[2]
    return _abi.sa_decode_desc(
        n_seq=n_seq, cache_len=L, chunk=chunk, n_gists=G, top_k=top_k, window=window,
        num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d,
        select_rule=select_rule, softmax_scale=softmax_scale, top_p=top_p,
        q_strides=(i64 * 2)(q.stride(0), q.stride(1)),
        gist_strides=(i64 * 3)(gist_k.stride(0), gist_k.stride(1), gist_k.stride(2)),
        cache_strides=(i64 * 3)(k_cache.stride(0), k_cache.stride(1), k_cache.stride(2)),
        o_strides=(i64 * 2)(o.stride(0), o.stride(1)))


def decode_workspace(ddesc, device="cuda") -> torch.Tensor:
    n = C.c_size_t()
    _check(lib().sa_gist_decode_workspace_size(C.byref(ddesc), C.byref(n)),
           "sa_gist_decode_workspace_size")
    return _workspace(n.value, device)


def sa_gist_decode(ddesc, q, gist_k, gist_v, k_cache, v_cache, sel, o, lse, ws, stream=None):
    _check(lib().sa_gist_decode(C.byref(ddesc), _ptr(q), _ptr(gist_k), _ptr(gist_v),
                                _ptr(k_cache), _ptr(v_cache), _ptr(sel), _ptr(o), _ptr(lse),
                                _ptr(ws), ws.numel(), _stream(stream)), "sa_gist_decode")


def gist_decode(q, gist_k, gist_v, k_cache, v_cache, chunk: int, top_k: int, window: int,
                softmax_scale: float = 0.0, stream=None, select_rule: int = 0, top_p: float = 1.0):
    """(sel int32 [n_seq, Hkv, top_k], o bf16 [n_seq, Hq, d], lse fp32 [n_seq, Hq]).
    select_rule: 0 top-k of summed logits, 1 top-k of summed per-head
    probabilities, 2 top-p (at most top_k chunks) of the summed logits, 3 each
    query head's own top-k (sel is then [n_seq, Hq, top_k])."""
    if gist_v.stride() != gist_k.stride() or v_cache.stride() != k_cache.stride():
        raise ValueError("K and V must share strides")
    n_seq, Hq, d = q.shape
    Hkv = gist_k.shape[1]
    o = torch.empty_like(q)
    lse = torch.empty(n_seq, Hq, dtype=torch.float32, device=q.device)
    rows = Hq if select_rule == _abi.SA_SELECT_TOP_K_PER_HEAD else Hkv
    sel = torch.empty(n_seq, rows, max(top_k, 1), dtype=torch.int32, device=q.device)
    dd = decode_desc(q, gist_k, k_cache, o, chunk, top_k, window, softmax_scale, select_rule, top_p)
    ws = decode_workspace(dd, q.device)
    sa_gist_decode(dd, q, gist_k, gist_v, k_cache, v_cache, sel, o, lse, ws, stream)
    gist_decode.last_workspace = ws
    return sel[:, :, :top_k], o, lse


def hier_decode_desc(q, gist2_k, gist_k, k_cache, o, chunk: int, fanout: int, top_k2: int,
                     top_k: int, window: int, softmax_scale: float = 0.0) -> _abi.sa_hier_decode_desc:
    n_seq, Hq, d = q.shape
    _, Hkv, G, _ = gist_k.shape
    return _abi.sa_hier_decode_desc(
        n_seq=n_seq, cache_len=k_cache.shape[2], chunk=chunk, n_gists=G, fanout=fanout,
        top_k2=top_k2, top_k=top_k, window=window, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d,
        softmax_scale=softmax_scale, q_strides=(i64 * 2)(q.stride(0), q.stride(1)),
        gist_strides=(i64 * 3)(*gist_k.stride()[:3]), gist2_strides=(i64 * 3)(*gist2_k.stride()[:3]),
        cache_strides=(i64 * 3)(*k_cache.stride()[:3]), o_strides=(i64 * 2)(o.stride(0), o.stride(1)))


def hier_decode_workspace(hdesc, device="cuda") -> torch.Tensor:
    n = C.c_size_t()
    _check(lib().sa_gist_hier_decode_workspace_size(C.byref(hdesc), C.byref(n)),
           "sa_gist_hier_decode_workspace_size")
    return _workspace(n.value, device)


def sa_gist_hier_decode(hdesc, q, gist2_k, gist2_v, gist_k, gist_v, k_cache, v_cache, sel2, sel1,
                        o, lse, ws, stream=None):
    _check(lib().sa_gist_hier_decode(C.byref(hdesc), _ptr(q), _ptr(gist2_k), _ptr(gist2_v),
                                     _ptr(gist_k), _ptr(gist_v), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(sel2), _ptr(sel1), _ptr(o), _ptr(lse), _ptr(ws),
                                     ws.numel(), _stream(stream)), "sa_gist_hier_decode")


def gist_hier_decode(q, gist2_k, gist2_v, gist_k, gist_v, k_cache, v_cache, chunk: int, fanout: int,
                     top_k2: int, top_k: int, window: int, softmax_scale: float = 0.0, stream=None):
    """Gist-of-gist decode: (sel2 int32 [n_seq, Hkv, top_k2], sel1 int32
    [n_seq, Hkv, top_k], o bf16 [n_seq, Hq, d], lse fp32 [n_seq, Hq])."""
    for a, b in ((gist2_k, gist2_v), (gist_k, gist_v), (k_cache, v_cache)):
        if a.stride() != b.stride():
            raise ValueError("K and V must share strides")
    n_seq, Hq, d = q.shape
    Hkv = gist_k.shape[1]
    o = torch.empty_like(q)
    lse = torch.empty(n_seq, Hq, dtype=torch.float32, device=q.device)
    sel2 = torch.empty(n_seq, Hkv, max(top_k2, 1), dtype=torch.int32, device=q.device)
    sel1 = torch.empty(n_seq, Hkv, max(top_k, 1), dtype=torch.int32, device=q.device)
    hd = hier_decode_desc(q, gist2_k, gist_k, k_cache, o, chunk, fanout, top_k2, top_k, window,
                          softmax_scale)
    ws = hier_decode_workspace(hd, q.device)
    sa_gist_hier_decode(hd, q, gist2_k, gist2_v, gist_k, gist_v, k_cache, v_cache, sel2, sel1, o, lse,
                        ws, stream)
    gist_hier_decode.last_workspace = ws
    return sel2[:, :, :top_k2], sel1[:, :, :top_k], o, lse


# -------------------------------------------------------------- paged cache
_PAGED_DTYPES = {torch.bfloat16: _abi.SA_DTYPE_BF16, torch.float16: _abi.SA_DTYPE_FP16,
                 torch.float8_e4m3fn: _abi.SA_DTYPE_E4M3}


def _paged_dtype(t: torch.Tensor) -> int:
    if t.dtype not in _PAGED_DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _PAGED_DTYPES[t.dtype]


def _need(cond: bool, message: str) -> None:
    if not cond:
        raise ValueError(message)


class PagedCache:
    """A paged key/value cache over the caller's tensors (sa_paged_cache).

    k, v: pools [n_pages, Hkv, page_size, d] (any strides shared by both, d
    contiguous, rows on 16-byte boundaries; for pools kept as [n_pages,
    page_size, Hkv, d] pass ``pool.transpose(1, 2)``), bf16, fp16 or
    float8_e4m3fn. page_table: int32 [n_seq, max_pages]. seq_lens: int32
    [n_seq], the positions each sequence holds. k_scale, v_scale: fp32 [Hkv]
    beside an 8-bit pool (None: 1). max_len: the longest sequence a call may
    meet (0: what the table has room for); calls over a table made for far
    longer ones cost less with it. The tensors stay the caller's: their
    contents may change between calls, and the object keeps them alive."""

    def __init__(self, k, v, page_table, seq_lens, k_scale=None, v_scale=None, max_len: int = 0):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype
              and k.stride() == v.stride(), "k and v must be 4-D and share shape, dtype and strides")
        _need(k.stride(3) == 1, "head_dim must be contiguous")
        _need(page_table.dtype == torch.int32 and page_table.dim() == 2
              and page_table.stride(1) == 1, "page_table must be int32 [n_seq, max_pages], rows contiguous")
        _need(seq_lens.dtype == torch.int32 and seq_lens.shape == page_table.shape[:1]
              and seq_lens.is_contiguous(), "seq_lens must be contiguous int32 [n_seq]")
        for t in (k_scale, v_scale):
            _need(t is None or (t.dtype == torch.float32 and t.shape == k.shape[1:2]
                                and t.is_contiguous()), "scales must be contiguous fp32 [Hkv]")
        self.tensors = (k, v, page_table, seq_lens, k_scale, v_scale)
        self.k, self.v, self.page_table, self.seq_lens, self.k_scale, self.v_scale = self.tensors
        _on_device(k.device, *self.tensors)
        self.device = k.device
        n_pages, hkv, page_size, d = k.shape
        n_seq, max_pages = page_table.shape
        self.n_seq, self.num_kv_heads, self.head_dim = n_seq, hkv, d
        self.page_size, self.capacity = page_size, max_len or max_pages * page_size
        self.struct = _abi.sa_paged_cache(
            dtype=_paged_dtype(k), n_seq=n_seq, num_kv_heads=hkv, head_dim=d, page_size=page_size,
            n_pages=n_pages, max_pages=max_pages, max_len=max_len, strides=(i64 * 3)(*k.stride()[:3]),
            table_stride=_table_stride(page_table), k=_ptr(k), v=_ptr(v),
            page_table=_ptr(page_table), seq_lens=_ptr(seq_lens), k_scale=_ptr(k_scale),
            v_scale=_ptr(v_scale))
        self.ref = C.byref(self.struct)
        self.index = k.device.index if k.device.type == "cuda" else None


def _table_stride(t: torch.Tensor) -> int:
    """Elements between a page table's rows (of no meaning for a single row)."""
    rows, pages = t.shape
    _need(rows == 1 or t.stride(0) >= pages, "a page table's rows must not overlap (expanded tensors do)")
    return pages if rows == 1 else t.stride(0)


def _on_device(device, *tensors, stream=None) -> None:
    """Checks the tensors of a call; on a stream of its own they are kept from
    being handed out again while the call may still use them."""
    for t in tensors:
        _need(t is None or t.device == device, f"every tensor must be on {device}")
        if t is not None and stream is not None:
            t.record_stream(stream)


def _call_on(cache, stream, name: str, *args) -> None:
    """Calls an entry point on a stream of the cache's device (None: its
    current one), with that device current. A step of a decode loop spends
    its host time here, so nothing is looked up twice."""
    index = cache.index
    if index is None:
        raise ValueError("the tensors must be on a CUDA device")
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(index)
    else:
        _need(stream.device == cache.device, "the stream must belong to the tensors' device")
        s = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if index == torch._C._cuda_getDevice():
        st = fn(cache.ref, *args, s)
    else:
        with torch.cuda.device(index):
            st = fn(cache.ref, *args, s)
    if st:
        raise SAError(st, name)


def _alloc_on(device, stream):
    """Allocations of a call belong to the stream it runs on, so that their
    memory is not handed out again before the kernels have used it."""
    _need(device.type == "cuda", "the tensors must be on a CUDA device")
    return torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream)


def _score_strides(scores):
    if scores is None:
        return (i64 * 2)(0, 0)
    _need(scores.dtype == torch.float32 and scores.dim() == 3 and scores.stride(2) == 1,
          "scores must be fp32 [n_seq, Hkv, positions], positions contiguous")
    return (i64 * 2)(scores.stride(0), scores.stride(1))


def _check_scores(cache, scores, positions: int) -> None:
    _need(scores.dtype == torch.float32 and scores.dim() == 3 and scores.stride(2) == 1
          and tuple(scores.shape[:2]) == (cache.n_seq, cache.num_kv_heads)
          and scores.shape[2] >= positions,
          f"scores must be fp32 [{cache.n_seq}, {cache.num_kv_heads}, >= {positions}]")


def _paged_workspace(name: str, cache, desc) -> torch.Tensor:
    n = C.c_size_t()
    _check(getattr(lib(), name)(C.byref(cache.struct), C.byref(desc), C.byref(n)), name)
    return _workspace(n.value, cache.device)


def paged_append_desc(k_new, v_new, scores=None) -> _abi.sa_paged_append_desc:
    """Descriptor from k_new, v_new [n_tokens, Hkv, d] and scores (or None)."""
    _need(k_new.dim() == 3 and k_new.shape == v_new.shape and k_new.dtype == v_new.dtype
          and k_new.stride(2) == 1 and v_new.stride(2) == 1,
          "k_new and v_new must be [n_tokens, Hkv, d] of one type, head_dim contiguous")
    return _abi.sa_paged_append_desc(
        dtype=_paged_dtype(k_new), n_tokens=k_new.shape[0], k_strides=(i64 * 2)(*k_new.stride()[:2]),
        v_strides=(i64 * 2)(*v_new.stride()[:2]), score_strides=_score_strides(scores))


def paged_append_workspace(cache: PagedCache, adesc) -> torch.Tensor:
    return _paged_workspace("sa_paged_append_workspace_size", cache, adesc)


def sa_paged_append(cache: PagedCache, adesc, k_new, v_new, cu_new, scores, ws, stream=None) -> None:
    _call_on(cache, stream, "sa_paged_append", C.byref(adesc), k_new.data_ptr(), v_new.data_ptr(),
             _ptr(cu_new), _ptr(scores), ws.data_ptr(), ws.numel())


def paged_append(cache: PagedCache, k_new, v_new, cu_new=None, scores=None, stream=None) -> None:
    """Writes k_new, v_new [n_tokens, Hkv, d] to the last positions of their
    sequences: rows cu_new[s] .. cu_new[s+1] - 1 (int32 [n_seq + 1] on the
    device) belong to sequence s, whose seq_lens entry counts them already; with
    cu_new None row s is the one new token of sequence s. scores (fp32 [n_seq,
    Hkv, >= capacity]) are zeroed at the new positions."""
    _need(tuple(k_new.shape[1:]) == (cache.num_kv_heads, cache.head_dim),
          f"k_new and v_new must be [n_tokens, {cache.num_kv_heads}, {cache.head_dim}]")
    if cu_new is not None:
        _need(cu_new.dtype == torch.int32 and cu_new.shape == (cache.n_seq + 1,)
              and cu_new.is_contiguous(), "cu_new must be contiguous int32 [n_seq + 1]")
    if scores is not None:
        _check_scores(cache, scores, cache.capacity)
    _on_device(cache.device, *cache.tensors, k_new, v_new, cu_new, scores, stream=stream)
    ad = paged_append_desc(k_new, v_new, scores)
    with _alloc_on(cache.device, stream):
        ws = paged_append_workspace(cache, ad)
    sa_paged_append(cache, ad, k_new, v_new, cu_new, scores, ws, stream)
    paged_append.last_workspace = ws


def paged_decode_desc(q, o, window: int = 0, sinks: int = 0, softmax_scale: float = 0.0,
                      scores=None, keep_tail: bool = False) -> _abi.sa_paged_decode_desc:
    """Descriptor from q, o [n_seq, Hq, d] and scores (None: not accumulated).
    keep_tail: see sa_paged_decode_desc."""
    _need(q.dim() == 3 and q.shape == o.shape and q.dtype == o.dtype and q.stride(2) == 1
          and o.stride(2) == 1, "q and o must be [n_seq, Hq, d] of one type, head_dim contiguous")
    return _abi.sa_paged_decode_desc(
        dtype=_paged_dtype(q), num_q_heads=q.shape[1], window=window, sinks=sinks,
        accumulate=int(scores is not None), softmax_scale=softmax_scale,
        q_strides=(i64 * 2)(*q.stride()[:2]), o_strides=(i64 * 2)(*o.stride()[:2]),
        score_strides=_score_strides(scores), keep_tail=int(keep_tail))


def paged_decode_workspace(cache: PagedCache, ddesc) -> torch.Tensor:
    return _paged_workspace("sa_paged_decode_workspace_size", cache, ddesc)


def sa_paged_decode(cache: PagedCache, ddesc, q, o, lse, scores_in, scores_out, ws,
                    stream=None) -> None:
    _call_on(cache, stream, "sa_paged_decode", C.byref(ddesc), q.data_ptr(), o.data_ptr(),
             lse.data_ptr(), _ptr(scores_in), _ptr(scores_out), ws.data_ptr(), ws.numel())


def paged_decode(cache: PagedCache, q, window: int = 0, sinks: int = 0, softmax_scale: float = 0.0,
                 scores=None, scores_out=None, stream=None, keep_tail: bool = True):
    """(o [n_seq, Hq, d] of q's type, lse fp32 [n_seq, Hq]): attention of one
    token per sequence over all of its cache, or over the first `sinks` and the
    last `window` positions. scores (fp32 [n_seq, Hkv, >= capacity]): each
    position's weights, summed over the heads of its group, are added to them in
    place; scores_out receives the sums of the positions below each sequence's
    length instead, and behind it stays as it was, or with keep_tail False
    receives scores too, up to the cache's capacity."""
    _need(q.dim() == 3 and q.shape[0] == cache.n_seq and q.shape[2] == cache.head_dim,
          f"q must be [{cache.n_seq}, Hq, {cache.head_dim}]")
    _need(scores is not None or scores_out is None, "scores_out needs scores")
    if scores is not None:
        scores_out = scores if scores_out is None else scores_out
        for t in (scores, scores_out):
            _check_scores(cache, t, cache.capacity)
        _need(scores.stride() == scores_out.stride(), "scores_out must have the strides of scores")
    _on_device(cache.device, *cache.tensors, q, scores, scores_out, stream=stream)
    with _alloc_on(cache.device, stream):
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        dd = paged_decode_desc(q, o, window, sinks, softmax_scale, scores, keep_tail)
        ws = paged_decode_workspace(cache, dd)
    sa_paged_decode(cache, dd, q, o, lse, scores, scores_out, ws, stream)
    paged_decode.last_workspace = ws
    return o, lse


def cache_evict_desc(scores, budget: int, sinks: int = 0, recent: int = 0, dst_table=None,
                     scores_out=None) -> _abi.sa_evict_desc:
    """Descriptor; dst_table None: in place, scores_out None: scores itself."""
    if dst_table is not None:
        _need(dst_table.dtype == torch.int32 and dst_table.dim() == 2 and dst_table.stride(1) == 1,
              "dst_table must be int32 [n_seq, pages], rows contiguous")
    return _abi.sa_evict_desc(
        budget=budget, sinks=sinks, recent=recent,
        dst_max_pages=0 if dst_table is None else dst_table.shape[1],
        dst_table_stride=0 if dst_table is None else _table_stride(dst_table),
        score_strides=_score_strides(scores),
        out_strides=_score_strides(scores if scores_out is None else scores_out))


def cache_evict_workspace(cache: PagedCache, edesc) -> torch.Tensor:
    return _paged_workspace("sa_cache_evict_workspace_size", cache, edesc)


def sa_cache_evict(cache: PagedCache, edesc, scores_in, dst_table, keep, scores_out, lens_out, ws,
                   stream=None) -> None:
    _call_on(cache, stream, "sa_cache_evict", C.byref(edesc), scores_in.data_ptr(), _ptr(dst_table),
             keep.data_ptr(), scores_out.data_ptr(), lens_out.data_ptr(), ws.data_ptr(), ws.numel())


def cache_evict(cache: PagedCache, scores, budget: int, sinks: int = 0, recent: int = 0,
                dst_table=None, scores_out=None, lens_out=None, stream=None) -> torch.Tensor:
    """Keeps the first `sinks`, the last `recent` and the highest-scored other
    positions of each (sequence, key/value head), `budget` in all, and moves
    them, in order, to the front: in place (scores and cache.seq_lens too), or
    to the pages of dst_table, scores_out and lens_out. Returns the kept
    positions, int32 [n_seq, Hkv, budget], ascending, -1 padded."""
    _check_scores(cache, scores, cache.capacity)
    if scores_out is not None:
        _check_scores(cache, scores_out, min(budget, cache.capacity))
    if dst_table is not None:
        _need(dst_table.shape[:1] == (cache.n_seq,), f"dst_table must have {cache.n_seq} rows")
    scores_to = scores if scores_out is None else scores_out
    lens_to = cache.seq_lens if lens_out is None else lens_out
    _need(lens_to.dtype == torch.int32 and lens_to.shape == (cache.n_seq,) and lens_to.is_contiguous(),
          "lens_out must be contiguous int32 [n_seq]")
    _on_device(cache.device, *cache.tensors, scores, dst_table, scores_to, lens_to, stream=stream)
    ed = cache_evict_desc(scores, budget, sinks, recent, dst_table, scores_to)
    with _alloc_on(cache.device, stream):
        ws = cache_evict_workspace(cache, ed)
        keep = torch.empty(cache.n_seq, cache.num_kv_heads, budget, dtype=torch.int32,
                           device=cache.device)
    sa_cache_evict(cache, ed, scores, dst_table, keep, scores_to, lens_to, ws, stream)
    cache_evict.last_workspace = ws
    return keep


def selftest_wait_timeout(n_ctas: int = 8, device="cuda", stream=None):
    """Runs the device failure-path self-test (about 4 s; a test-only export of
    the library, declared outside the public header); returns (status code,
    location) read from the status word after the stream synchronises."""
    ws = _workspace(256, device)
    _check(lib().sa_selftest_wait_timeout(_ptr(ws), ws.numel(), n_ctas, _stream(stream)),
           "sa_selftest_wait_timeout")
    torch.cuda.synchronize(ws.device)
    code, where = ws[:8].view(torch.int32).cpu().tolist()
    return code, where


def device_status(ws: torch.Tensor | None, stream=None) -> int:
    """The device status word of a workspace an earlier call used (None: the
    fixed scratch array of the allocation-free decode on the current device).
    Synchronises the stream."""
    st = C.c_int()
    _check(lib().sa_get_device_status(_ptr(ws), _stream(stream), C.byref(st)),
           "sa_get_device_status")
    return st.value
