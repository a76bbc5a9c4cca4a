"""Attention over a paged key/value cache, and the cache's operations (libfa's
fa_fwd_paged, fa_cache_append, fa_cache_commit and fa_cache_fork).

A cache is two tensors k_cache and v_cache, (pages, Hkv, page_size, D) of one
layer or (layers, pages, Hkv, page_size, D) of all (any strides with D
contiguous, so (pages, page_size, Hkv, D) storage works as a transposed view);
a block table (Z, max_pages) int32 names the page of every page_size positions
of each sequence, -1 where it has none; seq_lens (Z) int32 holds the positions
that each sequence has.  One step of speculative decoding:

    fa_cache_fork(k, v, table, lens, refs, room=T, missing=missing)   # pages for T more positions
    for layer in ...:
        fa_cache_append(k_new, v_new, k[layer], v[layer], table, lens)
        o, lse = fa_fwd_paged(q, k[layer], v[layer], table, lens, tree_mask=mask)
    fa_cache_commit(k, v, table, lens, accepted, accepted_lens)       # all layers
    lens += accepted_lens

Everything is argument marshalling: the work, the lengths and the page
bookkeeping stay on the device, and no call synchronises.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _binding
from ._binding import FA_DTYPE_BF16, FA_DTYPE_F16, FA_OK, FaError

# A decode step makes one or two of these calls a layer, each a few microseconds of GPU time, so the
# marshalling itself is kept short: torch is looked up once, a call's argument block (the structures
# of include/fa.h) is packed in one step, and the stream's handle comes from the call that torch's own
# launches use.
_CACHE = "@2P8q2qPqP7i4x"  # fa_paged_cache
_ATTEND = struct.Struct(_CACHE + "3P8q2PqPN2ifi").pack
_APPEND = struct.Struct(_CACHE + "2P8qPi4x").pack
_COMMIT = struct.Struct(_CACHE + "PqPi4x").pack
_FORK = struct.Struct(_CACHE + "4PNi4x").pack

torch = None
_int32 = _raw_stream = _get_device = None


def _setup():
    global torch, _int32, _raw_stream, _get_device
    import torch as t

    _int32 = t.int32
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: t.cuda.current_stream(index).cuda_stream)
    _get_device = t.cuda.current_device
    torch = t


def _ints(name, t, shape):
    if t.dtype is not _int32:
        raise TypeError(f"{name} must be int32")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _cache(k_cache, v_cache, block_table, seq_lens, Z, layers):
    """The fields of a fa_paged_cache, checked; layers: whether 5-D caches are allowed."""
    shape = k_cache.shape
    n = len(shape)
    if shape != v_cache.shape or not (n == 4 or layers and n == 5):
        want = "(pages, Hkv, page_size, D)" + (" or (layers, pages, Hkv, page_size, D)" if layers else "")
        raise ValueError(f"k_cache and v_cache must both be {want}, got {tuple(shape)}, {tuple(v_cache.shape)}")
    if k_cache.dtype is not v_cache.dtype or k_cache.element_size() != 2:
        raise TypeError("k_cache and v_cache must share one 16-bit dtype")
    if block_table.dtype is not _int32:
        raise TypeError("block_table must be int32")
    rows = block_table.shape
    if len(rows) != 2 or rows[0] != Z:
        raise ValueError(f"block_table must be (Z, max_pages) = ({Z}, ...), got {tuple(rows)}")
    M = rows[1]
    row, col = block_table.stride()
    if M > 1 and col != 1:
        raise ValueError("block_table rows must be contiguous")
    _ints("seq_lens", seq_lens, (Z,))
    ks, vs = k_cache.stride(), v_cache.stride()
    if n == 5:
        L, P, H, page, D = shape
        kl, vl, ks, vs = ks[0], vs[0], ks[1:], vs[1:]
    else:
        P, H, page, D = shape
        L, kl, vl = 1, 0, 0
    return (k_cache.data_ptr(), v_cache.data_ptr(), *ks, *vs, kl, vl, block_table.data_ptr(), row, seq_lens.data_ptr(),
            Z, L, P, H, page, D, M)


def _call(name, lead, stream, tensors, block):
    """Call libfa's `name` with its packed arguments on the device of the tensor `lead`."""
    index = lead.get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name}: every tensor must be on {lead.device}, got one on {t.device}")
    if index < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    fn = getattr(_binding._lib or _binding.load(), name)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if _get_device() == index:
        rc = fn(block, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(block, handle)
    if rc != FA_OK:
        raise FaError(rc, name)


def fa_fwd_paged_workspace_size(D: int, device=None) -> int:
    """Workspace bytes fa_fwd_paged needs for head dim D on `device` (default: current)."""
    if torch is None:
        _setup()
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = _binding.load().fa_fwd_paged_workspace_size(int(D), ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_paged_workspace_size")
    return n.value


def fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, o=None, lse=None, *, new_lens=None, tree_mask=None,
                 scale: float | None = None, workspace=None, stream=None, want_lse: bool = True):
    """Attention of the T newest tokens of every sequence over its paged cache (libfa's fa_fwd_paged).

    q: (Z, Hq, T, D) fp16 or bf16; k_cache, v_cache: (pages, Hkv, page_size, D)
    of the same dtype; block_table: (Z, max_pages) int32; seq_lens: (Z) int32,
    the positions before the new tokens, which are already in the cache behind
    them.  new_lens: (Z) int32, how many of the T new tokens a sequence has
    (default T).  tree_mask: int32 bit words, (T, ceil(T/32)) for all sequences
    or (Z, T, ceil(T/32)): bit j of token t's words says that t sees new token
    j; None is a chain (t sees 0 .. t).  Every new token sees all earlier
    positions.  Tokens that see nothing or do not exist get o = 0, lse = -inf.
    workspace: a CUDA uint8 tensor of fa_fwd_paged_workspace_size(D) bytes;
    one is allocated when omitted.  Returns (o, lse), lse (Z, Hq, T) fp32 or
    None, without synchronising.
    """
    if torch is None:
        _setup()
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be 4-D (Z, Hq, T, D)")
    Z, Hq, T, D = shape
    cache = _cache(k_cache, v_cache, block_table, seq_lens, Z, False)
    if cache[20] != D:
        raise ValueError(f"head dims differ: q has {D}, the cache {cache[20]}")
    dtype = q.dtype
    if dtype is torch.bfloat16:
        code = FA_DTYPE_BF16
    elif dtype is torch.float16:
        code = FA_DTYPE_F16
    else:
        raise TypeError(f"fa_fwd_paged takes float16 or bfloat16 tensors, got {dtype}")
    if k_cache.dtype is not dtype:
        raise TypeError("q and the caches must share one dtype")
    new_ptr = mask_ptr = lse_ptr = mask_stride = 0
    if new_lens is not None:
        _ints("new_lens", new_lens, (Z,))
        new_ptr = new_lens.data_ptr()
    if tree_mask is not None:
        words = (T + 31) // 32
        if tree_mask.dim() == 3:
            _ints("tree_mask", tree_mask, (Z, T, words))
            mask_stride = tree_mask.stride(0)
        else:
            _ints("tree_mask", tree_mask, (T, words))
        if T > 1 and tree_mask.stride(-2) != words:
            raise ValueError("tree_mask's words must be contiguous within a sequence")
        mask_ptr = tree_mask.data_ptr()
    if o is None:
        o = torch.empty(shape, dtype=dtype, device=q.device)
    elif o.shape != shape or o.dtype is not dtype:
        raise ValueError("o must match q's shape and dtype")
    if lse is None:
        if want_lse:
            lse = torch.empty((Z, Hq, T), dtype=torch.float32, device=q.device)
            lse_ptr = lse.data_ptr()
    elif lse.dtype is not torch.float32 or lse.shape != (Z, Hq, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (Z, Hq, T) tensor")
    else:
        lse_ptr = lse.data_ptr()
    if workspace is None and q.is_cuda:
        workspace = torch.empty(fa_fwd_paged_workspace_size(D, q.device), dtype=torch.uint8, device=q.device)
    _call("fa_fwd_paged", q, stream, (k_cache, v_cache, block_table, seq_lens, new_lens, tree_mask, o, lse, workspace),
          _ATTEND(*cache, q.data_ptr(), o.data_ptr(), lse_ptr, *q.stride(), *o.stride(), new_ptr, mask_ptr, mask_stride,
                  0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes, Hq, T,
                  1.0 / math.sqrt(D) if scale is None else scale, code))
    return o, lse


def fa_cache_append(k, v, k_cache, v_cache, block_table, seq_lens, *, new_lens=None, stream=None) -> None:
    """Write new rows into one layer's cache (libfa's fa_cache_append).

    k, v: (Z, Hkv, T, D) of the cache's dtype, any strides with D contiguous;
    row (z, :, t) goes to position seq_lens[z] + t for t < new_lens[z] (default
    T).  seq_lens is not changed.
    """
    if torch is None:
        _setup()
    shape = k.shape
    if len(shape) != 4 or shape != v.shape:
        raise ValueError(f"k and v must both be (Z, Hkv, T, D), got {tuple(shape)}, {tuple(v.shape)}")
    Z, H, T, D = shape
    cache = _cache(k_cache, v_cache, block_table, seq_lens, Z, False)
    if cache[18] != H or cache[20] != D:
        raise ValueError(f"k and v must both be (Z, {cache[18]}, T, {cache[20]}), got {tuple(shape)}")
    if k.dtype is not k_cache.dtype or v.dtype is not k_cache.dtype:
        raise TypeError("k and v must have the cache's dtype")
    new_ptr = 0
    if new_lens is not None:
        _ints("new_lens", new_lens, (Z,))
        new_ptr = new_lens.data_ptr()
    _call("fa_cache_append", k, stream, (v, k_cache, v_cache, block_table, seq_lens, new_lens),
          _APPEND(*cache, k.data_ptr(), v.data_ptr(), *k.stride(), *v.stride(), new_ptr, T))


def fa_cache_commit(k_cache, v_cache, block_table, seq_lens, accepted, accepted_lens, *, stream=None) -> None:
    """Keep the accepted ones of the drafted tokens (libfa's fa_cache_commit).

    Position seq_lens[z] + accepted[z, i] moves to seq_lens[z] + i, for i <
    accepted_lens[z], in every layer of the caches ((layers, pages, Hkv,
    page_size, D), or one layer without the first dimension).  accepted: (Z, A)
    int32, strictly increasing within accepted_lens[z]; accepted_lens: (Z)
    int32.  seq_lens is not changed: add accepted_lens to it.
    """
    if torch is None:
        _setup()
    if accepted.dim() != 2:
        raise ValueError("accepted must be (Z, A)")
    Z, A = accepted.shape
    _ints("accepted", accepted, (Z, A))
    _ints("accepted_lens", accepted_lens, (Z,))
    cache = _cache(k_cache, v_cache, block_table, seq_lens, Z, True)
    _call("fa_cache_commit", k_cache, stream, (v_cache, block_table, seq_lens, accepted, accepted_lens),
          _COMMIT(*cache, accepted.data_ptr(), accepted.stride(0), accepted_lens.data_ptr(), A))


def fa_cache_fork_workspace_size(Z: int, max_pages: int) -> int:
    """Workspace bytes fa_cache_fork needs (host only)."""
    n = ctypes.c_size_t(0)
    rc = _binding.load().fa_cache_fork_workspace_size(int(Z), int(max_pages), ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_cache_fork_workspace_size")
    return n.value


def fa_cache_fork(k_cache, v_cache, block_table, seq_lens, ref_counts, source=None, *, room: int = 0, missing=None,
                  workspace=None, stream=None) -> None:
    """Fork, free and give room to the sequences of a cache, in place (libfa's fa_cache_fork).

    source: (Z) int32, which sequence (as it was before the call) each one
    becomes a copy of -- itself: it stays; -1: it is emptied and its pages
    released; None: all stay.  Copies share full pages (ref_counts, (pages)
    int32, counts the table entries of a page; 0 is free) and get their own copy
    of the partly filled one, in every layer of the caches.  Then every sequence
    that is not emptied gets pages for `room` more positions.  missing: (1)
    int32, receives how many pages lacked (0: none).  workspace: a CUDA uint8
    tensor of fa_cache_fork_workspace_size(Z, max_pages) bytes; one is allocated
    when omitted.
    """
    if torch is None:
        _setup()
    if seq_lens.dim() != 1:
        raise ValueError("seq_lens must be (Z)")
    Z = seq_lens.shape[0]
    cache = _cache(k_cache, v_cache, block_table, seq_lens, Z, True)
    _ints("ref_counts", ref_counts, (cache[17],))
    source_ptr = missing_ptr = 0
    if source is not None:
        _ints("source", source, (Z,))
        source_ptr = source.data_ptr()
    if missing is not None:
        _ints("missing", missing, (1,))
        missing_ptr = missing.data_ptr()
    if workspace is None and k_cache.is_cuda:
        workspace = torch.empty(fa_cache_fork_workspace_size(Z, cache[21]), dtype=torch.uint8, device=k_cache.device)
    _call("fa_cache_fork", k_cache, stream, (v_cache, block_table, seq_lens, ref_counts, source, missing, workspace),
          _FORK(*cache, ref_counts.data_ptr(), source_ptr, missing_ptr, 0 if workspace is None else workspace.data_ptr(),
                0 if workspace is None else workspace.nbytes, int(room)))
