"""Attention over a paged key/value cache, and the cache's operations (libfa's
fa_fwd_paged, fa_cache_append, fa_cache_commit and fa_cache_fork).

A cache is two tensors k_cache and v_cache, (pages, Hkv, page_size, D) of one
layer or (layers, pages, Hkv, page_size, D) of all (any strides with D
contiguous, so (pages, page_size, Hkv, D) storage works as a transposed view);
a block table (Z, max_pages) int32 names the page of every page_size positions
of each sequence, -1 where it has none; seq_lens (Z) int32 holds the positions
that each sequence has.  One step of speculative decoding:

    fa_cache_fork(k, v, table, lens, refs, source, room=T, missing=missing, all_or_nothing=True)  # room for T more
    for layer in ...:
        fa_cache_append(k_new, v_new, k[layer], v[layer], table, lens, new_lens=new)
        o, lse = fa_fwd_paged(q, k[layer], v[layer], table, lens, new_lens=new, tree_mask=mask)
    fa_cache_commit(k, v, table, lens, accepted, accepted_lens)               # all layers
    lens += accepted_lens

If missing is not 0 the fork has changed nothing: free sequences and fork again.
new is T for every sequence that goes on; one that has ended keeps source -1, new
0 and accepted_lens 0 until it is used again (it has no pages, and a row for it
would be recorded as FA_ERR_PAGE).

Everything is argument marshalling: the work, the lengths and the page
bookkeeping stay on the device, and no call synchronises.
"""
from __future__ import annotations

import ctypes
import importlib.util

from . import _binding
from .build import EXT as _EXT
from ._binding import FA_OK, FaError

_ext = None      # the extension that marshals the calls (csrc/paged_ext.cpp)
_bound = None    # the build of libfa that it calls


def _calls():
    """The extension, bound to the loaded build of libfa; raises ImportError if either is not built."""
    global _ext, _bound
    lib = _binding._lib or _binding.load()
    if lib is not _bound:
        if _ext is None:
            import torch  # noqa: F401  (the extension's symbols)

            spec = importlib.util.spec_from_file_location("_paged_ext", _EXT)
            try:
                ext = importlib.util.module_from_spec(spec)
            except ImportError as e:
                raise ImportError(f"the paged-cache binding is not built ({_EXT}); run "
                                  "`python -m exact_attention_44_gb300.build`") from e
            spec.loader.exec_module(ext)
            _ext = ext
        names = ("fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_cache_append", "fa_cache_commit", "fa_cache_fork",
                 "fa_cache_fork_workspace_size", "fa_rope", "fa_cache_append_rope", "fa_cache_score",
                 "fa_cache_score_workspace_size", "fa_cache_evict", "fa_cache_evict_workspace_size")
        _ext.bind(FaError, *[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names])
        _bound = lib
    return _ext


def fa_fwd_paged_workspace_size(D: int, device=None) -> int:
    """Workspace bytes fa_fwd_paged needs for head dim D on `device` (default: current)."""
    import torch

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
    positions.  Tokens that see nothing or do not exist get o = 0, lse = -inf
    (what q holds for the latter does not matter).  Sums are fp32; the
    probabilities are cast to the input type before the product with V, as in
    fa_fwd.
    workspace: a CUDA uint8 tensor of fa_fwd_paged_workspace_size(D) bytes;
    one is allocated when omitted.  Returns (o, lse), lse (Z, Hq, T) fp32 or
    None, without synchronising.
    """
    ext = _ext if _bound is not None and _bound is _binding._lib else _calls()
    return ext.fwd_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, new_lens, tree_mask, scale, workspace,
                         None if stream is None else stream.cuda_stream, want_lse)


def fa_cache_append(k, v, k_cache, v_cache, block_table, seq_lens, *, new_lens=None, stream=None) -> None:
    """Write new rows into one layer's cache (libfa's fa_cache_append).

    k, v: (Z, Hkv, T, D) of the cache's dtype, any strides with D contiguous;
    row (z, :, t) goes to position seq_lens[z] + t for t < new_lens[z] (default
    T).  seq_lens is not changed.
    """
    ext = _ext if _bound is not None and _bound is _binding._lib else _calls()
    ext.cache_append(k, v, k_cache, v_cache, block_table, seq_lens, new_lens,
                     None if stream is None else stream.cuda_stream)


def fa_cache_commit(k_cache, v_cache, block_table, seq_lens, accepted, accepted_lens, *, stream=None) -> None:
    """Keep the accepted ones of the drafted tokens (libfa's fa_cache_commit).

    Position seq_lens[z] + accepted[z, i] moves to seq_lens[z] + i, for i <
    accepted_lens[z], in every layer of the caches ((layers, pages, Hkv,
    page_size, D), or one layer without the first dimension).  accepted: (Z, A)
    int32, strictly increasing within accepted_lens[z]; accepted_lens: (Z)
    int32.  seq_lens is not changed: add accepted_lens to it.
    """
    ext = _ext if _bound is not None and _bound is _binding._lib else _calls()
    ext.cache_commit(k_cache, v_cache, block_table, seq_lens, accepted, accepted_lens,
                     None if stream is None else stream.cuda_stream)


def fa_cache_fork_workspace_size(Z: int, max_pages: int) -> int:
    """Workspace bytes fa_cache_fork needs (host only)."""
    n = ctypes.c_size_t(0)
    rc = _binding.load().fa_cache_fork_workspace_size(int(Z), int(max_pages), ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_cache_fork_workspace_size")
    return n.value


def fa_cache_fork(k_cache, v_cache, block_table, seq_lens, ref_counts, source=None, *, room: int = 0, missing=None,
                  workspace=None, stream=None, all_or_nothing: bool = False) -> None:
    """Fork, free and give room to the sequences of a cache, in place (libfa's fa_cache_fork).

    source: (Z) int32, which sequence (as it was before the call) each one
    becomes a copy of -- itself: it stays; -1: it is emptied and its pages
    released; None: all stay.  Copies share full pages (ref_counts, (pages)
    int32, counts the table entries of a page; 0 is free) and get their own copy
    of the partly filled one, in every layer of the caches.  Then every sequence
    that is not emptied gets pages for `room` more positions.  missing: (1)
    int32, receives how many pages lacked (0: none).  all_or_nothing: if pages
    lack nothing is changed, so that sequences can be freed and the same call made
    again (it needs `missing`); otherwise the call does what it can, and a copy
    whose partly filled page lacked has lost the rows in it (`missing` counts it in
    every later call, until it is replaced or emptied).  workspace: a CUDA uint8
    tensor of fa_cache_fork_workspace_size(Z, max_pages) bytes; one is allocated
    when omitted.
    """
    ext = _ext if _bound is not None and _bound is _binding._lib else _calls()
    ext.cache_fork(k_cache, v_cache, block_table, seq_lens, ref_counts, source, room, missing, workspace,
                   None if stream is None else stream.cuda_stream, all_or_nothing)
