"""Rotary positions, and a paged cache that is held to a budget (libfa's fa_rope,
fa_cache_append_rope, fa_cache_score and fa_cache_evict).

A model keeps the frequencies of its rotary positions as turns, on the host:

    turns = fa_rope_turns(fa_rope_frequencies(rotary_dim))
    q, k = fa_rope(q, k, turns)                       # or rotary(...), with autograd

A decode step over a cache of at most budget + slack positions a sequence (pages and
lengths as for the other fa_cache_* calls; positions: how many tokens each sequence has
seen, which runs ahead of seq_lens once positions have been evicted):

    fa_cache_fork(k, v, table, lens, refs, source, room=1, missing=missing, all_or_nothing=True)
    for i in range(layers):
        qi = fa_cache_append_rope(q[i], k_new[i], v_new[i], k[i], v[i], table, lens, turns,
                                  positions=positions[:, None])
        o, lse = fa_fwd_paged(qi, k[i], v[i], table, lens)
        fa_cache_score(qi, lse, k[i], table, lens, scores[i])
    lens += 1
    positions += 1
    fa_cache_evict(k, v, table, lens, refs, scores, budget, missing, keep=keep)   # now and then

A sequence's scores follow it only where the caller moves them: after a fork that gives
sequence z the cache of another, scores[:, z] = scores[:, source[z]].  Everything is
argument marshalling, and no call synchronises.
"""
from __future__ import annotations

import ctypes

from . import _binding, paged
from ._binding import FA_OK, FaError

_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}


class _Scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int)] + [(n, ctypes.c_double) for n in ("base", "stretch", "context", "slow", "fast")]


def _calls():
    return paged._ext if paged._bound is not None and paged._bound is _binding._lib else paged._calls()


def fa_rope_frequencies(rotary_dim: int, *, base: float = 10000.0, scaling: str = "none", stretch: float = 1.0,
                        context: float = 0.0, slow: float = 1.0, fast: float = 32.0):
    """Radians a position of each of rotary_dim / 2 pairs, base^(-2 i / rotary_dim): a float64 tensor on the host.

    scaling, for a context `stretch` times as long as the one the frequencies were made
    for: "none"; "linear" (all divided by stretch); "base" (base times
    stretch^(rotary_dim / (rotary_dim - 2))); "ramp" (pairs that turn at most `slow` times
    over `context` positions divided by stretch, those that turn at least `fast` times as
    they are, linear in the number of turns between).
    """
    import torch

    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}, got {scaling!r}")
    if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > 1 << 20:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    out = torch.empty(rotary_dim // 2, dtype=torch.float64)
    s = _Scaling(_SCALINGS[scaling], base, stretch, context, slow, fast)
    rc = _binding.load().fa_rope_frequencies(int(rotary_dim), ctypes.addressof(s), out.data_ptr())
    if rc != FA_OK:
        raise FaError(rc, "fa_rope_frequencies")
    return out


def fa_rope_turns(inv_freq):
    """The frequencies (radians a position, a 1-D tensor) as fa_rope takes them: an int64 tensor on the host.

    Turns a position in units of 2^-64, which wrap after a whole turn, so that angles keep
    their precision at any position.  Made once for a model; calls pass them on as launch
    arguments.
    """
    import torch

    f = inv_freq.detach().to(device="cpu", dtype=torch.float64).contiguous()
    if f.dim() != 1:
        raise ValueError(f"inv_freq must be 1-D, got {tuple(f.shape)}")
    out = torch.empty(f.shape, dtype=torch.int64)
    rc = _binding.load().fa_rope_turns(f.numel(), f.data_ptr(), out.data_ptr())
    if rc != FA_OK:
        raise FaError(rc, "fa_rope_turns")
    return out


def fa_rope(q, k, turns, positions=None, *, interleaved: bool = False, inverse: bool = False, factor: float = 1.0,
            q_out=None, k_out=None, stream=None):
    """Turn the rows of q (Z, Hq, N, D) and k (Z, Hk, N, D; or None) by their positions (libfa's fa_rope).

    turns: int64 (rotary_dim / 2), from fa_rope_turns: the first rotary_dim elements of a
    row are pairs (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved; the rest
    stays.  positions: int32 (N) for all sequences or (Z, N); default 0 .. N - 1.  factor
    multiplies the turned elements.  inverse turns back (the gradient).  fp16 or bf16, any
    strides with D contiguous; fp32 arithmetic, rounded once.  q_out and k_out may be q and
    k themselves.  Returns (q_out, k_out), new tensors in the inputs' layout when omitted.
    """
    return _calls().rope(q, k, turns, positions, interleaved, inverse, factor, q_out, k_out,
                         None if stream is None else stream.cuda_stream)


def fa_cache_append_rope(q, k, v, k_cache, v_cache, block_table, seq_lens, turns, *, positions=None, new_lens=None,
                         interleaved: bool = False, factor: float = 1.0, q_out=None, stream=None):
    """fa_cache_append with rotary positions (libfa's fa_cache_append_rope): one launch for q, k and v.

    q (Z, Hq, T, D), k and v (Z, Hkv, T, D) of the new tokens, before their turn; k rows go
    turned, v rows unchanged to slots seq_lens[z] + t of the cache for t < new_lens[z]
    (default T), and q rows turned to q_out (may be q).  positions: int32 (T) or (Z, T),
    default the slots' own.  Returns q_out (a new tensor when omitted; its rows of tokens t
    >= new_lens[z] are not written).  seq_lens is not changed.
    """
    return _calls().cache_append_rope(q, k, v, k_cache, v_cache, block_table, seq_lens, turns, positions, new_lens,
                                      interleaved, factor, q_out, None if stream is None else stream.cuda_stream)


def fa_cache_score_workspace_size(device=None) -> int:
    """Workspace bytes fa_cache_score needs on `device` (default: current)."""
    import torch

    n = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = _binding.load().fa_cache_score_workspace_size(ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_cache_score_workspace_size")
    return n.value


def fa_cache_score(q, lse, k_cache, block_table, seq_lens, scores, *, new_lens=None, scale: float | None = None,
                   decay: float = 1.0, workspace=None, stream=None) -> None:
    """Add to scores the attention weight that each cached position receives from the new tokens (libfa's fa_cache_score).

    q (Z, Hq, T, D) as fa_fwd_paged took it and lse (Z, Hq, T) as it left it, with the same
    seq_lens, new_lens, scale and one layer's k_cache; new token t sees positions up to
    seq_lens[z] + t.  scores: float32 (Z, Hkv, >= max_pages * page_size):
    scores[z, hk, j] = decay * scores[z, hk, j] + the sum of exp(q k_j scale - lse) over
    the tokens and the heads of the group that see j; positions from seq_lens[z] on had no
    score yet, and with decay 0 none had.  With drafted tokens call it after
    fa_cache_commit, with the rows of the accepted ones.  workspace: a CUDA uint8 tensor of
    fa_cache_score_workspace_size() bytes; one is allocated when omitted.
    """
    _calls().cache_score(q, lse, k_cache, block_table, seq_lens, scores, new_lens, scale, decay, workspace,
                         None if stream is None else stream.cuda_stream)


def fa_cache_evict_workspace_size(L: int, Z: int, Hkv: int, max_pages: int, budget: int) -> int:
    """Workspace bytes fa_cache_evict needs (host only)."""
    n = ctypes.c_size_t(0)
    rc = _binding.load().fa_cache_evict_workspace_size(int(L), int(Z), int(Hkv), int(max_pages), int(budget),
                                                       ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_cache_evict_workspace_size")
    return n.value


def fa_cache_evict(k_cache, v_cache, block_table, seq_lens, ref_counts, scores, budget: int, missing, *, keep=None,
                   first: int = 0, recent: int = 0, workspace=None, stream=None) -> None:
    """Cut the sequences of a cache back to their best positions, in place (libfa's fa_cache_evict).

    Sequence z, if it has more than n = min(budget, keep[z]) positions (keep: int32 (Z),
    negative: it stays as it is; default: budget for all), keeps n: in each layer and kv
    head the first `first`, the last `recent` and of the others those with the highest
    scores (float32 (layers, Z, Hkv, >= max_pages * page_size), without the first dimension
    for a cache of one layer; ties: the lowest position).  They keep their order, their
    scores move along, seq_lens[z] becomes n, and pages behind are released.  Shared pages
    that would be written are replaced by free ones; missing, (1) int32, receives how many
    lacked: if it is not 0 nothing else has changed; then cut in several calls, through
    keep: the sequences that share nothing first, the others one by one.  Every row behind
    the first one that goes moves, so cut by many positions now and then, not by one every
    step.  workspace: a CUDA uint8 tensor of fa_cache_evict_workspace_size(layers, Z, Hkv,
    max_pages, budget) bytes; one is allocated when omitted.
    """
    _calls().cache_evict(k_cache, v_cache, block_table, seq_lens, ref_counts, scores, budget, missing, keep, first, recent,
                         workspace, None if stream is None else stream.cuda_stream)
