"""The plain statement of fork with lost tails agrees with the other one where no tail has been lost, and
keeps every row of an all-or-nothing run; the flag of such a call is checked."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_44_gb300 as fa
import fork_util as fu
import paged_util as pu
from test_paged_host import PTR, Fork, _cache


def test_statements_agree_and_whole_calls_keep_the_state_valid():
    r = np.random.RandomState(1)
    page, P, Z, M = 16, 30, 6, 8
    table, lens, refs = [[-1] * M for _ in range(Z)], [0] * Z, [0] * P
    refused = 0
    for _ in range(300):
        source = [int(r.choice([z, z, r.randint(Z), -1])) for z in range(Z)]
        room = int(r.randint(0, 40))
        assert fu.fork(table, lens, refs, source, room, page) == pu.fork(table, lens, refs, source, room, page)
        before = (table, lens, refs)
        table, lens, refs, missing, tails = fu.fork(table, lens, refs, source, room, page, True)
        if missing:
            refused += 1
            assert (table, lens, refs) == before and not tails
        assert np.bincount([p for t in table for p in t if p >= 0], minlength=P).tolist() == refs
        for z in range(Z):
            held = sum(p >= 0 for p in table[z])
            assert all(p >= 0 for p in table[z][:pu.cdiv(lens[z], page)])
            lens[z] = min(held * page, lens[z] + int(r.randint(0, room + 1)))
    assert 20 < refused < 280


class ForkWhole(ctypes.Structure):
    _fields_ = Fork._fields_ + [("all_or_nothing", ctypes.c_int)]


def test_flag_is_refused_unless_0_or_1_and_reads_as_off_where_it_is_not_set():
    fa.build()
    lib = fa.load()
    # (the flag takes the place of padding: a zeroed structure without it has the same size and reads as 0)
    assert ctypes.sizeof(ForkWhole) == ctypes.sizeof(Fork) and ForkWhole.all_or_nothing.offset == Fork.room.offset + 4
    for flag, miss, code in ((2, PTR, fa.FA_ERR_INVALID_ARG), (-1, PTR, fa.FA_ERR_INVALID_ARG),
                             (0, PTR, fa.FA_ERR_WORKSPACE), (0, None, fa.FA_ERR_WORKSPACE),
                             (1, PTR, fa.FA_ERR_WORKSPACE), (1, None, fa.FA_ERR_INVALID_ARG)):
        x = ForkWhole(cache=_cache(), refs=PTR, src=PTR, miss=miss, ws=None, all_or_nothing=flag)
        assert lib.fa_cache_fork(ctypes.addressof(x), None) == code
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros(9, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="all_or_nothing needs missing"):
        fa.fa_cache_fork(cache, cache, z(2, 4), z(2), z(9), all_or_nothing=True)
