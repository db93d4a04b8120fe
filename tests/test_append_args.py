"""CPU: arguments of append_tokens that are refused."""
import ctypes

import pytest
import torch



def _L():
    from paged_kv_cache_57_gb300 import build
    build.build()
    from paged_kv_cache_57_gb300 import lazy_attn
    return lazy_attn


def _params(**kw):
    base = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=128, num_pool_blocks=10, max_blocks_per_seq=4)
    return _L().make_params(**{**base, **kw})


def test_lengths_in_the_place_of_tail_start():
    # but for pos itself, whose old values the call keeps in q_start
    L = _L()
    new, lens, pos, start, free, words, len_out, pos_out, q_start, cu, indptr, slots = (ctypes.c_void_p(1 << 20 | i << 12) for i in range(12))
    for l, p in ((len_out, start), (start, pos_out), (start, pos)):
        rc = L._lib.lazy_attn_append_tokens(ctypes.byref(_params()), new, lens, pos, start, free, 4, None, 16, 8, words, l, p, q_start, cu,
                                            indptr, slots, None, None)
        assert rc == L.LAZY_ERR_INVALID_ARG


def test_sums_of_more_sequences_than_the_call_has():
    # block_indptr[-1:] goes on where the call ended: an entry that the call does not write would hand blocks out twice
    L = _L()
    p, big = _params(), _params(num_seqs=3)
    z = lambda n: torch.zeros(n, dtype=torch.int32)
    args = dict(new_lens=z(2), seq_lens=z(2), pos=z(2), tail_start=z(2), free_blocks=z(9), block_words=z(8))
    t = L.AppendTables.empty(big, 5, "cpu")
    small = dict(cu_rows=t.cu_rows[:3], block_indptr=t.block_indptr[:3])
    for out in (t, t.replace(cu_rows=t.cu_rows[:3]), t.replace(block_indptr=t.block_indptr[:3])):
        with pytest.raises(ValueError, match="must have 3 entries"):
            L.append_tokens(p, **args, out=out)
    with pytest.raises(ValueError, match="CUDA"):  # on to the next check
        L.append_tokens(p, **args, out=t.replace(**small))
